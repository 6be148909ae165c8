// rotary.cu -- rows of heads rotated by their positions, and rows written into
// the pages of a cache: one kernel, bound by memory traffic.
//
// Mathematics: pair i of a head turns by phi = position * inv_freq[i].  With
// f = inv_freq / (2 pi) in units of 2^-64, position * f in 64-bit integers is
// the angle in turns modulo 1, exact but for the one rounding of f; its upper
// 32 bits as a signed number over 2^31 are the angle over pi in [-1, 1), which
// sincospif takes.  No range reduction in floating point, no 64-bit floats.
//
// Split: a thread has 16 values of a head -- two runs of 8, lo and hi, that hold
// both members of its 8 pairs -- and walks over the heads of its row, so that
// one sine and cosine per pair serve all heads of all tensors of the call.
// With (x[i], x[i + pairs]) lo and hi are the two members; interleaved, each run
// holds four whole pairs.  Either way the D/16 threads of a row read whole
// 128-byte lines per run.
#include <algorithm>

#include "paged.h"
#include "sm103_ptx.cuh"

namespace jfa {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ void load8(const void* base, int64_t at, bool f32, float (&x)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void store8(void* base, int64_t at, bool f32, const float (&x)[8]) {
  if (f32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  }
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kRowThreads)
rows_kernel(const __grid_constant__ RowsArgs a, int heads_per_block) {
  const int units = a.D / 16;  // threads of a row: 4 or 8
  const int u = threadIdx.x % units;
  const int64_t row = int64_t(blockIdx.x) * (kRowThreads / units) + threadIdx.x / units;
  if (row >= a.rows) return;
  const int pairs = a.turns.pairs;
  const bool turning = u < pairs / 8;
  // the two runs of 8 values this thread has in every head
  const int lo = turning ? 8 * u : 2 * pairs + 16 * (u - pairs / 8);
  const int hi = turning ? lo + pairs : lo + 8;

  float c[8], s[8];
  if (turning) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = !kInterleaved ? lo + i : i < 4 ? lo / 2 + i : hi / 2 + i - 4;
      const int pos = a.positions[row * a.pos_row + a.turns.axis[pair] * a.pos_axis];
      const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * a.turns.turn[pair];
      const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
      sincospif(half_turns, &s[i], &c[i]);
      if (a.inverse) s[i] = -s[i];
    }
  }

  int64_t page_at = -1;  // offset of this row's slot for scattered jobs, in rows and pages
  int page = 0, in_page = 0;
  if (a.slots) {
    const int slot = a.slots[row];
    if (slot >= a.num_slots) {
      if (u == 0) atomicOr(a.status, kPagerBadPage);
    } else if (slot >= 0) {
      page = a.div.quot(slot);
      in_page = slot - page * a.div.d;
      page_at = 0;
    }
  }

  const int first = blockIdx.y * heads_per_block;
  const int last = min(a.heads, first + heads_per_block);
  int before = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const RowJob& job = a.job[j];
    const int h0 = max(first - before, 0), h1 = min(last - before, job.heads);
    before += job.heads;
    if (job.scatter && page_at < 0) continue;
    const int64_t in = row * job.in_row;
    const int64_t out = job.scatter ? page * job.out_page + in_page * job.out_row : row * job.out_row;
    for (int h = h0; h < h1; ++h) {
      float x[8], y[8];
      const int64_t from = in + int64_t(h) * a.D, to = out + h * job.out_head;
      load8(job.in, from + lo, job.f32, x);
      load8(job.in, from + hi, job.f32, y);
      if (turning && job.rotate) {
        if (kInterleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1], v = y[2 * i], w = y[2 * i + 1];
            x[2 * i] = p * c[i] - q * s[i];
            x[2 * i + 1] = q * c[i] + p * s[i];
            y[2 * i] = v * c[4 + i] - w * s[4 + i];
            y[2 * i + 1] = w * c[4 + i] + v * s[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float p = x[i], q = y[i];
            x[i] = p * c[i] - q * s[i];
            y[i] = q * c[i] + p * s[i];
          }
        }
      }
      store8(job.out, to + lo, job.f32, x);
      store8(job.out, to + hi, job.f32, y);
    }
  }
}

}  // namespace

cudaError_t launch_rows(const RowsArgs& a, int sms, cudaStream_t stream) {
  if (a.rows == 0 || a.heads == 0) return cudaSuccess;
  const int64_t per_block = kRowThreads / (a.D / 16);
  const int64_t blocks = (a.rows + per_block - 1) / per_block;
  const int split = 1;
  const int per = (a.heads + split - 1) / split;
  const dim3 grid(static_cast<unsigned>(blocks), (a.heads + per - 1) / per);
  if (a.turns.interleaved)
    rows_kernel<true><<<grid, kRowThreads, 0, stream>>>(a, per);
  else
    rows_kernel<false><<<grid, kRowThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

}  // namespace jfa
