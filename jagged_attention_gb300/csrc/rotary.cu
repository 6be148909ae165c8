// rotary.cu -- rows of heads rotated by their positions, and rows written into
// the pages of a cache: one kernel, bound by memory traffic.
//
// Mathematics: pair i of a head turns by phi = position * inv_freq[i].  With
// f = inv_freq / (2 pi) in units of 2^-64, position * f in 64-bit integers is
// the angle in turns modulo 1, exact but for the one rounding of f; its upper
// 32 bits as a signed number over 2^31 are the angle over pi in [-1, 1), which
// sincospif takes, rounded to fp32: by 2^-26 turns at most, half a step of fp32
// below 1.  No range reduction in floating point, no 64-bit floats.
//
// Split: a thread has 16 values of a head -- two runs of 8, lo and hi, that hold
// both members of its 8 pairs -- and walks over the heads of its row, so that
// one sine and cosine per pair serve all heads of all tensors of the call.
// With (x[i], x[i + pairs]) lo and hi are the two members; interleaved, each run
// holds four whole pairs.  Either way the D/16 threads of a row read whole
// 128-byte lines per run.
//
// Measured (GB300, 6.67 TB/s copied): 786432 rows of 8 heads, 3.2 GB in 472 us,
// 6.84 TB/s; 17311 rows of 4 fp32 and 4 bf16 heads, 106 MB in 18.9 us, 5.6 TB/s;
// 32769 rows into pages, 268 MB in 43.7 us, 6.1 TB/s; 256 rows of 4 heads in 2.7
// us, 64 rows of 48 in 3.1 us, of which 2 us are the launch.
#include <algorithm>

#include "paged.h"
#include "sm103_ptx.cuh"

namespace jfa {
namespace {

// Blocks of 64 threads, 1024 threads an SM, the 16-byte loads of two heads under way
// in each: 64 KB an SM.  786432 rows of 8 heads take 470 us so; with four heads at
// once in half the threads 514 us, with fewer registers (1280 threads) 529 us.
constexpr int kRowThreads = 64, kBlocksPerSm = 16;
// Heads of a thread, on the average, an fp32 one counting double.  8980 rows of 32
// fp32 and 8 bf16 heads: 57 us, all heads in a thread 66; 60000 rows of 8 and 8: 115
// us and 120; 20000 rows of 16 bf16 heads: 31.4 and 34.3.  Between 6 and 16 it makes
// 3% on the average, and 12% at most: 20000 rows of 12 heads 24.1 us with 10, 26.7
// with 12.
constexpr int kHeadsAThread = 12;

// 8 values as they lie in memory.
template <bool kF32>
struct Run {
  uint4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (kF32 ? 4 : 2));
    w[0] = p[0];
    if (kF32) w[kF32 ? 1 : 0] = p[1];
  }
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + at * (kF32 ? 4 : 2));
    p[0] = w[0];
    if (kF32) p[1] = w[kF32 ? 1 : 0];
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4& q = w[kF32 ? i / 4 : 0];
      const int e = kF32 ? i % 4 : i / 2;
      const uint32_t v = e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w;
      x[i] = __uint_as_float(kF32 ? v : i % 2 ? v & 0xffff0000u : v << 16);
    }
  }
  __device__ __forceinline__ void pack(const float (&x)[8]) {
    if (kF32) {
      w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      w[kF32 ? 1 : 0] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
      w[0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
  }
};

// Heads [h0, h1) of one row of a job; `in` and `out` are the row's offsets.
// The loads of kAtOnce heads are under way together.
template <bool kInterleaved, bool kF32>
__device__ __forceinline__ void walk_heads(const RowJob& job, int D, int64_t in, int64_t out, int h0, int h1, int lo,
                                           int hi, bool turn, const float (&c)[8], const float (&s)[8]) {
  constexpr int kAtOnce = kF32 ? 1 : 2;
  for (int h = h0; h < h1; h += kAtOnce) {
    Run<kF32> a[kAtOnce], b[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (h + i < h1) {
        a[i].load(job.in, in + int64_t(h + i) * D + lo);
        b[i].load(job.in, in + int64_t(h + i) * D + hi);
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (h + i >= h1) break;
      if (turn) {
        float x[8], y[8];
        a[i].unpack(x);
        b[i].unpack(y);
        if (kInterleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = x[2 * e], q = x[2 * e + 1], v = y[2 * e], w = y[2 * e + 1];
            x[2 * e] = p * c[e] - q * s[e];
            x[2 * e + 1] = q * c[e] + p * s[e];
            y[2 * e] = v * c[4 + e] - w * s[4 + e];
            y[2 * e + 1] = w * c[4 + e] + v * s[4 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float p = x[e], q = y[e];
            x[e] = p * c[e] - q * s[e];
            y[e] = q * c[e] + p * s[e];
          }
        }
        a[i].pack(x);
        b[i].pack(y);
      }
      const int64_t to = out + (h + i) * job.out_head;
      a[i].store(job.out, to + lo);
      b[i].store(job.out, to + hi);
    }
  }
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kRowThreads, kBlocksPerSm)
rows_kernel(const __grid_constant__ RowsArgs a, int heads_per_block) {
  wait_for_launch_before();
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
      const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      sincospif(half_turns, &s[i], &c[i]);
      if (a.inverse) s[i] = -s[i];
    }
  }

  bool placed = false;  // whether the row has a slot, and where
  int page = 0, in_page = 0;
  if (a.slots) {
    const int slot = a.slots[row];
    if (slot >= a.num_slots) {
      if (u == 0) atomicOr(a.status, kPagerBadPage);
    } else if (slot >= 0) {
      page = a.div.quot(slot);
      in_page = slot - page * a.div.d;
      placed = true;
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
    if (job.scatter && !placed) continue;
    const int64_t in = row * job.in_row;
    const int64_t out = job.scatter ? page * job.out_page + in_page * job.out_row : row * job.out_row;
    if (job.f32)
      walk_heads<kInterleaved, true>(job, a.D, in, out, h0, h1, lo, hi, turning && job.rotate, c, s);
    else
      walk_heads<kInterleaved, false>(job, a.D, in, out, h0, h1, lo, hi, turning && job.rotate, c, s);
  }
}

}  // namespace

cudaError_t launch_rows(const RowsArgs& a, int sms, cudaStream_t stream) {
  if (a.rows == 0 || a.heads == 0) return cudaSuccess;
  const int64_t per_block = kRowThreads / (a.D / 16);
  const int64_t blocks = (a.rows + per_block - 1) / per_block;
  // As many threads to a row as its heads' weight over kHeadsAThread: more heads in a
  // thread even out less over the SMs, fewer form their sines too often.  Of rows too
  // few to fill the SMs (1024 threads each) the heads are dealt to more.  They are
  // dealt by their number alone: of fp32 and bf16 heads some threads have more weight.
  int64_t weight = 0;
  for (const RowJob& job : a.job) weight += int64_t(job.heads) * (job.f32 ? 2 : 1);
  const int64_t fill = int64_t(sms) * 1024 / kRowThreads;
  constexpr int64_t kMostSplit = 65535;  // the grid's second dimension
  const int split = static_cast<int>(std::min<int64_t>(
      {a.heads, kMostSplit, std::max({fill / blocks, (weight + kHeadsAThread - 1) / kHeadsAThread, int64_t(1)})}));
  const int per = (a.heads + split - 1) / split;
  const dim3 grid(static_cast<unsigned>(blocks), (a.heads + per - 1) / per);
  return launch_overlapped(a.turns.interleaved ? rows_kernel<true> : rows_kernel<false>, grid, kRowThreads, 0, stream, a,
                           per);
}

}  // namespace jfa
