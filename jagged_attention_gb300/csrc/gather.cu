// gather.cu -- cached rows of requests read back into packed bf16 rows: bound by memory
// traffic, most of which is the rows that are written.
//
// Packed row r belongs to the request b with offsets[b] <= r < offsets[b + 1] and is
// its cached row starts[b] + r - offsets[b].  Codes times scales are exact in bf16.
//
// Split: a block has up to 32 packed rows.  Its first warp finds the requests of the first
// and last of them, 32 places of the offsets at a time, and then a lane a row's page; all
// threads then take 16 values of a row's head of K and of V at a time.
//
// Measured (GB300, 6.79 TB/s copied): 394,687 rows of 8 heads, 1.6 GB from 4 bits in 251 us,
// 6.4 TB/s; from 8 bits, 1.9 GB in 292 us, 6.5 TB/s; 32,657 rows, 171 MB from 4 bits in 33.5
// us, 5.1 TB/s; 720 rows of 4 heads in 2.2 us, which is the launch.
#include <algorithm>

#include "coded.cuh"
#include "kernels.h"
#include "paged.h"

namespace jfa {
namespace {

constexpr int kGatherThreads = 128;
constexpr int kGatherRows = 32;    // most packed rows of a block: a lane looks each up
// Pieces, of 16 values of K and V, that a block has where there are many: 1.6 GB from 4
// bits take 251 us so, with 512 pieces 259, with 256 threads and 512 pieces 263, 1024 260.
constexpr int kGatherUnits = 256;

// The last b of [0, n) with offsets[b] <= r, for two r at a time; -1 where there is none:
// 32 places at a time.  Offsets that decrease somewhere give some b of the range.
__device__ __forceinline__ void requests_of(const int32_t* offsets, int n, const int64_t (&r)[2], int (&b)[2]) {
  const int lane = threadIdx.x & 31;
  int left[2] = {n, n};
  b[0] = b[1] = 0;
  for (int step = (n + 31) / 32;; step = (step + 31) / 32) {  // as many steps for both
    bool below[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) below[i] = lane * step < left[i] && offsets[b[i] + lane * step] <= r[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int before = max(__popc(__ballot_sync(~0u, below[i])) - 1, 0);
      b[i] += before * step;
      left[i] = min(step, left[i] - before * step);
    }
    if (step == 1) break;
  }
}

template <int kBits>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherArgs a, int block_rows) {
  __shared__ int page_of[kGatherRows], row_of[kGatherRows];  // page -1: zeros, -2: the row stays as it was
  wait_for_launch_before();
  const int64_t r0 = int64_t(blockIdx.x) * block_rows;
  const int rows = static_cast<int>(min(int64_t(block_rows), a.rows - r0));
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int64_t ends[2] = {r0, r0 + rows - 1}, r = min(r0 + lane, ends[1]);
    int b[2];
    requests_of(a.offsets, a.B, ends, b);
    while (b[0] < b[1]) {  // the lane's row lies between
      const int mid = b[0] + (b[1] - b[0] + 1) / 2;
      if (a.offsets[mid] <= r)
        b[0] = mid;
      else
        b[1] = mid - 1;
    }
    const int64_t from = a.offsets[b[0]], to = a.offsets[b[0] + 1];
    int page = -2, in_page = 0;
    if (r >= from && r < to) {
      const int64_t pos = int64_t(a.starts ? a.starts[b[0]] : 0) + r - from;
      page = -1;
      if (pos < 0 || pos >= int64_t(a.max_pages) * a.div.d) {
        atomicOr(a.status, kPagerBadLength);
      } else {
        const int t = a.div.quot(static_cast<int>(pos));
        page = a.table[b[0] * a.table_row + t];
        in_page = static_cast<int>(pos) - t * a.div.d;
        if (page < 0 || page >= a.num_pages) {
          atomicOr(a.status, kPagerBadPage);
          page = -1;
        }
      }
    }
    page_of[lane] = page;
    row_of[lane] = in_page;
    if (blockIdx.x == 0 && lane == 0 && a.offsets[a.B] > a.rows) atomicOr(a.status, kPagerBadLength);
  }
  __syncthreads();
  const int runs = a.D / 16, per_row = a.Hkv * runs;
  for (int i = threadIdx.x; i < rows * per_row; i += kGatherThreads) {
    const int row = i / per_row, h = (i - row * per_row) / runs, u = i % runs;
    const int page = page_of[row];
    if (page == -2) continue;
    uint4 c[2][kBits == 16 ? 2 : 1] = {};  // 16 codes of K and of V
    int byte[2] = {};
    if (page >= 0) {
      const int64_t at = page * a.page + row_of[row] * a.row + h * a.head + u * (2 * kBits);
      const int64_t scales = page * a.scales.page + row_of[row] * a.scales.row + h * a.scales.head + (kBits == 4 ? u : 0);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const unsigned char* from = (x ? a.v : a.k) + at;
        if constexpr (kBits == 4) {
          const uint2 w = *reinterpret_cast<const uint2*>(from);
          c[x][0] = make_uint4(w.x, w.y, 0u, 0u);
        } else {
          c[x][0] = reinterpret_cast<const uint4*>(from)[0];
          if constexpr (kBits == 16) c[x][1] = reinterpret_cast<const uint4*>(from)[1];
        }
        if constexpr (kBits < 16) byte[x] = (x ? a.scales.v : a.scales.k)[scales];
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint4 lo = c[x][0], hi = c[x][kBits == 16 ? 1 : 0];
      if constexpr (kBits < 16) {
        uint32_t w[8];
        float by;
        if constexpr (kBits == 8) {
          halves_of_e4m3x4(c[x][0].x, w[0], w[1]);
          halves_of_e4m3x4(c[x][0].y, w[2], w[3]);
          halves_of_e4m3x4(c[x][0].z, w[4], w[5]);
          halves_of_e4m3x4(c[x][0].w, w[6], w[7]);
          by = power_value(byte[x]);
        } else {
          uint32_t p[4], q[4];
          halves_of_e2m1x8(c[x][0].x, p);
          halves_of_e2m1x8(c[x][0].y, q);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = p[e], w[4 + e] = q[e];
          by = scale_value(byte[x]);
        }
        lo = make_uint4(bf16_of(w[0], by), bf16_of(w[1], by), bf16_of(w[2], by), bf16_of(w[3], by));
        hi = make_uint4(bf16_of(w[4], by), bf16_of(w[5], by), bf16_of(w[6], by), bf16_of(w[7], by));
      }
      uint4* to = reinterpret_cast<uint4*>((x ? a.v_out + (r0 + row) * a.v_row : a.k_out + (r0 + row) * a.k_row) + h * a.D + 16 * u);
      to[0] = lo;
      to[1] = hi;
    }
  }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, int sms, cudaStream_t stream) {
  // As many rows to a block as have that many pieces, fewer where that would not make two
  // blocks an SM: 64 rows of 8 heads take 2.3 us so, with 16 rows a block 6.0.
  const int64_t per_row = int64_t(a.Hkv) * (a.D / 16);
  const int64_t few = a.rows / (2 * sms), many = std::max<int64_t>(1, kGatherUnits / per_row);
  const int block_rows = static_cast<int>(std::max<int64_t>(1, std::min({few, many, int64_t(kGatherRows)})));
  const dim3 grid(static_cast<unsigned>((a.rows + block_rows - 1) / block_rows));
  auto* kernel = a.bits == 8 ? gather_kernel<8> : a.bits == 4 ? gather_kernel<4> : gather_kernel<16>;
  return launch_overlapped(kernel, grid, kGatherThreads, 0, stream, a, block_rows);
}

}  // namespace jfa
