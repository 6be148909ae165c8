// gather.cu -- cached rows of requests read back into packed bf16 rows.
//
// Packed row r belongs to the request b with offsets[b] <= r < offsets[b + 1] and is
// its cached row starts[b] + r - offsets[b].  Codes times scales are exact in bf16.
#include "coded.cuh"
#include "kernels.h"
#include "paged.h"

namespace jfa {
namespace {

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 16;  // packed rows of a block

// The last b of [0, n) with offsets[b] <= r, -1 where there is none: 32 places at a
// time.  Offsets that decrease somewhere give some b of the range.
__device__ __forceinline__ int request_of(const int32_t* offsets, int n, int64_t r) {
  int lo = 0, left = n;
  const int lane = threadIdx.x & 31;
  while (true) {
    const int step = (left + 31) / 32, at = lane * step;
    const int before = __popc(__ballot_sync(~0u, at < left && offsets[lo + at] <= r));
    if (before == 0) return lo - (lo == 0);  // only in the first round, if offsets do not decrease
    lo += (before - 1) * step;
    left = min(step, left - (before - 1) * step);
    if (step == 1) return lo;
  }
}

template <int kBits>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
  __shared__ int page_of[kGatherRows], row_of[kGatherRows];  // page -1: zeros, -2: the row stays as it was
  wait_for_launch_before();
  const int64_t r0 = int64_t(blockIdx.x) * kGatherRows;
  const int rows = static_cast<int>(min(int64_t(kGatherRows), a.rows - r0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = warp; i < rows; i += kGatherThreads / 32) {
    const int64_t r = r0 + i;
    const int b = request_of(a.offsets, a.B, r);
    if (lane) continue;
    int page = -2, in_page = 0;
    if (b >= 0 && r < a.offsets[b + 1]) {
      const int64_t pos = int64_t(a.starts ? a.starts[b] : 0) + r - a.offsets[b];
      page = -1;
      if (pos < 0 || pos >= int64_t(a.max_pages) * a.div.d || r < a.offsets[b]) {
        atomicOr(a.status, kPagerBadLength);
      } else {
        const int t = a.div.quot(static_cast<int>(pos));
        page = a.table[b * a.table_row + t];
        in_page = static_cast<int>(pos) - t * a.div.d;
        if (page < 0 || page >= a.num_pages) {
          atomicOr(a.status, kPagerBadPage);
          page = -1;
        }
      }
    }
    page_of[i] = page;
    row_of[i] = in_page;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.offsets[a.B] > a.rows) atomicOr(a.status, kPagerBadLength);
  __syncthreads();
  const int runs = a.D / 16, per_row = a.Hkv * runs;
  for (int i = threadIdx.x; i < rows * per_row; i += kGatherThreads) {
    const int row = i / per_row, h = (i - row * per_row) / runs, u = i % runs;
    const int page = page_of[row];
    if (page == -2) continue;
    const int64_t at = page * a.page + row_of[row] * a.row + h * a.head;
    const int64_t scales = page * a.scales.page + row_of[row] * a.scales.row + h * a.scales.head;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const unsigned char* from = (x ? a.v : a.k) + at + u * (2 * kBits);
      const uint8_t* bytes = (x ? a.scales.v : a.scales.k) + scales;
      uint32_t w[8] = {};
      if (page >= 0) {
        if constexpr (kBits == 16) {
          const uint4 lo = reinterpret_cast<const uint4*>(from)[0], hi = reinterpret_cast<const uint4*>(from)[1];
          w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
        } else if constexpr (kBits == 8) {
          const uint4 c = *reinterpret_cast<const uint4*>(from);
          const float by = power_value(*bytes);
          halves_of_e4m3x4(c.x, w[0], w[1]);
          halves_of_e4m3x4(c.y, w[2], w[3]);
          halves_of_e4m3x4(c.z, w[4], w[5]);
          halves_of_e4m3x4(c.w, w[6], w[7]);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = bf16_of(w[e], by);
        } else {
          const uint2 c = *reinterpret_cast<const uint2*>(from);
          const float by = scale_value(bytes[u]);
          uint32_t p[4], q[4];
          halves_of_e2m1x8(c.x, p);
          halves_of_e2m1x8(c.y, q);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = bf16_of(p[e], by), w[4 + e] = bf16_of(q[e], by);
        }
      }
      uint4* to = reinterpret_cast<uint4*>((x ? a.v_out + (r0 + row) * a.v_row : a.k_out + (r0 + row) * a.k_row) + h * a.D + 16 * u);
      to[0] = make_uint4(w[0], w[1], w[2], w[3]);
      to[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, int, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.rows + kGatherRows - 1) / kGatherRows));
  auto* kernel = a.bits == 8 ? gather_kernel<8> : a.bits == 4 ? gather_kernel<4> : gather_kernel<16>;
  return launch_overlapped(kernel, grid, kGatherThreads, 0, stream, a);
}

}  // namespace jfa
