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
// Measured (GB300, 6.79 TB/s copied): 394,687 rows of 8 heads, 1.6 GB from 4 bits in 240 us,
// 6.7 TB/s; from 8 bits, 1.9 GB in 279 us, 6.8 TB/s; from 16, 2.5 GB in 366 us, 6.9 TB/s; 32,657 rows, 171 MB from 4 bits in 30.5
// us, 5.6 TB/s; 720 rows of 4 heads in 2.1 us, which is the launch.
#include <algorithm>

#include "coded.cuh"
#include "kernels.h"
#include "paged.h"

namespace jfa {
namespace {

constexpr int kGatherThreads = 128;
constexpr int kGatherRows = 32;    // most packed rows of a block: a lane looks each up
// Pieces, of 16 values of K and V, that a block has where there are many: 12,000 rows of 3
// heads take 5.1 us so, with 512 pieces 5.7; 394,687 of 8 heads 240 and 241.
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
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherArgs a, int block_rows,
                                                               const __grid_constant__ PageDiv per_row, bool whole) {
  // Where a row's head 0 and its scale bytes are; codes kZeros: zeros, kLeft: the row stays as it was.
  constexpr int64_t kZeros = -1, kLeft = -2;
  __shared__ int64_t codes_at[kGatherRows], scales_at[kGatherRows];
  wait_for_launch_before();
  if (a.rows == 0) {  // launched for this alone
    if (threadIdx.x == 0 && a.offsets[a.B] > 0) atomicOr(a.status, kPagerBadLength);
    return;
  }
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
    int64_t codes = kLeft, scales = 0;
    if (r >= from && r < to) {
      const int64_t pos = int64_t(a.starts ? a.starts[b[0]] : 0) + r - from;
      codes = kZeros;
      if (pos < 0 || pos >= int64_t(a.max_pages) * a.div.d) {
        atomicOr(a.status, kPagerBadLength);
      } else {
        const int t = a.div.quot(static_cast<int>(pos)), in_page = static_cast<int>(pos) - t * a.div.d;
        const int page = a.table[b[0] * a.table_row + t];
        if (page < 0 || page >= a.num_pages) {
          atomicOr(a.status, kPagerBadPage);
        } else {
          codes = page * a.page + in_page * a.row;
          scales = page * a.scales.page + in_page * a.scales.row;
        }
      }
    }
    codes_at[lane] = codes;
    scales_at[lane] = scales;
    if (blockIdx.x == 0 && lane == 0 && a.offsets[a.B] > a.rows) atomicOr(a.status, kPagerBadLength);
  }
  __syncthreads();
  const int run_bits = a.D == 128 ? 3 : 2;  // a head's pieces
  for (int i = threadIdx.x; i < rows * per_row.d; i += kGatherThreads) {
    const int row = per_row.quot(i), place = i - row * per_row.d, h = place >> run_bits, u = place & ((1 << run_bits) - 1);
    const int64_t from_row = codes_at[row];
    if (from_row == kLeft) continue;
    uint4 c[2][kBits == 16 ? 2 : 1] = {};  // 16 codes of K and of V
    int byte[2] = {};
    if (from_row != kZeros) {
      const int64_t at = from_row + h * a.head + u * (2 * kBits);
      const int64_t scales = scales_at[row] + h * a.scales.head + (kBits == 4 ? u : 0);
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
      uint4* to = reinterpret_cast<uint4*>((x ? a.v_out + (r0 + row) * a.v_row : a.k_out + (r0 + row) * a.k_row) + 16 * place);
      if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                     "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w) : "memory");
      } else {
        to[0] = lo;
        to[1] = hi;
      }
    }
  }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, int sms, cudaStream_t stream) {
  // As many rows to a block as have that many pieces, fewer where that would not make two
  // blocks an SM: 64 rows of 8 heads take 2.3 us so, with 16 rows a block 6.0.
  const int per_row = std::max(1, a.Hkv * (a.D / 16));
  const int64_t few = a.rows / (2 * sms), many = std::max(1, kGatherUnits / per_row);
  const int block_rows = static_cast<int>(std::max<int64_t>(1, std::min({few, many, int64_t(kGatherRows)})));
  // A piece's 32 bytes go out at once where they are a sector of memory: 1.6 GB from 4 bits
  // take 240 us so, in halves 297.
  const bool whole = (reinterpret_cast<uintptr_t>(a.k_out) | reinterpret_cast<uintptr_t>(a.v_out) | 2 * a.k_row | 2 * a.v_row) % 32 == 0;
  const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, (a.rows + block_rows - 1) / block_rows)));
  auto* kernel = a.bits == 8 ? gather_kernel<8> : a.bits == 4 ? gather_kernel<4> : gather_kernel<16>;
  return launch_overlapped(kernel, grid, kGatherThreads, 0, stream, a, block_rows, make_page_div(per_row), whole);
}

}  // namespace jfa
