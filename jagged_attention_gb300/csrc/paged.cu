// paged.cu -- block tables and slots from request lengths.
#include <climits>

#include "kernels.h"
#include "paged.h"

namespace jfa {
namespace {

// ---------------------------------------------------------------------------
// Block tables and slots.
//
// Per request: pages(n) = ceil(n / page_size), held = pages(lens),
// need = pages(lens + delta).  Three prefix sums in the order of the requests
// -- new rows, pages given back, pages taken -- place everything: a page given
// back goes to free_list[n_free + give + i], the i-th page a request takes is
// free_list[top - 1 - take - i] with top = n_free + all pages given back.
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 1024;

struct Need {
  int64_t rows, give, take;
};

__device__ __forceinline__ int clamp_int(int64_t v) { return v > INT_MAX ? INT_MAX : static_cast<int>(v); }

// Inclusive sums over the block's threads; *total receives the block's sum.
__device__ Need block_scan(Need v, Need (&warp_sum)[32], Need* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r = __shfl_up_sync(~0u, v.rows, o), g = __shfl_up_sync(~0u, v.give, o),
                  t = __shfl_up_sync(~0u, v.take, o);
    if (lane >= o) v.rows += r, v.give += g, v.take += t;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  Need before{0, 0, 0}, all{0, 0, 0};
  for (int w = 0; w < kTableThreads / 32; ++w) {
    const Need s = warp_sum[w];
    if (w < warp) before.rows += s.rows, before.give += s.give, before.take += s.take;
    all.rows += s.rows, all.give += s.give, all.take += s.take;
  }
  __syncthreads();
  *total = all;
  return {v.rows + before.rows, v.give + before.give, v.take + before.take};
}

__global__ void __launch_bounds__(kTableThreads) tables_kernel(const __grid_constant__ TablesArgs a) {
  extern __shared__ int sm[];
  int* row_at = sm;              // [B + 1] first new row of each request
  int* give_at = sm + a.B + 1;   // [B] pages given back before it; -1: left as it was
  int* take_at = give_at + a.B;  // [B] pages taken before it; -1: left as it was
  __shared__ Need warp_sum[32];
  __shared__ int problem;
  const int capacity = a.max_pages * a.div.d;
  const int tid = threadIdx.x;
  if (tid == 0) problem = 0;
  __syncthreads();

  Need carry{0, 0, 0};
  for (int base = 0; base < a.B; base += kTableThreads) {
    const int b = base + tid;
    Need n{0, 0, 0};
    int64_t len = 0, after = 0;
    if (b < a.B) {
      len = a.lens[b];
      after = len + a.delta[b];
      n.rows = max(a.delta[b], 0);
    }
    Need total;
    Need rows_only{n.rows, 0, 0};
    const int64_t row_end = carry.rows + block_scan(rows_only, warp_sum, &total).rows;
    const int64_t rows_total = total.rows;
    bool ok = false;
    if (b < a.B) {
      ok = len >= 0 && len <= capacity && after >= 0 && after <= capacity &&
           (after <= len || row_end <= a.rows);
      if (ok) {
        const int held = a.div.quot(static_cast<int>(len) + a.div.d - 1);
        const int need = a.div.quot(static_cast<int>(after) + a.div.d - 1);
        n.give = max(held - need, 0);
        n.take = max(need - held, 0);
      } else {
        atomicOr(&problem, kPagerBadLength);
      }
    }
    const Need incl = block_scan({0, n.give, n.take}, warp_sum, &total);
    if (b < a.B) {
      row_at[b] = clamp_int(row_end - n.rows);
      give_at[b] = ok ? clamp_int(carry.give + incl.give - n.give) : -1;
      take_at[b] = ok ? clamp_int(carry.take + incl.take - n.take) : -1;
    }
    carry.rows += rows_total;
    carry.give += total.give;
    carry.take += total.take;
  }
  if (tid == 0) row_at[a.B] = clamp_int(carry.rows);
  __syncthreads();

  const int64_t n_free = a.n_free[0];
  const int64_t top = n_free + carry.give;
  const bool sound = n_free >= 0 && top <= a.num_pages;
  if (!sound && tid == 0) atomicOr(&problem, kPagerBadPage);

  // pages given back, a warp per request
  const int lane = tid & 31;
  if (sound) {
    for (int b = tid >> 5; b < a.B; b += kTableThreads / 32) {
      if (give_at[b] < 0 || a.delta[b] >= 0) continue;
      const int len = a.lens[b];
      const int held = a.div.quot(len + a.div.d - 1), need = a.div.quot(len + a.delta[b] + a.div.d - 1);
      for (int i = need + lane; i < held; i += 32)
        a.free_list[n_free + give_at[b] + (i - need)] = a.table[b * a.table_row + i];
    }
  }
  __syncthreads();

  // pages taken, and the new lengths
  for (int b = tid >> 5; b < a.B; b += kTableThreads / 32) {
    const int len = a.lens[b], delta = a.delta[b];
    bool ok = sound && give_at[b] >= 0;
    if (ok && delta > 0) {
      const int held = a.div.quot(len + a.div.d - 1), need = a.div.quot(len + delta + a.div.d - 1);
      if (need > held && int64_t(take_at[b]) + (need - held) > top) {
        ok = false;
        if (lane == 0) atomicOr(&problem, kPagerNoPages);
      } else {
        for (int i = held + lane; i < need; i += 32)
          a.table[b * a.table_row + i] = a.free_list[top - 1 - take_at[b] - (i - held)];
      }
    }
    __syncwarp();
    if (lane == 0 && !ok) give_at[b] = -1;  // from here on: whether the request was served
  }
  __syncthreads();

  // the lowest refused need marks where the takers stop
  if (tid == 0) {
    int64_t taken = 0;
    for (int b = 0; b < a.B; ++b) {
      if (give_at[b] < 0) continue;
      const int len = a.lens[b];
      taken += max(a.div.quot(len + a.delta[b] + a.div.d - 1) - a.div.quot(len + a.div.d - 1), 0);
    }
    a.n_free_out[0] = static_cast<int>(sound ? top - taken : n_free);
  }
  for (int64_t r = tid; r < a.rows; r += kTableThreads) {
    int slot = -1, position = 0;
    if (r < row_at[a.B]) {
      int lo = 0, hi = a.B;  // the last request whose rows begin at or before r, and has rows
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (row_at[mid] <= r) lo = mid; else hi = mid;
      }
      position = static_cast<int>(int64_t(a.lens[lo]) + (r - row_at[lo]));
      if (give_at[lo] >= 0) {
        const int i = a.div.quot(position);
        const int page = a.table[lo * a.table_row + i];
        if (page >= 0 && page < a.num_pages)
          slot = page * a.div.d + (position - i * a.div.d);
        else
          atomicOr(&problem, kPagerBadPage);
      }
    }
    a.slots[r] = slot;
    a.positions[r] = position;
  }
  for (int b = tid; b <= a.B; b += kTableThreads) a.row_offsets[b] = row_at[b];
  __syncthreads();
  for (int b = tid; b < a.B; b += kTableThreads) {
    const int len = a.lens[b];
    a.lens_out[b] = give_at[b] >= 0 ? len + a.delta[b] : len;
  }
  if (tid == 0 && problem) atomicOr(a.status, problem);
}

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream) {
  const int smem = (3 * a.B + 1) * 4;
  cudaError_t e = set_smem_limit_once<tables_kernel>((3 * 16384 + 1) * 4);
  if (e != cudaSuccess) return e;
  tables_kernel<<<1, kTableThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace jfa
