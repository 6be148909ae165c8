// paged.cu -- block tables and slots from request lengths.
#include <algorithm>
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
// -- new rows, pages given back, pages taken -- place everything: the p-th page
// given back goes to free_list[n_free + p], the p-th page taken is
// free_list[top - 1 - p] with top = n_free + all pages given back.  A page or row
// finds its request by a search in the sums.
//
// Bound: a handful of dependent loads.  One launch does it all: each CTA forms the
// sums for itself -- cheaper than a second launch -- and pages and rows are shared
// out.  No CTA waits for another: a page that is given back and taken again in the
// same call is read where it comes from, the table of the request that gives it
// back, and where lengths are overwritten in place, the CTA that is done last does
// it.
// Measured on GB300: 256 requests and tokens 6.4 us; 96 requests and 50141 rows 8.0
// us (a CTA for 8192 pages or rows: 11.9); 157,000 pages given back 9.6 us; 16384
// requests, 2 of which grow, 35 us, most of it the sums.
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 1024;
constexpr int64_t kTableWork = 2048;  // pages and rows that a CTA is started for

// Sums that stop at 2^32 - 1: what goes beyond is refused whatever its size.
struct Need {
  uint32_t rows, give, take;
  static __device__ __forceinline__ uint32_t sum(uint32_t a, uint32_t b) { return a + b < a ? UINT_MAX : a + b; }
  __device__ __forceinline__ void add(const Need& o) {
    rows = sum(rows, o.rows), give = sum(give, o.give), take = sum(take, o.take);
  }
};

__device__ __forceinline__ int clamp_int(uint32_t v) { return static_cast<int>(min(v, uint32_t(INT_MAX))); }

__device__ __forceinline__ Need warp_scan(Need v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Need u{__shfl_up_sync(~0u, v.rows, o), __shfl_up_sync(~0u, v.give, o), __shfl_up_sync(~0u, v.take, o)};
    if (lane >= o) v.add(u);
  }
  return v;
}

// Sums over the threads of the block before this one; *total receives the block's.
__device__ Need block_scan(Need v, Need (&warp_sum)[32], Need* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Need upto = warp_scan(v);
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  const Need sums = warp_scan(warp_sum[lane]);
  auto from = [&](const Need& n, int w) -> Need {
    return {__shfl_sync(~0u, n.rows, w), __shfl_sync(~0u, n.give, w), __shfl_sync(~0u, n.take, w)};
  };
  *total = from(sums, 31);
  Need before = from(sums, max(warp - 1, 0));
  if (warp == 0) before = {0, 0, 0};
  Need lower{__shfl_up_sync(~0u, upto.rows, 1), __shfl_up_sync(~0u, upto.give, 1), __shfl_up_sync(~0u, upto.take, 1)};
  if (lane > 0) before.add(lower);
  __syncthreads();  // the sums are read
  return before;
}

// The last b in [lo, n) with at[b] <= p; at[lo] <= p.
__device__ __forceinline__ int owner_of(const int* at, int lo, int n, int p) {
  int hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= p) lo = mid; else hi = mid;
  }
  return lo;
}

// No pointer is __restrict__ and nothing goes through the read-only cache: lens
// and n_free may be overwritten in place.
__global__ void __launch_bounds__(kTableThreads, 1) tables_kernel(const __grid_constant__ TablesArgs a) {
  wait_for_launch_before();
  extern __shared__ int sm[];
  int* row_at = sm;              // [B + 1] new rows before each request
  int* give_at = sm + a.B + 1;   // [B] pages given back before it
  int* take_at = give_at + a.B;  // [B] pages taken before it
  auto* served = reinterpret_cast<unsigned char*>(take_at + a.B);  // [B] whether it is served
  __shared__ Need warp_sum[32];
  __shared__ int problem, taken, last;
  const int capacity = a.max_pages * a.div.d;
  const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
  const int all = tid + rank * kTableThreads, stride = ranks * kTableThreads;
  const int64_t n_free = a.n_free[0];
  if (tid == 0) problem = taken = 0;
  auto pages = [&](int n) { return a.div.quot(n + a.div.d - 1); };

  // Sums over all requests.  The first round takes it that `rows` holds the new
  // rows; where it does not, a second one leaves out those that do not fit.
  auto sound_length = [&](int64_t len, int64_t after) {
    return len >= 0 && len <= capacity && after >= 0 && after <= capacity;
  };
  Need carry{0, 0, 0};
  bool fits = true;
  for (int round = 0; round < 2; ++round) {
    carry = {0, 0, 0};
    for (int base = 0; base < a.B; base += kTableThreads) {
      const int b = base + tid;
      Need n{0, 0, 0};
      if (b < a.B) {
        const int64_t len = a.lens[b], delta = a.delta[b];
        n.rows = static_cast<uint32_t>(max(delta, int64_t(0)));
        if (sound_length(len, len + delta) && (fits || delta <= 0 || row_at[b] + delta <= a.rows)) {
          const int held = pages(static_cast<int>(len)), need = pages(static_cast<int>(len + delta));
          n.give = max(held - need, 0);
          n.take = max(need - held, 0);
        }
      }
      Need total;
      Need before = block_scan(n, warp_sum, &total);
      before.add(carry);
      if (b < a.B) {
        row_at[b] = clamp_int(before.rows);
        give_at[b] = clamp_int(before.give);
        take_at[b] = clamp_int(before.take);
      }
      carry.add(total);
    }
    if (carry.rows <= a.rows) break;
    fits = false;
  }
  if (tid == 0) row_at[a.B] = clamp_int(carry.rows);
  const int64_t top = n_free + carry.give;
  const bool sound = n_free >= 0 && top <= a.num_pages;
  __syncthreads();

  // who is served
  for (int b = tid; b < a.B; b += kTableThreads) {
    const int64_t len = a.lens[b], delta = a.delta[b], after = len + delta;
    bool ok = sound_length(len, after) && (fits || delta <= 0 || row_at[b] + delta <= a.rows);
    if (!ok) {
      if (rank == 0) atomicOr(&problem, kPagerBadLength);
    } else if (!sound) {
      ok = false;
    } else if (const int n = pages(static_cast<int>(after)) - pages(static_cast<int>(len)); n > 0) {
      if (int64_t(take_at[b]) + n <= top) {
        atomicMax(&taken, take_at[b] + n);
      } else {
        ok = false;
        if (rank == 0) atomicOr(&problem, kPagerNoPages);
      }
    }
    served[b] = ok;
  }
  __syncthreads();

  // the p-th page given back, and the p-th page taken
  auto given = [&](int p) {
    const int b = owner_of(give_at, 0, a.B, p);
    return a.table[b * a.table_row + pages(a.lens[b] + a.delta[b]) + (p - give_at[b])];
  };
  auto page_taken = [&](int p) {
    const int64_t at = top - 1 - p;
    return at < n_free ? a.free_list[at] : given(static_cast<int>(at - n_free));
  };

  // A warp has stretches of 32 * run rows, a lane every 32nd of them: it searches
  // for the first one's request and from there on for the next ones' (requests
  // without new rows may lie between), the pages of kTogether rows under way at once.
  constexpr int kTogether = 4;
  const int lane = tid & 31;
  const int run = static_cast<int>(min(int64_t(8), (a.rows + stride - 1) / stride));
  const int new_rows = row_at[a.B];
  for (int64_t base = int64_t(all - lane) * run; base < a.rows; base += int64_t(stride) * run) {
    int b = -1;
    for (int k0 = 0; k0 < run; k0 += kTogether) {
      int position[kTogether], page[kTogether];
      bool live[kTogether];
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        const int64_t r = base + 32 * (k0 + k) + lane;
        position[k] = page[k] = 0;
        live[k] = false;
        if (k0 + k < run && r < new_rows) {
          const int row = static_cast<int>(r);
          if (b < 0) b = owner_of(row_at, 0, a.B, row);
          if (row_at[b + 1] <= row) b = owner_of(row_at, b + 1, a.B, row);
          const int len = a.lens[b];
          position[k] = static_cast<int>(int64_t(len) + (row - row_at[b]));
          live[k] = served[b];
          if (live[k]) {
            const int i = a.div.quot(position[k]), held = pages(len);
            // entries of new pages are on their way into the table: take them where they come from
            page[k] = i < held ? a.table[b * a.table_row + i] : page_taken(take_at[b] + (i - held));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        const int64_t r = base + 32 * (k0 + k) + lane;
        if (k0 + k >= run || r >= a.rows) continue;
        int slot = -1;
        if (live[k]) {
          if (page[k] >= 0 && page[k] < a.num_pages)
            slot = page[k] * a.div.d + (position[k] - a.div.quot(position[k]) * a.div.d);
          else
            atomicOr(&problem, kPagerBadPage);
        }
        a.slots[r] = slot;
        a.positions[r] = position[k];
      }
    }
  }
  for (int p = all; p < taken; p += stride) {
    const int b = owner_of(take_at, 0, a.B, p);
    a.table[b * a.table_row + pages(a.lens[b]) + (p - take_at[b])] = page_taken(p);
  }
  const int give = sound ? static_cast<int>(carry.give) : 0;
  for (int p = all; p < give; p += stride) a.free_list[n_free + p] = given(p);
  for (int b = all; b <= a.B; b += stride) a.row_offsets[b] = row_at[b];

  int from = all, step = stride;
  bool writes = true;
  if (a.lens_out == a.lens || a.n_free_out == a.n_free) {  // nobody may read them any more
    __syncthreads();
    if (ranks > 1) {
      if (tid == 0) last = last_of(a.counter, ranks);
      __syncthreads();
      writes = last;
      from = tid;
      step = kTableThreads;
    }
  }
  if (writes) {
    for (int b = from; b < a.B; b += step) a.lens_out[b] = served[b] ? a.lens[b] + a.delta[b] : a.lens[b];
    if (from == 0) a.n_free_out[0] = static_cast<int>(sound ? top - taken : n_free);
  }
  __syncthreads();
  if (tid == 0) {
    const int bits = problem | (sound ? 0 : kPagerBadPage);
    if (bits) atomicOr(a.status, bits);
  }
}

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, int sms, cudaStream_t stream) {
  constexpr int kMostSeqs = 16384;
  cudaError_t e = set_smem_limit_once<tables_kernel>((3 * kMostSeqs + 1) * 4 + kMostSeqs);
  if (e != cudaSuccess) return e;
  // how many pages change hands only the device knows: at most all of the table
  const int64_t most = a.rows + std::min(int64_t(a.B) * a.max_pages, 2 * a.num_pages);
  const int ctas = static_cast<int>(std::min<int64_t>(sms, 1 + most / kTableWork));
  return launch_overlapped(tables_kernel, dim3(ctas), kTableThreads, (3 * a.B + 1) * 4 + a.B, stream, a);
}

}  // namespace jfa
