// decode.cu -- attention of one new token per request over the paged cache.
//
// Mathematics: with s_t = scale q . k_t, a stretch of rows yields the running
// maximum m, the sum l = sum exp(s_t - m) and O = sum exp(s_t - m) v_t; stretches
// of one row of queries join as m = max m_i, l = sum l_i exp(m_i - m), likewise O.
// Everything but the operands of the tensor cores is fp32.  A weight goes into
// the product with V as the sum of two bf16 values (its upper half and what that
// leaves), 16 bits in all: one bf16 alone would add as much error to the output
// as its own rounding to bf16 does, and saves 0.5% of the time (9% at G = 24).
// Both are above 0 where the weight is, so that an infinite value of V stays one.
//
// Bound: every cached row is read once, 4 D bytes for 4 D G flops (G query heads
// to a key/value head), so memory bandwidth bounds it while G is small.  The
// products use mma.sync, transposed -- rows of the cache are the long side of the
// 16 x 8 tile, up to 8 query heads (16: two tiles) the short one -- which wastes
// least of the tile and leaves the cache rows in the layout that ldmatrix reads;
// tcgen05 would want 64 or 128 query rows per product.  The tensor pipe is 12%
// busy at G = 8.
//
// Split: a tile is 32 cached rows for one key/value head.  All tiles of all
// requests in the order (request, head, row) are dealt in equal contiguous shares
// to the CTAs, and a CTA's share to its warps; a warp streams its tiles by
// cp.async through a stage for K and one for V -- the next K is on its way while V
// is used, and the other way round -- over the ends of rows and requests, and
// meets no barrier on the way.  What is left at the ends of the warps' shares is
// joined in shared memory, what is left at the ends of the CTAs' shares in global
// memory by the CTA that arrives last, in the order of the shares: the same
// arguments give the same bits.  So one row of any length and thousands of short
// ones spread alike, without a schedule from the host.
//
// More than 16 query heads to a key/value head are taken in 2, 4 or 8 parts by as
// many warps side by side, which walk over the same tiles at the same pace: memory
// is read once, for the others the cache is in L2 (64 requests, 1.1 GB, 24 heads on
// each of 2: 225 us, one part after the other 340 us).
//
// Measured (GB300, 6.67 TB/s copied): 96 requests up to 32768 rows, 64 heads on 8,
// 7.2 GB in 1016 to 1048 us (by GPU), 6.9 TB/s; 128 requests of 0 to 8192 rows, 443 MB in 73 us,
// 6.1 TB/s; one request of 131072, 268 MB in 48.5 us, 5.5 TB/s; one of 300 rows in
// 6.2 us.  What is left of the middle sizes is about 2.5 us until the first rows
// arrive (lengths, table, rows: three dependent trips to memory), 3 to 6 us of
// joining, and SMs whose memory is 7% slower than others'.  128 KB of K and V in
// the stages of 8 warps measured best: with 192 KB the full cache took 1126 us for
// 1070, with 6 warps 1094 for 1064.
#include <climits>
#include <type_traits>

#include "kernels.h"
#include "paged.h"
#include "sm103_ptx.cuh"

namespace jfa {
namespace {

constexpr int kTile = 32;        // cached rows of a tile
constexpr int kDecodeWarps = 8;
constexpr int kMostHeads = 16;   // query heads that a warp holds
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, int NT>  // NT: tiles of 8 query heads
struct DecodeCfg {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kStageBytes = kTile * D * 2;  // a tile's K, or its V
  static constexpr int kOutBytes = kHeads * D * 4;   // a stretch's O
  static_assert(kOutBytes <= kStageBytes, "the stage of V holds a stretch's O when it is read");
  static constexpr int kWarpBytes = 2 * kStageBytes + kOutBytes;  // K, V, park
  static constexpr int kSmemBytes = kDecodeWarps * kWarpBytes;
  static constexpr int kCtasPerSm = D == 64 ? 2 : 1;
};

// Units of work: the n tiles of a (request, key/value head) count n units, and
// kRowUnits behind them stand for its beginning and end (256 requests up to 300
// rows: 34.6 us without, 32.5 with; 128 mixed ones 74.7 and 74.2).
constexpr int kRowUnits = 2;

// Parts of a row that one CTA joins at a time, where a row has more than three times
// as many (38 parts of 16 heads: 22.9 us, all at once 28.7; up to 24 parts it makes
// no difference).
constexpr int kGroup = 8;

// Few rows of at most this many tiles get a CTA each.  4 rows of 8 heads on 2: of 250
// 5.5 us, spread over more CTAs and joined 6.9; of 380 (12 tiles) 6.4 and 7.0; of 440
// 6.6 and 6.9, of 512 6.8 and 7.1, so that up to 16 it would gain as well, of 540 7.6
// and 7.3.
constexpr int kApartTiles = 12;

// Where a warp stands: tile t of n of (request b, key/value head and pass vh), unit
// u of all.
template <typename U>
struct Cursor {
  U u;
  int b, vh, t, n, len;
};

// A stretch that does not hold all tiles of its (request b, part x of the query
// heads): tiles [t0, t1) of n.
struct Stretch {
  int64_t u0;  // unit of its tile 0
  int b, x, t0, t1, n;  // n 0: none
};

// Sum of stretches of one row for 4 values of a head, taken up in batches.
struct Joined {
  float top = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N]) {  // ml: maximum, sum
    float up = top;
#pragma unroll
    for (int i = 0; i < N; ++i) up = fmaxf(up, ml[i].x);
    const float ref = up == -INFINITY ? 0.f : up;
    const float keep = fast_exp2(top - ref);
    sum *= keep;
    o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = fast_exp2(ml[i].x - ref);
      sum += w * ml[i].y;
      o.x += w * v[i].x, o.y += w * v[i].y, o.z += w * v[i].z, o.w += w * v[i].w;
    }
    top = up;
  }
};

template <int D, int NT>
struct DecodeShared {
  Stretch part[2 * kDecodeWarps];                 // first and last of each warp
  float m[2 * kDecodeWarps][8 * NT], l[2 * kDecodeWarps][8 * NT];
  int64_t scan_units[kDecodeWarps];
  int scan_rows[kDecodeWarps], scan_most[kDecodeWarps];
  int64_t first_unit[kDecodeWarps * 32];  // of the requests that a thread adds up
  int from[2], to[2], last[2];
};

__device__ __forceinline__ int length_of(const DecodeArgs& a, int b) {
  const int len = a.lens[b];
  return len < 0 || len > a.max_pages * a.div.d ? 0 : len;
}

__device__ __forceinline__ int tiles_of(int len) { return len / kTile + (len % kTile != 0); }

// The cache is read once a launch: its lines are the first to leave L2, before the
// lengths, tables and queries (1 to 6% of a call of 23 to 75 us).
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take, uint64_t policy) {
  const int bytes = take ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Weights p0 and p1 as hi + lo, each a pair of bf16 values: hi is cut off, lo is what
// that leaves, rounded, and at least the smallest normal number where hi is not 0 (a
// weight is 0 or normal).
__device__ __forceinline__ void split_weights(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  hi = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
  lo = pack_bf16x2(p0 - __uint_as_float(__float_as_uint(p0) & 0xffff0000u),
                   p1 - __uint_as_float(__float_as_uint(p1) & 0xffff0000u));
  uint32_t least;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(least) : "r"(hi), "r"(0x00800080u));
  asm("max.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(least));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Place of value (head, d) of a stretch's O in shared memory: the exclusive or
// sends the 32 lanes of a fragment to 32 banks and keeps runs of 8 together.
template <int D>
__device__ __forceinline__ int o_at(int head, int d) {
  return head * D + (d ^ (((head >> 1) & 3) << 3));
}

// Items dealt to takers in equal contiguous shares, the first `more` of them with one more.
template <typename U>
struct Deal {
  U per, more;
  __device__ __forceinline__ Deal(U items, int takers) : per(items / U(takers)), more(items - per * U(takers)) {}
  __device__ __forceinline__ U from(int i) const { return per * U(i) + min(U(i), more); }
  __device__ __forceinline__ int taker(U item) const {
    const U big = more * (per + 1);
    return static_cast<int>(item < big ? item / (per + 1) : more + (item - big) / per);
  }
};

// Query heads [first, first + count) of part x of all, a.parts to a key/value head:
// one where the parts are not side by side.
template <bool kSide>
__device__ __forceinline__ void heads_of(const DecodeArgs& a, int x, int* first, int* count) {
  const int kv = kSide ? x / a.parts : x, g0 = kSide ? (x - kv * a.parts) * a.part_heads : 0;
  *first = kv * a.group + g0;
  *count = kSide ? max(0, min(a.part_heads, a.group - g0)) : a.group;  // 0: more parts than heads fill
}

// 4 values of out, normalised already.
__device__ __forceinline__ void store_out4(const DecodeArgs& a, int D, int b, int head, int d, float4 o) {
  *reinterpret_cast<uint2*>(a.out + (int64_t(b) * a.H + head) * D + d) =
      make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}
// Log-sum-exp from a maximum of scores in units of log2 e and a sum of at least 1 (or
// 0 where there is no row): the hardware's log2 is off by 2^-22 up to a sum of 2, an
// error of 1.7e-7 in the result, and by two units in its last place above.
__device__ __forceinline__ float lse_of(float m, float l) { return (m + __log2f(l)) * kLn2; }
// 1 / l for such a sum, 2 units in the last place, where 0 stays 0.
__device__ __forceinline__ float inverse_of(float l) { return l == 0.f ? 0.f : __fdividef(1.f, l); }

// A finished row: normalised, with its log-sum-exp.
__device__ __forceinline__ void store_joined(const DecodeArgs& a, int D, int b, int head, int d, const Joined& s) {
  const float by = inverse_of(s.sum);
  store_out4(a, D, b, head, d, make_float4(s.o.x * by, s.o.y * by, s.o.z * by, s.o.w * by));
  if (d == 0) a.lse[int64_t(head) * a.B + b] = lse_of(s.top == -INFINITY ? 0.f : s.top, s.sum);
}

// U: unsigned type that counts all units.  32 bits hold them unless the table is
// wide enough for more; 64 bits cost 0.3 to 0.6 us.
// kSide: parts of query heads side by side.
template <int D, int NT, bool kSide, typename U>
__global__ void __launch_bounds__(kDecodeWarps * 32, DecodeCfg<D, NT>::kCtasPerSm)
decode_kernel(const __grid_constant__ DecodeArgs a) {
  using C = DecodeCfg<D, NT>;
  extern __shared__ __align__(256) unsigned char smem[];
  __shared__ DecodeShared<D, NT> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_launch_before();
  // A CTA's share is dealt to `subs` sets of `together` warps, one for each part of
  // the query heads; a line is a warp's place with those of its part in a row.
  const int passes = kSide ? a.passes : 1, vheads = a.Hkv * passes, together = kSide ? a.together : 1;
  const int sub_bits = kSide ? __ffs(kDecodeWarps / together) - 1 : __builtin_ctz(kDecodeWarps), subs = 1 << sub_bits;
  const int part = kSide ? warp & (together - 1) : 0, sub = kSide ? warp / together : warp;
  const int line = (part << sub_bits) + sub;

  // ---- units of all requests, and where this CTA's warps begin.  Up to 32 requests
  // a warp adds up by itself, a lane for each, and waits for no other warp.
  const bool few = a.B <= 32;
  const int slab = few ? 1 : (a.B + kDecodeWarps * 32 - 1) / (kDecodeWarps * 32);
  const int b_lo = min(a.B, (few ? lane : tid) * slab), b_hi = min(a.B, b_lo + slab);
  U units = 0;
  int rows = 0, most = 0, last_len = 0;  // rows: requests that have any
  for (int b = b_lo; b < b_hi; ++b) {
    last_len = length_of(a, b);
    const int n = tiles_of(last_len);
    units += n > 0 ? n + kRowUnits : 0;
    rows += n > 0;
    most = max(most, n);
  }
  U units_to = units;
  int rows_to = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const U x = __shfl_up_sync(~0u, units_to, o);
    const int y = __shfl_up_sync(~0u, rows_to, o);
    if (lane >= o) units_to += x, rows_to += y;
  }
  most = __reduce_max_sync(~0u, most);
  if (lane < 2) sh.part[2 * line + lane].n = 0;
  U total = __shfl_sync(~0u, units_to, 31);
  int all_rows = __shfl_sync(~0u, rows_to, 31);
  if (!few) {
    if (lane == 0) {
      sh.scan_units[warp] = total;
      sh.scan_rows[warp] = all_rows;
      sh.scan_most[warp] = most;
    }
    __syncthreads();
    total = 0;
    all_rows = 0;
#pragma unroll
    for (int w = 0; w < kDecodeWarps; ++w) {
      const U x = static_cast<U>(sh.scan_units[w]);
      const int y = sh.scan_rows[w];
      if (w < warp) units_to += x, rows_to += y;
      total += x;
      all_rows += y;
      most = max(most, sh.scan_most[w]);
    }
  }
  // few and short rows: a CTA for each, so that nothing is left to be joined between CTAs
  const bool apart = most <= kApartTiles / together && int64_t(all_rows) * vheads <= gridDim.x;
  if (apart) {
    units = U(rows) * U(most);
    units_to = U(rows_to) * U(most);
    total = U(all_rows) * U(most);
  }
  auto units_of = [&](int n) -> U { return n == 0 ? 0 : apart ? most : n + kRowUnits; };
  total *= vheads;
  // fewer CTAs than there are where each warp would not have a unit
  int ctas = static_cast<int>(gridDim.x);
  if (apart)
    ctas = max(1, all_rows * vheads);
  else if (total < U(ctas) << sub_bits)
    ctas = max(1, static_cast<int>(total >> sub_bits));
  const int cta = blockIdx.x;
  const Deal<U> deal(total, ctas);
  const U cta_lo = cta < ctas ? deal.from(cta) : 0, cta_n = cta < ctas ? deal.from(cta + 1) - cta_lo : 0;
  auto sub_from = [&](int i) -> U { return cta_lo + (cta_n >> sub_bits) * U(i) + min(U(i), cta_n & U(subs - 1)); };
  const U first_unit = (units_to - units) * vheads;  // of this thread's requests
  if (!few) {
    sh.first_unit[tid] = first_unit;
    __syncthreads();
  }

  const U lo = sub_from(sub), hi = sub_from(sub + 1);

  unsigned char* mine_smem = smem + line * C::kWarpBytes;
  const uint32_t k_stage = smem_u32(mine_smem), v_stage = k_stage + C::kStageBytes;
  float* v_floats = reinterpret_cast<float*>(mine_smem + C::kStageBytes);
  float* park = reinterpret_cast<float*>(mine_smem + 2 * C::kStageBytes);

  if (lo < hi) {
    // on to the next (b, vh); beyond the share only the unit counts
    auto next_row = [&](Cursor<U>& c) {
      c.u += units_of(c.n) - U(c.t);
      if (c.u >= hi) return;
      c.t = 0;
      if (++c.vh < vheads) return;
      c.vh = 0;
      c.len = length_of(a, ++c.b);
      // requests without rows: 32 lengths at a time, up to the next that has some (it
      // is there, as the share goes on)
      while (c.len == 0 && c.b + 1 < a.B) {
        const int b = c.b + 1 + lane, len = b < a.B ? length_of(a, b) : 0;
        const uint32_t some = __ballot_sync(~0u, len > 0);
        const int to = some ? __ffs(some) - 1 : 31;
        c.b = min(c.b + 1 + to, a.B - 1);
        c.len = __shfl_sync(~0u, len, to);
      }
      c.n = tiles_of(c.len);
    };
    Cursor<U> at;  // of the tile whose rows are looked up next
    {
      // the last thread whose requests begin at or before the share
      at.u = lo;
      U r;
      if (few) {
        at.b = __popc(__ballot_sync(~0u, first_unit <= lo)) - 1;  // lanes behind the last begin at the end
        r = lo - __shfl_sync(~0u, first_unit, at.b);
        at.len = __shfl_sync(~0u, last_len, at.b);
        at.n = tiles_of(at.len);
      } else {
        // by groups of kDecodeWarps threads and then within the group
        auto begins = [&](int t) { return static_cast<U>(sh.first_unit[t]) <= lo; };
        static_assert(kDecodeWarps <= 32, "a group's threads have a lane each");
        const int t0 = (__popc(__ballot_sync(~0u, begins(lane * kDecodeWarps))) - 1) * kDecodeWarps;
        const int t = t0 + __popc(__ballot_sync(~0u, lane < kDecodeWarps && begins(t0 + (lane % kDecodeWarps)))) - 1;
        r = lo - static_cast<U>(sh.first_unit[t]);
        for (at.b = t * slab;; ++at.b) {
          at.len = length_of(a, at.b);
          at.n = tiles_of(at.len);
          const U all = units_of(at.n) * vheads;
          if (r < all || at.b + 1 >= a.B) break;
          r -= all;
        }
      }
      const U per = units_of(at.n);
      at.vh = static_cast<int>(r / per);
      at.t = static_cast<int>(r - U(at.vh) * per);
    }
    if (at.t >= at.n) next_row(at);
    Cursor<U> now = at;  // of the tile computed next
    const int32_t* table = nullptr;  // at's
    int64_t head_off = 0;
    auto row_of_at = [&] {
      table = a.table + at.b * a.table_row;
      head_off = (at.vh / passes) * a.head;
    };
    row_of_at();

    // What is known of the next tile's row `lane`: its page (kNoRow behind the last
    // row) and its offset from the page's first value.  The page is not looked at
    // before the row is asked for, so that the load from the table is under way
    // meanwhile.
    constexpr int kNoRow = INT_MIN;
    int page = kNoRow;
    int64_t in_page = 0;
    auto look_up = [&] {
      const int pos = at.t * kTile + lane;
      page = kNoRow;
      if (pos >= at.len) return;
      const int i = a.div.quot(pos);
      page = max(table[i], kNoRow + 1);  // an entry of INT_MIN is as bad as any negative one
      in_page = static_cast<uint32_t>(pos - i * a.div.d) * static_cast<uint64_t>(static_cast<uint32_t>(a.row)) + head_off;
    };
    // Its place in the cache in bytes, and which rows of the tile count.
    int64_t off = 0;
    uint32_t live = 0;
    auto locate = [&] {
      const bool in_cache = page >= 0 && page < a.num_pages;
      if (!in_cache && page != kNoRow) atomicOr(a.status, kPagerBadPage);
      off = in_cache ? (page * a.page + in_page) * 2 : 0;
      live = __ballot_sync(~0u, in_cache);
    };
    // Rows of a tile into a stage: 8 lanes copy 128 bytes of a row, chunk c of row r
    // to place c ^ (r % 8) of its 8.
    const uint64_t policy = read_once_policy();
    const uint32_t to_even = (lane >> 3) * (D * 2) + (((lane & 7) ^ (lane >> 3)) << 4), to_odd = to_even ^ 64;
    auto copy = [&](uint32_t stage, const uint16_t* from) {
      const char* base = reinterpret_cast<const char*>(from) + (lane & 7) * 16;
#pragma unroll
      for (int i = 0; i < kTile / 4; ++i) {  // rows 4 i + lane / 8
        const char* src = base + __shfl_sync(~0u, off, 4 * i + (lane >> 3));
        const bool take = (live >> (4 * i + (lane >> 3))) & 1;
        const uint32_t dst = stage + 4 * i * (D * 2) + (i & 1 ? to_odd : to_even);
#pragma unroll
        for (int half = 0; half < D / 64; ++half) cp_async16(dst + 128 * half, src + 128 * half, take, policy);
      }
    };

    bool more = at.u < hi;
    if (more) look_up();
    locate();
    copy(k_stage, a.k);
    cp_async_commit();
    copy(v_stage, a.v);
    cp_async_commit();
    uint32_t live_now = live;
    // looks up the tile behind the one asked for, if the share has one
    auto find_next = [&] {
      ++at.t;
      ++at.u;
      if (at.t >= at.n) {
        next_row(at);
        row_of_at();
      }
      more = at.u < hi;
      if (more) look_up();
    };
    if (more) find_next();

    float o_acc[D / 16][NT][4], m[NT][2], l[NT][2];
    uint32_t qf[D / 16][NT][2];
    const int g = lane >> 2, j = lane & 3;
    int t0 = 0, first = 0, heads = 0;
    bool fresh = true;
    const float scale_log2 = a.scale * kLog2e;
    // ldmatrix: lane's row of the first 16 and its chunk, exclusive or included; what
    // is added for later chunks touches other bits
    const uint32_t k_lane = k_stage + (lane & 15) * (D * 2) + (((lane >> 4) ^ (lane & 7)) << 4);
    const uint32_t v_lane = v_stage + ((lane & 7) + (lane >> 4) * 8) * (D * 2) + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);

    while (now.u < hi) {
      if (fresh) {
        fresh = false;
        t0 = now.t;
        heads_of<kSide>(a, now.vh * together + part, &first, &heads);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bool have = 8 * n + g < heads;
          const uint16_t* q = a.q + now.b * a.q_row + int64_t(first + 8 * n + (have ? g : 0)) * D + 2 * j;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            qf[ks][n][0] = have ? *reinterpret_cast<const uint32_t*>(q + 16 * ks) : 0u;
            qf[ks][n][1] = have ? *reinterpret_cast<const uint32_t*>(q + 16 * ks + 8) : 0u;
          }
          m[n][0] = m[n][1] = -INFINITY;
          l[n][0] = l[n][1] = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o_acc[i][n][e] = 0.f;
        }
      }
      cp_async_wait<1>();  // K is here, V may be on its way
      __syncwarp();

      // scores of rows 16 x + (g, g + 8) and heads (2 j, 2 j + 1)
      float s[2][NT][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][n][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t kf[4];
          ldmatrix4(kf, (k_lane ^ (ks << 5)) + x * 16 * (D * 2));
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16816(s[x][n], kf, qf[ks][n][0], qf[ks][n][1]);
        }
      }
      __syncwarp();  // K is read
      if (more) {
        locate();
        copy(k_stage, a.k);
      }
      cp_async_commit();

      uint32_t hi_f[2][NT][2], lo_f[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool counts = (live_now >> (16 * x + g + (e >> 1) * 8)) & 1;
            s[x][n][e] = counts ? s[x][n][e] * scale_log2 : -INFINITY;
            top[e & 1] = fmaxf(top[e & 1], s[x][n][e]);
          }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          top[0] = fmaxf(top[0], __shfl_xor_sync(~0u, top[0], x));
          top[1] = fmaxf(top[1], __shfl_xor_sync(~0u, top[1], x));
        }
        if (__any_sync(~0u, top[0] > m[n][0] || top[1] > m[n][1])) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float up = fmaxf(m[n][e], top[e]);
            // all scores so far -inf: there is nothing to keep
            const float keep = m[n][e] == -INFINITY ? 0.f : fast_exp2(m[n][e] - up);
            m[n][e] = up;
            l[n][e] *= keep;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o_acc[i][n][e] *= keep, o_acc[i][n][2 + e] *= keep;
          }
        }
        const float ref[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = fast_exp2(s[x][n][e] - ref[e & 1]);
            l[n][e & 1] += p[e];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t upper, lower;
            split_weights(p[2 * e], p[2 * e + 1], upper, lower);
            hi_f[x][n][e] = transpose8x8(upper);
            lo_f[x][n][e] = transpose8x8(lower);
          }
        }
      }
      cp_async_wait<1>();  // V is here, the next K may be on its way
      __syncwarp();
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t vf[4];
          ldmatrix4_trans(vf, (v_lane ^ (i << 5)) + x * 16 * (D * 2));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816(o_acc[i][n], vf, hi_f[x][n][0], hi_f[x][n][1]);
            mma_16816(o_acc[i][n], vf, lo_f[x][n][0], lo_f[x][n][1]);
          }
        }
      }
      __syncwarp();  // V is read

      const bool row_ends = now.t + 1 == now.n;
      const bool share_ends = (row_ends ? now.u + (units_of(now.n) - U(now.t)) : now.u + 1) >= hi;
      if (row_ends || share_ends) {
        const bool whole = row_ends && t0 == 0;
        // a part of a row: the share's first waits in the park, its last where V was
        const bool parked = !whole && !share_ends;
        float* to = parked ? park : v_floats;
        const int slot = 2 * line + (parked ? 0 : 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], x);
            const int head = 8 * n + 2 * j + e;
            if (whole) {
              if (g == 0 && head < heads) a.lse[int64_t(first + head) * a.B + now.b] = lse_of(m[n][e], l[n][e]);
            } else if (g == 0) {
              sh.m[slot][head] = m[n][e];
              sh.l[slot][head] = l[n][e];
            }
            const float by = whole ? inverse_of(l[n][e]) : 1.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              to[o_at<D>(head, 16 * i + g)] = o_acc[i][n][e] * by;
              to[o_at<D>(head, 16 * i + g + 8)] = o_acc[i][n][2 + e] * by;
            }
          }
        }
        __syncwarp();
        if (whole) {
          constexpr int kLanes = D / 4;
          for (int h = lane / kLanes; h < heads; h += 32 / kLanes) {
            const int d = 4 * (lane % kLanes);
            store_out4(a, D, now.b, first + h, d, *reinterpret_cast<const float4*>(to + o_at<D>(h, d)));
          }
          __syncwarp();
        } else if (lane == 0) {
          sh.part[slot] = {int64_t(now.u - U(now.t)), now.b, now.vh * together + part, t0, now.t + 1, now.n};
        }
        fresh = true;
      }
      ++now.t;
      ++now.u;
      if (now.t >= now.n) next_row(now);

      if (more) {
        copy(v_stage, a.v);
        live_now = live;
        find_next();
      }
      cp_async_commit();
    }
    cp_async_wait<0>();
  }

  // ---- requests without rows
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (length_of(a, b) > 0) continue;
    if (tid == 0 && a.lens[b] != 0) atomicOr(a.status, kPagerBadLength);
    for (int i = tid; i < a.H * (D / 4); i += kDecodeWarps * 32)
      store_out4(a, D, b, i / (D / 4), 4 * (i % (D / 4)), make_float4(0.f, 0.f, 0.f, 0.f));
    for (int h = tid; h < a.H; h += kDecodeWarps * 32) a.lse[int64_t(h) * a.B + b] = -INFINITY;
  }
  if (cta_n == 0) return;
  __syncthreads();

  // ---- parts of a row within this CTA's share
  auto part_o = [&](int slot) -> const float* {
    return reinterpret_cast<const float*>(smem + (slot >> 1) * C::kWarpBytes + (slot & 1 ? 1 : 2) * C::kStageBytes);
  };
  constexpr int kQuads = D / 4;
  uint32_t held, heads_at;  // slots that hold a part, and those where a row's first part is
  {
    const Stretch p = sh.part[lane & (2 * kDecodeWarps - 1)];
    const bool have = lane < 2 * kDecodeWarps && p.n > 0;
    held = __ballot_sync(~0u, have);
    const uint32_t below = held & ((1u << lane) - 1);
    const int prev = below ? 31 - __clz(below) : lane;
    const int prev_b = __shfl_sync(~0u, p.b, prev), prev_x = __shfl_sync(~0u, p.x, prev);
    heads_at = __ballot_sync(~0u, have && (!below || prev_b != p.b || prev_x != p.x));
  }
  // as many rows at once as have threads for their heads
  int row_threads = 32;
  while (row_threads < a.part_heads * kQuads && row_threads < kDecodeWarps * 32) row_threads *= 2;
  const int row_tid = tid & (row_threads - 1), my_turn = tid / row_threads, turns = kDecodeWarps * 32 / row_threads;
  // a slot of what goes on in other CTAs, by its place in global memory: 0 begun
  // before, 1 begun here (all parts of its query heads alike)
  int open[2] = {-1, -1};
  for (int turn = 0; heads_at; ++turn) {
    const int s = __ffs(heads_at) - 1;
    heads_at &= heads_at - 1;
    const int end = heads_at ? __ffs(heads_at) - 1 : 2 * kDecodeWarps;
    const uint32_t parts = held & ((1u << end) - (1u << s));
    const Stretch& p = sh.part[s];
    const bool whole = p.t0 == 0 && sh.part[31 - __clz(parts)].t1 == p.n;
    const int place = p.t0 == 0 ? 1 : 0;
    if (!whole) (place == 0 ? open[0] : open[1]) = s;
    if ((turn & (turns - 1)) != my_turn) continue;
    int first, heads;
    heads_of<kSide>(a, p.x, &first, &heads);
    for (int i = row_tid; i < heads * kQuads; i += row_threads) {
      const int h = i / kQuads, d = 4 * (i % kQuads);
      Joined sum;
      for (uint32_t left = parts; left;) {
        constexpr int kBatch = 4;
        float2 ml[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          ml[x] = make_float2(-INFINITY, 0.f);
          v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (left) {
            const int slot = __ffs(left) - 1;
            left &= left - 1;
            ml[x] = make_float2(sh.m[slot][h], sh.l[slot][h]);
            v[x] = *reinterpret_cast<const float4*>(part_o(slot) + o_at<D>(h, d));
          }
        }
        sum.add(ml, v);
      }
      if (whole) {
        store_joined(a, D, p.b, first + h, d, sum);
      } else {
        const int at = (2 * cta + place) * together + (p.x & (together - 1));
        __stcg(reinterpret_cast<float4*>(a.part_o + (at * C::kHeads + h) * D + d), sum.o);
        if (d == 0)
          __stcg(reinterpret_cast<float2*>(a.part_ml + (at * C::kHeads + h) * 2), make_float2(sum.top, sum.sum));
      }
    }
  }

  // ---- rows that several CTAs share: the last to arrive joins them.  Of many parts
  // groups of kGroup are joined first, each by its own last: what one SM reads in a
  // row costs more than a second arrival does.
  if (open[0] < 0 && open[1] < 0) return;
  int* counter = nullptr;  // where thread `place` arrives, one of `arrivals`
  int arrivals = 0;
  if (tid < 2) {
    const int slot = tid == 0 ? open[0] : open[1];
    sh.last[tid] = 0;
    if (slot >= 0) {
      const Stretch& p = sh.part[slot];
      const int from = tid == 1 ? cta : deal.taker(static_cast<U>(p.u0)), to = deal.taker(static_cast<U>(p.u0) + p.n - 1);
      const bool grouped = to - from + 1 > 3 * kGroup;
      const int lead = grouped ? from + (cta - from) / kGroup * kGroup : from;
      sh.from[tid] = from;
      sh.to[tid] = to;
      counter = grouped ? a.counters + gridDim.x + 2 * lead + (lead == from) : a.counters + from;
      arrivals = grouped ? min(kGroup, to + 1 - lead) : to - from + 1;
    }
  }
  __syncthreads();
  if (counter) sh.last[tid] = last_of(counter, arrivals);
  __syncthreads();
#pragma unroll 1
  for (int place = 0; place < 2; ++place) {
    if (!sh.last[place]) continue;
    const Stretch& p = sh.part[place == 0 ? open[0] : open[1]];
    const int from = sh.from[place], to = sh.to[place];
    bool grouped = to - from + 1 > 3 * kGroup;
    int base = grouped ? from + (cta - from) / kGroup * kGroup : from, step = 1;
    int count = grouped ? min(kGroup, to + 1 - base) : to - from + 1;
    for (;;) {
      for (int y = 0; y < together; ++y) {
        int first, heads;
        heads_of<kSide>(a, (p.x & -together) + y, &first, &heads);
        // Where the parts are: a CTA's last place if the row begins in it, else its
        // first.  32 bits hold the whole workspace.
        const int first_at = (2 * base + (base == from ? 1 : 0)) * together + y;
        const int next_at = 2 * base * together + y, step_at = 2 * step * together;
        // 4 values of kItems heads to a thread, the loads of a batch of parts under way together
        constexpr int kThreads = kDecodeWarps * 32;
        constexpr int kItems = C::kHeads * kQuads > kThreads ? C::kHeads * kQuads / kThreads : 1;
        static_assert(kItems * kThreads >= C::kHeads * kQuads, "one round for all heads");
        Joined sum[kItems];
        auto add_batch = [&](auto size, int x0) {
          constexpr int kBatch = decltype(size)::value;
          float2 ml[kItems][kBatch];
          float4 v[kItems][kBatch];
#pragma unroll
          for (int z = 0; z < kItems; ++z) {
            const int i = tid + z * kThreads, h = i / kQuads, d = 4 * (i % kQuads);
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
              ml[z][x] = make_float2(-INFINITY, 0.f);
              v[z][x] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (x0 + x < count && h < heads) {
                const int at = x0 + x == 0 ? first_at : next_at + (x0 + x) * step_at;
                ml[z][x] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (at * C::kHeads + h) * 2));
                v[z][x] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (at * C::kHeads + h) * D + d));
              }
            }
          }
#pragma unroll
          for (int z = 0; z < kItems; ++z) sum[z].add(ml[z], v[z]);
        };
        // a batch costs its size, and most rows have two parts: 128 mixed requests take 1
        // us more with batches of 16 for all, long rows 1 us with batches of 4
        constexpr int kFew = 2, kMany = 8;
        if (count <= kFew) {
          add_batch(std::integral_constant<int, kFew>(), 0);
        } else {
          for (int x0 = 0; x0 < count; x0 += kMany) add_batch(std::integral_constant<int, kMany>(), x0);
        }
        // a group's sum takes the place of its first part, which a head's warp alone reads
        static_assert(32 % kQuads == 0, "a head's values lie in one warp");
        __syncwarp();
#pragma unroll
        for (int z = 0; z < kItems; ++z) {
          const int i = tid + z * kThreads, h = i / kQuads, d = 4 * (i % kQuads);
          if (h >= heads) continue;
          if (grouped) {
            __stcg(reinterpret_cast<float4*>(a.part_o + (first_at * C::kHeads + h) * D + d), sum[z].o);
            if (d == 0)
              __stcg(reinterpret_cast<float2*>(a.part_ml + (first_at * C::kHeads + h) * 2),
                     make_float2(sum[z].top, sum[z].sum));
          } else {
            store_joined(a, D, p.b, first + h, d, sum[z]);
          }
        }
      }
      if (!grouped) break;
      grouped = false;
      base = from;
      step = kGroup;
      count = (to - from) / kGroup + 1;
      __syncthreads();
      if (tid == 0) sh.last[place] = last_of(a.counters + from, count);
      __syncthreads();
      if (!sh.last[place]) break;
    }
  }
}

template <int D, int NT, bool kSide, typename U>
cudaError_t launch(const DecodeArgs& a, int sms, cudaStream_t stream) {
  using C = DecodeCfg<D, NT>;
  static_assert(C::kCtasPerSm * (C::kSmemBytes + sizeof(DecodeShared<D, NT>) + 1024) <= 233472, "shared memory of an SM");
  cudaError_t e = set_smem_limit_once<decode_kernel<D, NT, kSide, U>>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_overlapped(decode_kernel<D, NT, kSide, U>, dim3(sms * C::kCtasPerSm), kDecodeWarps * 32, C::kSmemBytes,
                           stream, a);
}

template <int D, typename U>
cudaError_t launch_by_heads(const DecodeArgs& a, int sms, cudaStream_t stream) {
  if (a.together > 1) return launch<D, 2, true, U>(a, sms, stream);
  return a.part_heads <= 8 ? launch<D, 1, false, U>(a, sms, stream) : launch<D, 2, false, U>(a, sms, stream);
}

}  // namespace

DecodeSpace decode_space(int D, const QueryParts& parts, int sms) {
  const int heads = parts.part_heads <= 8 ? 8 : 16;
  const int ctas = sms * (D == 64 ? DecodeCfg<64, 1>::kCtasPerSm : DecodeCfg<128, 1>::kCtasPerSm);
  static_assert(DecodeCfg<64, 1>::kCtasPerSm == DecodeCfg<64, 2>::kCtasPerSm &&
                    DecodeCfg<128, 1>::kCtasPerSm == DecodeCfg<128, 2>::kCtasPerSm, "one grid for each D");
  // a counter for the row that begins in a CTA's share, two for groups that a CTA
  // leads; two places for each CTA and part
  const int64_t places = int64_t(ctas) * 2 * parts.together;
  return {3 * ctas, places * heads * 2, places * heads * D};
}

QueryParts query_parts(int group) {
  QueryParts k{1, 1, 1, group};
  while (k.together < kDecodeWarps && k.together * kMostHeads < group) k.together *= 2;
  k.passes = (group + kMostHeads * k.together - 1) / (kMostHeads * k.together);
  k.parts = k.passes * k.together;
  k.part_heads = (group + k.parts - 1) / k.parts;  // above 8 where there are parts
  return k;
}

cudaError_t launch_decode(const DecodeArgs& a, int sms, cudaStream_t stream) {
  // the units of B full table rows
  const int64_t most = int64_t(a.B) * (int64_t(a.max_pages) * a.div.d / kTile + 1 + kRowUnits);
  if (most > UINT32_MAX / (a.Hkv * a.passes))
    return a.D == 128 ? launch_by_heads<128, uint64_t>(a, sms, stream) : launch_by_heads<64, uint64_t>(a, sms, stream);
  return a.D == 128 ? launch_by_heads<128, uint32_t>(a, sms, stream) : launch_by_heads<64, uint32_t>(a, sms, stream);
}

}  // namespace jfa
