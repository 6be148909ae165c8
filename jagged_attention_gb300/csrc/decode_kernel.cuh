// decode_kernel.cuh -- attention of one new token per request over the paged cache.
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
// Codes (coded.cuh) become fp16 on their way from shared memory to the tensor cores, which
// is exact: cvt takes two e4m3 or e2m1 codes, 4-bit ones are then multiplied by their
// scale.  q becomes fp16 too, times a power of two of its head that leaves its 8 bits.  8 bits: with
// 2^e_t and 2^f_t the powers of two of row t of K and V, s_t = scale 2^e_t q . c_t and
//     out = sum 2^(s_t + f_t - r) c'_t / sum 2^(s_t - r)   (s_t in units of log2 e),
// where r is the running maximum of s_t + f_t rather than of s_t: the weights of the codes
// are then at most 1 whatever the rows' sizes, and those of the sum within 2^48 of that.
// A weight enters the product as one fp16 number of 11 bits, times 2^15 so that it is not
// subnormal before 2^-29 of the largest; its rounding, 2^-11 at most, is an eighth of that
// of the output to bf16, and a second number would cost as many products again.
// The 2^15 is taken off r in fp32, which is exact enough while r is small (kNear).  In a
// stretch of larger scores r is the largest score as it is, rounded to fp32; weights are
// powers of two of z = (s_t - r) + f_t, over 2^(rho - 15) with rho the largest z, and l and
// O are held over that too until the stretch ends.  With all scores so large the full caches
// take 556 us of 8 bits and 440 of 4, 543 and 391 with none.
//
// Bound: every cached row is read once, 4 D bytes for 4 D G flops (G query heads
// to a key/value head), so memory bandwidth bounds it while G is small.  The
// products use mma.sync, transposed -- rows of the cache are the long side of the
// 16 x 8 tile, up to 8 query heads (16: two tiles) the short one -- which wastes
// least of the tile and leaves the cache rows in the layout that ldmatrix reads;
// tcgen05 would want 64 or 128 query rows per product.  The tensor pipe is 12%
// busy at G = 8.  Of 4-bit codes the conversions (an instruction for two values, one for
// their scale) and the rest of a value's instructions bound it before memory does: a
// tile of 64 rows takes 1,390 instructions, 9,216 bytes.
//
// Split: a tile is 32 cached rows (of codes 64) for one key/value head.  All tiles of all
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
// each of 2: 223 us, one part after the other 340 us).
//
// Measured (GB300, 6.67 TB/s copied): 96 requests up to 32768 rows, 64 heads on 8,
// 7.2 GB in 1016 to 1048 us (by GPU), 6.9 TB/s; 128 requests of 0 to 8192 rows, 443 MB in 73 us,
// 6.1 TB/s; one request of 131072, 268 MB in 48.5 us, 5.5 TB/s; one of 300 rows in
// 6.2 us.  What is left of the middle sizes is about 2.5 us until the first rows
// arrive (lengths, table, rows: three dependent trips to memory), 3 to 6 us of
// joining, and SMs whose memory is 7% slower than others'.  128 KB of K and V in
// the stages of 8 warps measured best: with 192 KB the full cache took 1126 us for
// 1070, with 6 warps 1094 for 1064.
//
// Codes, by GPU: the full cache, 3.6 GB of 8 bits in 525 to 543 us, 6.9 to 6.7 TB/s; 2.0 GB of
// 4 bits in 391 to 395 us, 5.1 TB/s (by heads outside rows 398); 128 mixed requests, 224 MB in 43
// to 45 us and 126 MB in 40; one of 131072, 76 MB of 4 bits in 30 us; one of 300 rows in 6.3.
// Codes in the warps' registers want tiles of 64 rows: of 32 the full caches take 590 and 417 us.
// 4 bits run best with 16 warps an SM of 128 registers each; with 8 of 255 they take 8% fewer
// instructions and 415 us.  Scores of two groups of 16 rows are summed side by side (4% of the
// full cache of 4 bits).  Bit moves in place of cvt are slower, and so are 4-bit integers
// (values per clock of an SM, conversion and product alone: e2m1 62, 4-bit integers 45).
#pragma once
#include <climits>
#include <type_traits>

#include "coded.cuh"
#include "kernels.h"
#include "paged.h"
#include "sm103_ptx.cuh"

namespace jfa {
namespace {

constexpr int kMostHeads = 16;   // query heads that a warp holds
constexpr int kMostTogether = 8;  // warps side by side
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kWeightBits = 15.f;  // of codes: the largest weight is 2^15, as fp16 has it
// The largest running reference, in units of log2 e, that 15 is taken off as it is.  4 bits:
// it is rounded by 1/8 at most then, and the largest weight is 2^15.125.  8 bits: a weight's
// exponent is off by 2^-13 at most for its row's power of two, a sixth of fp16's rounding.
template <int kBits>
constexpr float kNear = kBits == 8 ? 0x1p10f : 0x1p22f;

template <int kBits, int D, int NT>  // NT: tiles of 8 query heads
struct DecodeCfg {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kTile = kBits == 16 ? 32 : 64;       // cached rows of a tile
  static constexpr int kSub = kTile / 32;                   // of which a lane looks up so many
  static constexpr int kRowBytes = D * kBits / 8;
  static constexpr int kScaleBytes = kBits == 4 ? D / kBlock : 0;  // of a row, in the stage
  static constexpr int kStageBytes = kTile * (kRowBytes + kScaleBytes);  // a tile's K, or its V
  static constexpr int kOutBytes = kHeads * D * 4;          // a stretch's O
  static constexpr int kVBytes = kOutBytes > kStageBytes ? kOutBytes : kStageBytes;  // holds a stretch's O when V is read
  static constexpr int kWarpBytes = kStageBytes + kVBytes + kOutBytes;  // K, V, park
  static constexpr int kWarps = 8;
  static constexpr int kSmemBytes = kWarps * kWarpBytes;
  // 64 values with 16 heads a warp, the full cache: 8 bits 398 us so, with two CTAs of 128
  // registers, which spill, 596; 4 bits with two, which spill less, 352, with one 357.
  static constexpr int kCtasPerSm = kBits == 16 ? (D == 64 ? 2 : 1) : kBits == 8 ? (D == 64 && NT == 1 ? 2 : 1)
                                                                              : (D == 64 || NT == 1 ? 2 : 1);
};

// Units of work: the n tiles of a (request, key/value head) count n units, and
// kRowUnits behind them stand for its beginning and end (256 requests up to 300
// rows: 34.6 us without, 32.5 with; 128 mixed ones 74.7 and 74.2).  Of codes, whose tiles
// are larger, one: 500 requests up to 900 rows in 4 bits 69.2 us, with two 72.0, none 73.2,
// 512 mixed ones in 8 bits 147, 152 and 149, 128 mixed ones 45.2, 46.2 and 52.0.
template <int kBits>
constexpr int kRowUnits = kBits == 16 ? 2 : 1;

// Parts of a row that one CTA joins at a time, where a row has more than three times
// as many (38 parts of 16 heads: 22.9 us, all at once 28.7; up to 24 parts it makes
// no difference).
constexpr int kGroup = 8;

// Few requests of at most so many rows get a CTA each.  4 rows of 8 heads on 2: of 250
// 5.5 us, spread over more CTAs and joined 6.9; of 380 (12 tiles) 6.4 and 7.0; of 440
// 6.6 and 6.9, of 512 6.8 and 7.1, so that up to 16 it would gain as well, of 540 7.6
// and 7.3.
constexpr int kApartRows = 12 * 32;

// Of codes a CTA's share is 2^kLeastBits units at least.
constexpr int kLeastBits = 2;

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

template <int kWarps, int NT>
struct DecodeShared {
  Stretch part[2 * kWarps];                 // first and last of each warp
  float m[2 * kWarps][8 * NT], l[2 * kWarps][8 * NT];
  int64_t scan_units[kWarps];
  int scan_rows[kWarps], scan_most[kWarps];
  int64_t first_unit[kWarps * 32];  // of the requests that a thread adds up
  int from[2], to[2], last[2];
};

__device__ __forceinline__ int length_of(const DecodeArgs& a, int b) {
  const int len = a.lens[b];
  return len < 0 || len > a.max_pages * a.div.d ? 0 : len;
}

template <int kTile>
__device__ __forceinline__ int tiles_of(int len) { return len / kTile + (len % kTile != 0); }

// The cache is read once a launch: its lines are the first to leave L2, before the
// lengths, tables and queries (1 to 6% of a call of 23 to 75 us).
__device__ __forceinline__ uint64_t read_once_policy(bool twice) {
  uint64_t p;
  if (twice)
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  else
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take, uint64_t policy) {
  const int bytes = take ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy) : "memory");
}
// N bytes, 4 or 8, of scales.
template <int N>
__device__ __forceinline__ void cp_async_few(uint32_t dst, const void* src, bool take) {
  const int bytes = take ? N : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
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

__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ T at_shared(const unsigned char* p) {
  return *reinterpret_cast<const T*>(p);
}

// Place of value (head, d) of a stretch's O in shared memory: the exclusive or
// sends the 32 lanes of a fragment to 32 banks and keeps runs of 8 together (of codes,
// whose fragments hold pairs of d: runs of 4, two lanes to a bank).
template <int kBits, int D>
__device__ __forceinline__ int o_at(int head, int d) {
  return head * D + (d ^ (((head >> 1) & 3) << (kBits == 16 ? 3 : 2)));
}

// Codes in a stage: lines of 128 bytes hold one row, two or four, and a row's 16-byte
// chunks stand at exclusive-or'd places of its line, so that the lanes that load together
// -- of K 8 rows at 4 places, of V 4 rows at 8 -- find 32 banks.
template <int kRowBytes>
__device__ __forceinline__ int swizzle_of(int row, bool v) {
  return v ? 2 * ((row >> 2) & 3) : kRowBytes == 128 ? 4 * (row & 1) : kRowBytes == 64 ? 0 : 4 * ((row >> 2) & 1);
}
template <int kRowBytes>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk, bool v) {
  constexpr int kRows = 128 / kRowBytes;
  return row / kRows * 128 + (((row % kRows * (kRowBytes / 16) + chunk) ^ swizzle_of<kRowBytes>(row, v)) << 4);
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

// x / a.parts, which is a power of two times a.passes, mostly 1.  Divisions cost every CTA
// instructions before its first row: 16 requests of 64 heads on 2 28.7 us with, 28.1 without.
__device__ __forceinline__ int kv_of(const DecodeArgs& a, int x) {
  const int y = x >> (__ffs(a.together) - 1);
  return a.passes == 1 ? y : y / a.passes;
}

// Query heads [first, first + count) of part x of all, a.parts to a key/value head:
// one where the parts are not side by side.
template <bool kSide>
__device__ __forceinline__ void heads_of(const DecodeArgs& a, int x, int* first, int* count) {
  const int kv = kSide ? kv_of(a, x) : x, g0 = kSide ? (x - kv * a.parts) * a.part_heads : 0;
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
// Of codes the sum may have any size, and log2f is right to a unit in its last place.
template <int kBits>
__device__ __forceinline__ float lse_of(float m, float l) { return (m + (kBits == 16 ? __log2f(l) : log2f(l))) * kLn2; }
// 1 / l for such a sum, 2 units in the last place, where 0 stays 0.
__device__ __forceinline__ float inverse_of(float l) { return l == 0.f ? 0.f : __fdividef(1.f, l); }

// A finished row: normalised, with its log-sum-exp.
template <int kBits>
__device__ __forceinline__ void store_joined(const DecodeArgs& a, int D, int b, int head, int d, const Joined& s) {
  const float by = inverse_of(s.sum);
  store_out4(a, D, b, head, d, make_float4(s.o.x * by, s.o.y * by, s.o.z * by, s.o.w * by));
  if (d == 0) a.lse[int64_t(head) * a.B + b] = lse_of<kBits>(s.top == -INFINITY ? 0.f : s.top, s.sum);
}

template <int kBits>
using ArgsOf = std::conditional_t<kBits == 16, DecodeArgs, CodedDecodeArgs>;

// U: unsigned type that counts all units.  32 bits hold them unless the table is
// wide enough for more; 64 bits cost 0.3 to 0.6 us.
// kSide: parts of query heads side by side.
template <int kBits, int D, int NT, bool kSide, typename U>
__global__ void __launch_bounds__(DecodeCfg<kBits, D, NT>::kWarps * 32, DecodeCfg<kBits, D, NT>::kCtasPerSm)
decode_kernel(const __grid_constant__ ArgsOf<kBits> a) {
  using C = DecodeCfg<kBits, D, NT>;
  constexpr int kTile = C::kTile, kSub = C::kSub, kWarps = C::kWarps;
  extern __shared__ __align__(256) unsigned char smem[];
  __shared__ DecodeShared<kWarps, NT> sh;
  // Of codes, for each head of a warp the unit of a product of its q and codes, in units of
  // log2 e, not negative (in registers the full cache of 4 bits takes 404 us for 395).  Of a
  // stretch with large scores its largest score m, rho, and the unit: q_units is 1 then and
  // the register m 0, so that what else is done is the same for all scores.
  __shared__ __align__(8) float q_units[kBits < 16 ? kWarps : 1][8 * NT];
  __shared__ struct { float m, rho, unit; } large_of[kBits < 16 ? kWarps : 1][8 * NT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_launch_before();
  // ---- units of all requests, and where this CTA's warps begin.  Up to 32 requests
  // a warp adds up by itself, a lane for each, and waits for no other warp.
  const bool few = a.B <= 32;
  const int slab = few ? 1 : (a.B + kWarps * 32 - 1) / (kWarps * 32);
  const int b_lo = min(a.B, (few ? lane : tid) * slab), b_hi = min(a.B, b_lo + slab);
  U units = 0;
  int rows = 0, most = 0, last_len = 0;  // rows: requests that have any
  for (int b = b_lo; b < b_hi; ++b) {
    last_len = length_of(a, b);
    const int n = tiles_of<C::kTile>(last_len);
    units += n > 0 ? n + kRowUnits<kBits> : 0;
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
    for (int w = 0; w < kWarps; ++w) {
      const U x = static_cast<U>(sh.scan_units[w]);
      const int y = sh.scan_rows[w];
      if (w < warp) units_to += x, rows_to += y;
      total += x;
      all_rows += y;
      most = max(most, sh.scan_most[w]);
    }
  }
  // A CTA's share is dealt to `subs` sets of `together` warps, one for each part of
  // the query heads, or for each of a few key/value heads whose rows lie side by side; a
  // line is a warp's place with those of its part in a row.
  int vheads = a.Hkv * (kSide ? a.passes : 1), together = kSide ? a.together : 1;
  bool twice = false;  // lines of the cache are read by two warps with more than L2 holds between
  if constexpr (kBits < 16 && kSide) {
    if (a.mates > 1 && total >= a.mates_units) {
      vheads = a.Hkv / a.mates;
      together = a.mates;
      twice = total >= a.far_units;
    }
  }
  const int side_bits = kSide ? __ffs(together) - 1 : 0, sub_bits = __builtin_ctz(kWarps) - side_bits, subs = 1 << sub_bits;
  const int part = warp & (together - 1), sub = warp >> side_bits;
  const int line = (part << sub_bits) + sub;
  if (lane < 2) sh.part[2 * line + lane].n = 0;  // its own: no barrier stands before what it writes there

  // few and short rows: a CTA for each, so that nothing is left to be joined between CTAs
  const bool apart = most <= (kApartRows / C::kTile) >> side_bits && int64_t(all_rows) * vheads <= gridDim.x;
  if (apart) {
    units = U(rows) * U(most);
    units_to = U(rows_to) * U(most);
    total = U(all_rows) * U(most);
  }
  auto units_of = [&](int n) -> U { return n == 0 ? 0 : apart ? most : n + kRowUnits<kBits>; };
  total *= vheads;
  // fewer CTAs than there are where each warp, or few of them, would not have a unit
  const int least_bits = kBits == 16 ? sub_bits : min(sub_bits, kLeastBits);
  int ctas = static_cast<int>(gridDim.x);
  if (apart)
    ctas = max(1, all_rows * vheads);
  else if (total < U(ctas) << least_bits)
    ctas = max(1, static_cast<int>(total >> least_bits));
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
  const unsigned char *k_codes = mine_smem, *v_codes = mine_smem + C::kStageBytes;
  const uint32_t k_stage = smem_u32(mine_smem), v_stage = k_stage + C::kStageBytes;
  float* v_floats = reinterpret_cast<float*>(mine_smem + C::kStageBytes);
  float* park = reinterpret_cast<float*>(mine_smem + C::kStageBytes + C::kVBytes);

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
      c.n = tiles_of<C::kTile>(c.len);
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
        at.n = tiles_of<C::kTile>(at.len);
      } else {
        // by groups of kWarps threads and then within the group
        auto begins = [&](int t) { return static_cast<U>(sh.first_unit[t]) <= lo; };
        static_assert(kWarps <= 32, "a group's threads have a lane each");
        const int t0 = (__popc(__ballot_sync(~0u, begins(lane * kWarps))) - 1) * kWarps;
        const int t = t0 + __popc(__ballot_sync(~0u, lane < kWarps && begins(t0 + (lane % kWarps)))) - 1;
        r = lo - static_cast<U>(sh.first_unit[t]);
        for (at.b = t * slab;; ++at.b) {
          at.len = length_of(a, at.b);
          at.n = tiles_of<C::kTile>(at.len);
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
    // Offsets in the cache: of bf16 rows and in large caches bytes in 64 bits, else 32 bits
    // that count 16 bytes of codes, a row's bytes of scales.
    constexpr bool kWide = kBits == 16 || sizeof(U) == 8;
    constexpr int kUnit = kWide ? 1 : 16, kScaleUnit = kWide || kBits == 8 ? 1 : D / kBlock;
    using Off = std::conditional_t<kWide, int64_t, uint32_t>;
    auto distance = [](int64_t bytes, int unit) { return static_cast<Off>(kWide ? bytes : bytes / unit); };
    const int32_t* table = nullptr;  // at's
    int64_t head_off = 0;
    int kv_at = 0;
    auto row_of_at = [&] {
      table = a.table + at.b * a.table_row;
      kv_at = kSide ? kv_of(a, at.vh * together + part) : at.vh;
      head_off = kv_at * a.head;
    };
    row_of_at();

    // What is known of the next tile's row `lane` (and those 32 and more behind): its
    // page (kNoRow behind the last row) and its offset from the page's first value, or of
    // codes its place in the page.  The page is not looked at before the row is asked
    // for, so that the load from the table is under way meanwhile.
    constexpr int kNoRow = INT_MIN;
    int page[kSub], place[kSub];
    int64_t in_page[kSub];
#pragma unroll
    for (int z = 0; z < kSub; ++z) page[z] = kNoRow, place[z] = 0, in_page[z] = 0;  // for a share without a tile
    auto look_up = [&] {
#pragma unroll
      for (int z = 0; z < kSub; ++z) {
        const int pos = at.t * kTile + 32 * z + lane;
        page[z] = kNoRow;
        if (pos >= at.len) continue;
        const int i = a.div.quot(pos);
        page[z] = max(table[i], kNoRow + 1);  // an entry of INT_MIN is as bad as any negative one
        if constexpr (kBits == 16)
          in_page[z] = static_cast<uint32_t>(pos - i * a.div.d) * static_cast<uint64_t>(static_cast<uint32_t>(a.row)) + head_off;
        else
          place[z] = pos - i * a.div.d;
      }
    };
    // Its place in the cache in bytes, and which rows of the tile count; of codes the
    // scale bytes: 8 bits: that of the lane's row, 4 bits: where the row's are.
    Off off[kSub], scale_at[kSub];
    uint32_t live[kSub];
    int k_power[kSub], v_power[kSub];
    auto locate = [&] {
#pragma unroll
      for (int z = 0; z < kSub; ++z) {
        const bool in_cache = page[z] >= 0 && page[z] < a.num_pages;
        if (!in_cache && page[z] != kNoRow) atomicOr(a.status, kPagerBadPage);
        if constexpr (kBits == 16) {
          off[z] = in_cache ? (page[z] * a.page + in_page[z]) * 2 : 0;
        } else {
          // distances of rows are below 2^32
          auto place_of = [&](int64_t page_d, int64_t row_d, int64_t head_d, int unit) -> Off {
            if constexpr (kWide)
              return page[z] * page_d + static_cast<int64_t>(static_cast<uint32_t>(place[z]) * static_cast<uint64_t>(row_d)) + kv_at * head_d;
            else
              return page[z] * distance(page_d, unit) + place[z] * distance(row_d, unit) + kv_at * distance(head_d, unit);
          };
          off[z] = in_cache ? place_of(a.page, a.row, a.head, kUnit) : 0;
          scale_at[z] = in_cache ? place_of(a.scales.page, a.scales.row, a.scales.head, kScaleUnit) : 0;
          if constexpr (kBits == 8) {
            k_power[z] = in_cache ? a.scales.k[scale_at[z]] : kLeastPower;
            v_power[z] = in_cache ? a.scales.v[scale_at[z]] : kLeastPower;
          }
        }
        live[z] = __ballot_sync(~0u, in_cache);
      }
    };
    auto all_of = [](const uint32_t (&mask)[kSub]) {
      uint32_t every = ~0u;
#pragma unroll
      for (int z = 0; z < kSub; ++z) every &= mask[z];
      return every == ~0u;
    };
    // Rows of a tile into a stage.  bf16: 8 lanes copy 128 bytes of a row, chunk c of row
    // r to place c ^ (r % 8) of its 8.  Codes: the lanes that a row has chunks of 16 bytes.
    const uint64_t policy = read_once_policy(twice);
    const uint32_t to_even = (lane >> 3) * (D * 2) + (((lane & 7) ^ (lane >> 3)) << 4), to_odd = to_even ^ 64;
    auto copy = [&](uint32_t stage, const uint16_t* from, bool v) {
      if constexpr (kBits == 16) {
        const char* base = reinterpret_cast<const char*>(from) + (lane & 7) * 16;
#pragma unroll
        for (int i = 0; i < kTile / 4; ++i) {  // rows 4 i + lane / 8
          const char* src = base + __shfl_sync(~0u, off[0], 4 * i + (lane >> 3));
          const bool take = (live[0] >> (4 * i + (lane >> 3))) & 1;
          const uint32_t dst = stage + 4 * i * (D * 2) + (i & 1 ? to_odd : to_even);
#pragma unroll
          for (int half = 0; half < D / 64; ++half) cp_async16(dst + 128 * half, src + 128 * half, take, policy);
        }
      } else {
        constexpr int kChunks = C::kRowBytes / 16, kRows = 32 / kChunks;
        const int row0 = lane / kChunks;
        const char* base = reinterpret_cast<const char*>(from) + (lane % kChunks) * 16;
        const uint32_t to = stage + chunk_at<C::kRowBytes>(row0, lane % kChunks, v);
        const uint8_t* scales = v ? a.scales.v : a.scales.k;
        const uint32_t to_scale = stage + kTile * C::kRowBytes + lane * C::kScaleBytes;
        auto rows_at = [&](auto all) {  // all: no row is left out
#pragma unroll
          for (int i = 0; i < kTile / kRows; ++i) {
            const int z = i * kRows / 32, row = i * kRows % 32 + row0;
            const char* src = base + static_cast<int64_t>(__shfl_sync(~0u, off[z], row)) * kUnit;
            const uint32_t dst = (to ^ (swizzle_of<C::kRowBytes>(i * kRows, v) << 4)) + i * kRows * C::kRowBytes;
            if constexpr (decltype(all)::value)
              cp_async16(dst, src, policy);
            else
              cp_async16(dst, src, (live[z] >> row) & 1, policy);
          }
          if constexpr (kBits == 4) {
#pragma unroll
            for (int z = 0; z < kSub; ++z)
              cp_async_few<C::kScaleBytes>(to_scale + 32 * z * C::kScaleBytes, scales + static_cast<int64_t>(scale_at[z]) * kScaleUnit,
                                           decltype(all)::value || (live[z] >> lane) & 1);
          }
        };
        if (all_of(live))
          rows_at(std::true_type());
        else
          rows_at(std::false_type());
      }
    };

    bool more = at.u < hi;
    if (more) look_up();
    locate();
    copy(k_stage, a.k, false);
    cp_async_commit();
    copy(v_stage, a.v, true);
    cp_async_commit();
    // 8 bits: the upper half of its keys' power of two, the byte of its values', kNanValues
    constexpr uint32_t kNanValues = 0x100;
    uint32_t live_now[kSub], powers_now[kSub];
    auto take_over = [&] {  // the tile asked for is the one computed next
#pragma unroll
      for (int z = 0; z < kSub; ++z) {
        live_now[z] = live[z];
        if constexpr (kBits == 8)
          powers_now[z] = (__float_as_uint(power_value(k_power[z])) & 0xffff0000u) |
                          (v_power[z] == kNanScale ? kNanValues | 127u : static_cast<uint32_t>(min(max(v_power[z], kLeastPower), kMostPower)));
      }
    };
    take_over();
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
    bool beyond = false;  // of codes: the stretch has a reference beyond kNear
    uint32_t qf[D / 16][NT][2];
    const int g = lane >> 2, j = lane & 3;
    int t0 = 0, first = 0, heads = 0;
    bool fresh = true;
    const float scale_log2 = a.scale * kLog2e;
    // ldmatrix: lane's row of the first 16 and its chunk, exclusive or included; what
    // is added for later chunks touches other bits
    const uint32_t k_lane = k_stage + (lane & 15) * (D * 2) + (((lane >> 4) ^ (lane & 7)) << 4);
    const uint32_t v_lane = v_stage + ((lane & 7) + (lane >> 4) * 8) * (D * 2) + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);

    // Codes.  A fragment's row index i of 16 stands for row 4 (i / 2 % 4) + 2 (i / 8) + i % 2
    // of its group, so that the rows of K and of weights that a lane has in the products
    // with V are four neighbours; its places along D are the lane's own bytes of a row.
    constexpr int kGroups = kTile / 16;  // of 16 rows
    const int row_a = 4 * (g >> 1) + (g & 1);
    // first of the 4 values of D that the lane has in step ks
    auto k_first = [&](int ks) { return kBits == 4 ? D / 4 * j + 4 * ks : 16 * (j + 4 * (ks / 4)) + 4 * (ks % 4); };
    // q as fp16, times the sign of the scale and for each head the power of two that takes its
    // largest value to 2^14 and more: heads do not touch each other.
    auto to_halves = [&](uint32_t (&w)[D / 16][NT][2]) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t top = 0;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) top = max_of(top, max_of(w[ks][n][0], w[ks][n][1]));
        top = top_of(top);
        top = max(top, __shfl_xor_sync(~0u, top, 1));  // a head's values are in four lanes
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const int e = max(static_cast<int>(top >> 7) - 127 - 14, -126);
        const float by = copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), scale_log2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            w[ks][n][i] = pack_f16x2(__uint_as_float(w[ks][n][i] << 16) * by, __uint_as_float(w[ks][n][i] & 0xffff0000u) * by);
        // normal numbers: times a product of 0 it is that, and times -infinity
        const float unit = fminf(fmaxf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23) * fabsf(scale_log2), 0x1p-126f), 0x1.fffffep127f);
        if (j == 0) q_units[warp][8 * n + g] = unit;
      }
      __syncwarp();
    };
    // Words of codes of K that a lane takes up at a time from a row: 4 (of 8 codes for 2
    // steps, or of 4 for one), a 16-byte chunk, or the 2 that there are.
    constexpr int kWords = kBits == 4 ? D / 32 : 4, kParts = kBits == 8 ? D / 64 : 1, kSteps = kBits == 4 ? 2 : 1;
    // Part h of rows 16 x + row_a + 2 i.
    auto load_k = [&](int x, int i, int h, uint32_t (&w)[kWords], uint32_t (&by)[2]) {
      const int row = 16 * x + row_a + 2 * i;
      if constexpr (kBits == 8 || D == 128) {
        const uint4 q = at_shared<uint4>(k_codes + chunk_at<C::kRowBytes>(row, j + 4 * h, false));
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
      } else {
        const uint2 q = at_shared<uint2>(k_codes + chunk_at<C::kRowBytes>(row, j >> 1, false) + 8 * (j & 1));
        w[0] = q.x, w[1] = q.y;
      }
      if constexpr (kBits == 4) {
        const unsigned char* scales = k_codes + kTile * C::kRowBytes + row * C::kScaleBytes;
        if constexpr (D == 128) {
          const uint32_t c = at_shared<uint16_t>(scales + 2 * j);
          by[0] = (c & 0xffu) * 0x00800080u;
          by[1] = (c >> 8) * 0x00800080u;
        } else {
          by[0] = by[1] = at_shared<uint8_t>(scales + j) * 0x00800080u;
        }
      }
    };
    // Word t of a part: rows row_a + 2 i of the fragments of its steps.
    auto halves_of_k = [&](uint32_t w, const uint32_t (&by)[2], int t, int i, uint32_t (&f)[kSteps][4]) {
      if constexpr (kBits == 8) {
        halves_of_e4m3x4(w, f[0][i], f[0][2 + i]);
      } else {
        uint32_t h[4];
        halves_of_e2m1x8(w, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e / 2][2 * (e % 2) + i] = mul_f16x2(h[e], by[t / 2]);
      }
    };
    // Values D / 8 g and on of V, of rows 16 x + 4 j + r: words, and (4 bits) scales.
    constexpr int kVWords = kBits == 8 ? D / 32 : D / 64, kVTiles = kBits == 8 ? 2 : 4;  // of O a word
    auto load_v = [&](int x, uint32_t (&w)[4][kVWords], uint32_t (&by)[2]) {
      by[0] = by[1] = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * x + 4 * j + r;
        if constexpr (kVWords == 4) {
          const uint4 q = at_shared<uint4>(v_codes + chunk_at<C::kRowBytes>(row, g, true));
          w[r][0] = q.x, w[r][1] = q.y, w[r][2] = q.z, w[r][3] = q.w;
        } else if constexpr (kVWords == 2) {
          const uint2 q = at_shared<uint2>(v_codes + chunk_at<C::kRowBytes>(row, g >> 1, true) + 8 * (g & 1));
          w[r][0] = q.x, w[r][1] = q.y;
        } else {
          w[r][0] = at_shared<uint32_t>(v_codes + chunk_at<C::kRowBytes>(row, g >> 2, true) + 4 * (g & 3));
        }
        if constexpr (kBits == 4) {
          const unsigned char* scales = v_codes + kTile * C::kRowBytes + row * C::kScaleBytes;
          by[r / 2] += at_shared<uint8_t>(scales + (D == 128 ? g : g >> 1)) * (r % 2 ? 1u << 23 : 1u << 7);
        }
      }
    };
    // Word t of the rows: fragments of O's tiles kVTiles t and on.
    auto halves_of_v = [&](const uint32_t (&w)[4][kVWords], const uint32_t (&by)[2], int t, uint32_t (&f)[kVTiles][4]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // rows 2 i, 2 i + 1 of the four
        const uint32_t a = w[2 * i][t], b = w[2 * i + 1][t];
        if constexpr (kBits == 8) {
          halves_of_e4m3x4(__byte_perm(a, b, 0x5140), f[0][2 * i], f[0][2 * i + 1]);
          halves_of_e4m3x4(__byte_perm(a, b, 0x7362), f[1][2 * i], f[1][2 * i + 1]);
        } else {
          uint32_t even[4], odd[4];  // first and second value of each pair
          halves_of_e2m1x8((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), even);
          halves_of_e2m1x8(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), odd);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e][2 * i] = mul_f16x2(even[e], by[i]);
            f[e][2 * i + 1] = mul_f16x2(odd[e], by[i]);
          }
        }
      }
    };

    while (now.u < hi) {
      if (fresh) {
        fresh = false;
        beyond = false;
        t0 = now.t;
        heads_of<kSide>(a, now.vh * together + part, &first, &heads);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bool have = 8 * n + g < heads;
          const uint16_t* q = a.q + now.b * a.q_row + int64_t(first + 8 * n + (have ? g : 0)) * D + (kBits == 16 ? 2 * j : 0);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            if constexpr (kBits == 16) {
              qf[ks][n][0] = have ? *reinterpret_cast<const uint32_t*>(q + 16 * ks) : 0u;
              qf[ks][n][1] = have ? *reinterpret_cast<const uint32_t*>(q + 16 * ks + 8) : 0u;
            } else {
              const uint2 w = have ? *reinterpret_cast<const uint2*>(q + k_first(ks)) : make_uint2(0u, 0u);
              qf[ks][n][0] = w.x;
              qf[ks][n][1] = w.y;
            }
          }
          m[n][0] = m[n][1] = -INFINITY;
          l[n][0] = l[n][1] = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o_acc[i][n][e] = 0.f;
        }
        if constexpr (kBits < 16) to_halves(qf);
      }
      cp_async_wait<1>();  // K is here, V may be on its way
      __syncwarp();

      // scores of heads (2 j, 2 j + 1) and rows 16 x + (g, g + 8), of codes 16 x + (row_a, row_a + 2)
      float s[kGroups][NT][4];
#pragma unroll
      for (int x = 0; x < kGroups; ++x)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][n][e] = 0.f;
      if constexpr (kBits == 16) {
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
      } else {
        // two groups at a time: two chains of sums side by side
#pragma unroll
        for (int x = 0; x < kGroups; x += 2) {
#pragma unroll
          for (int h = 0; h < kParts; ++h) {
            uint32_t w[2][2][kWords], by[2][2][2];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int i = 0; i < 2; ++i) load_k(x + y, i, h, w[y][i], by[y][i]);
#pragma unroll
            for (int t = 0; t < kWords; ++t) {
              uint32_t f[2][kSteps][4];
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int i = 0; i < 2; ++i) halves_of_k(w[y][i][t], by[y][i], t, i, f[y]);
#pragma unroll
              for (int z = 0; z < kSteps; ++z)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    const int ks = (h * kWords + t) * kSteps + z;
                    mma_16816_f16(s[x + y][n], f[y][z], qf[ks][n][0], qf[ks][n][1]);
                  }
            }
          }
        }
      }
      __syncwarp();  // K is read
      if (more) {
        locate();
        copy(k_stage, a.k, false);
      }
      cp_async_commit();

      // 8 bits, of a row: its keys' power of two, by which its products are multiplied; what
      // its values' adds to the exponent, and 2 to the minus that.
      float v_log2[kGroups][2], v_inverse[kGroups][2];
      uint32_t nan_now[kSub] = {};
      bool nan_rows = false;
      if constexpr (kBits == 8) {
#pragma unroll
        for (int z = 0; z < kSub; ++z) {
          nan_now[z] = __ballot_sync(~0u, (powers_now[z] & kNanValues) != 0);
          nan_rows |= nan_now[z] != 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = 2 * z + i / 2, from = 16 * (i / 2) + row_a + 2 * (i % 2);
            const uint32_t both = __shfl_sync(~0u, powers_now[z], from), c = both & 0xffu;
            const float of_k = __uint_as_float(both & 0xffff0000u);
#pragma unroll
            for (int n = 0; n < NT; ++n) s[x][n][2 * (i % 2)] *= of_k, s[x][n][2 * (i % 2) + 1] *= of_k;
            v_log2[x][i % 2] = __uint_as_float(0x4b000000u | c) - (0x1p23f + 127.f);  // 2^23 + c: c as a number
            v_inverse[x][i % 2] = __uint_as_float((254u - c) << 23);
          }
        }
      }
      if constexpr (kBits < 16) {  // rows that are left out
        if (!all_of(live_now)) {
#pragma unroll
          for (int x = 0; x < kGroups; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((live_now[x / 2] >> (16 * (x % 2) + row_a + 2 * e)) & 1)) {
                if constexpr (kBits == 8) v_log2[x][e] = -INFINITY;
#pragma unroll
                for (int n = 0; n < NT; ++n) s[x][n][2 * e] = s[x][n][2 * e + 1] = kBits == 8 ? 0.f : -INFINITY;
              }
        }
      }

      float unit_log2[NT][2];
      if constexpr (kBits < 16) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 of = *reinterpret_cast<const float2*>(q_units[warp] + 8 * n + 2 * j);
          unit_log2[n][0] = of.x, unit_log2[n][1] = of.y;
        }
      }
      // The heads' largest scores, of codes plus their rows' powers.
      auto tops_of = [&](int n, float (&top)[2]) {
        top[0] = top[1] = -INFINITY;
#pragma unroll
        for (int x = 0; x < kGroups; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kBits == 16) {
              const bool counts = (live_now[0] >> (16 * x + g + (e >> 1) * 8)) & 1;
              s[x][n][e] = counts ? s[x][n][e] * scale_log2 : -INFINITY;
            }
            top[e & 1] = fmaxf(top[e & 1], kBits == 8 ? fmaf(s[x][n][e], unit_log2[n][e & 1], v_log2[x][e >> 1]) : s[x][n][e]);
          }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          top[0] = fmaxf(top[0], __shfl_xor_sync(~0u, top[0], x));
          top[1] = fmaxf(top[1], __shfl_xor_sync(~0u, top[1], x));
        }
        if constexpr (kBits == 8) top[0] -= kWeightBits, top[1] -= kWeightBits;
        if constexpr (kBits == 4) top[0] = fmaf(top[0], unit_log2[n][0], -kWeightBits), top[1] = fmaf(top[1], unit_log2[n][1], -kWeightBits);
      };
      // The reference to the larger one of itself and top.
      auto raise = [&](int n, const float (&top)[2]) {
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
      };
      // The same in a stretch with large scores.  These are rounded first, so that the largest
      // less the reference is 0 whatever its size.  s becomes the exponents of the weights.
      auto raise_beyond = [&](int n) {
        auto* const kept = large_of[warp] + 8 * n + 2 * j;  // heads 2 j and 2 j + 1
        if (!beyond) {
          if (g == 0) kept[0] = {m[n][0], kWeightBits, unit_log2[n][0]}, kept[1] = {m[n][1], kWeightBits, unit_log2[n][1]};
          __syncwarp();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m_was = kept[e].m, unit = kept[e].unit;
          float top = -INFINITY, most = -INFINITY;
#pragma unroll
          for (int x = 0; x < kGroups; ++x)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool out = kBits == 8 && v_log2[x][i] == -INFINITY;  // with 4 bits s is -infinity
              float& t = s[x][n][2 * i + e];
              t = out ? -INFINITY : t * unit;
              top = fmaxf(top, t);
            }
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
          const float up = fmaxf(m_was, top), ref = up == -INFINITY ? 0.f : up;
#pragma unroll
          for (int x = 0; x < kGroups; ++x)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& t = s[x][n][2 * i + e];
              t -= ref;
              if constexpr (kBits == 8) t += v_log2[x][i];
              most = fmaxf(most, t);
            }
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, x));
          const float was = kept[e].rho + (m_was - up);  // NaN or -infinity where there was no score
          const float rho = fmaxf(fmaxf(was, most), -48.f);
          const float keep = m_was == -INFINITY ? 0.f : fast_exp2(was - rho);
          __syncwarp();
          if (g == 0) kept[e].m = up, kept[e].rho = rho, q_units[warp][8 * n + 2 * j + e] = 1.f;
          m[n][e] = 0.f;
          unit_log2[n][e] = 1.f;
          l[n][e] *= keep;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) o_acc[i][n][e] *= keep, o_acc[i][n][2 + e] *= keep;
#pragma unroll
          for (int x = 0; x < kGroups; ++x) s[x][n][e] += kWeightBits - rho, s[x][n][2 + e] += kWeightBits - rho;
        }
        __syncwarp();
      };

      uint32_t hi_f[kGroups][NT][2], lo_f[kGroups][NT][2]  /* of codes: weights as fp16 alone */;
      // Weights exp2(s - m), of codes exp2(s unit + power - m), and their sums.
      auto weights = [&](int n) {
        const float ref[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
        for (int x = 0; x < kGroups; ++x) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kBits == 8) {
              p[e] = fast_exp2(fmaf(s[x][n][e], unit_log2[n][e & 1], v_log2[x][e >> 1] - ref[e & 1]));
              l[n][e & 1] = fmaf(p[e], v_inverse[x][e >> 1], l[n][e & 1]);
            } else {
              p[e] = fast_exp2(kBits == 4 ? fmaf(s[x][n][e], unit_log2[n][e & 1], -ref[e & 1]) : s[x][n][e] - ref[e & 1]);
              l[n][e & 1] += p[e];
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (kBits == 16) {
              uint32_t upper, lower;
              split_weights(p[2 * e], p[2 * e + 1], upper, lower);
              hi_f[x][n][e] = transpose8x8(upper);
              lo_f[x][n][e] = transpose8x8(lower);
            } else {
              uint32_t w = pack_f16x2(p[2 * e], p[2 * e + 1]);
              if (kBits == 8 && nan_rows && (nan_now[x / 2] >> (16 * (x % 2) + row_a + 2 * e)) & 1) w = 0x7fff7fffu;
              hi_f[x][n][e] = transpose8x8(w);
            }
          }
        }
      };
      if constexpr (kBits == 16) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float top[2];
          tops_of(n, top);
          if (__any_sync(~0u, top[0] > m[n][0] || top[1] > m[n][1])) raise(n, top);
          weights(n);
        }
      } else {
        float top[NT][2];
        bool higher = beyond, large = beyond;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          tops_of(n, top[n]);
#pragma unroll
          for (int e = 0; e < 2; ++e) higher |= top[n][e] > m[n][e];
        }
        if (__any_sync(~0u, higher)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float up = fabsf(fmaxf(m[n][e], top[n][e]));
              large |= up > kNear<kBits> && up < INFINITY;
            }
          if (__any_sync(~0u, large)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) raise_beyond(n);
            beyond = true;
            if constexpr (kBits == 8) {
#pragma unroll
              for (int x = 0; x < kGroups; ++x)
#pragma unroll
                for (int i = 0; i < 2; ++i) v_log2[x][i] = 0.f;
            }
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) raise(n, top[n]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) weights(n);
      }
      cp_async_wait<1>();  // V is here, the next K may be on its way
      __syncwarp();
      if constexpr (kBits == 16) {
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
      } else {
#pragma unroll
        for (int x = 0; x < kGroups; ++x) {
          uint32_t w[4][kVWords], by[2];
          load_v(x, w, by);
#pragma unroll
          for (int t = 0; t < kVWords; ++t) {
            uint32_t f[kVTiles][4];
            halves_of_v(w, by, t, f);
#pragma unroll
            for (int i = 0; i < kVTiles; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816_f16(o_acc[kVTiles * t + i][n], f[i], hi_f[x][n][0], hi_f[x][n][1]);
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
            float back = 1.f;
            if (kBits < 16 && beyond) m[n][e] = large_of[warp][head].m, back = fast_exp2(large_of[warp][head].rho - kWeightBits);
            if (whole) {
              if (g == 0 && head < heads) a.lse[int64_t(first + head) * a.B + now.b] = lse_of<kBits>(m[n][e], l[n][e] * back);
            } else if (g == 0) {
              sh.m[slot][head] = m[n][e];
              sh.l[slot][head] = l[n][e] * back;
            }
            const float by = whole ? inverse_of(l[n][e]) : back;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              if constexpr (kBits == 16) {
                to[o_at<kBits, D>(head, 16 * i + g)] = o_acc[i][n][e] * by;
                to[o_at<kBits, D>(head, 16 * i + g + 8)] = o_acc[i][n][2 + e] * by;
              } else {
                *reinterpret_cast<float2*>(to + o_at<kBits, D>(head, D / 8 * g + 2 * i)) =
                    make_float2(o_acc[i][n][e] * by, o_acc[i][n][2 + e] * by);
              }
            }
          }
        }
        __syncwarp();
        if (whole) {
          constexpr int kLanes = D / 4;
          for (int h = lane / kLanes; h < heads; h += 32 / kLanes) {
            const int d = 4 * (lane % kLanes);
            store_out4(a, D, now.b, first + h, d, *reinterpret_cast<const float4*>(to + o_at<kBits, D>(h, d)));
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
        copy(v_stage, a.v, true);
        take_over();
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
    for (int i = tid; i < a.H * (D / 4); i += kWarps * 32)
      store_out4(a, D, b, i / (D / 4), 4 * (i % (D / 4)), make_float4(0.f, 0.f, 0.f, 0.f));
    for (int h = tid; h < a.H; h += kWarps * 32) a.lse[int64_t(h) * a.B + b] = -INFINITY;
  }
  if (cta_n == 0) return;
  __syncthreads();

  // ---- parts of a row within this CTA's share
  auto part_o = [&](int slot) -> const float* {
    return reinterpret_cast<const float*>(smem + (slot >> 1) * C::kWarpBytes + C::kStageBytes + (slot & 1 ? 0 : C::kVBytes));
  };
  constexpr int kQuads = D / 4;
  uint32_t held, heads_at;  // slots that hold a part, and those where a row's first part is
  {
    static_assert(2 * kWarps <= 32, "a lane for each slot");
    const Stretch p = sh.part[lane & (2 * kWarps - 1)];
    const bool have = lane < 2 * kWarps && p.n > 0;
    held = __ballot_sync(~0u, have);
    const uint32_t below = held & ((1u << lane) - 1);
    const int prev = below ? 31 - __clz(below) : lane;
    const int prev_b = __shfl_sync(~0u, p.b, prev), prev_x = __shfl_sync(~0u, p.x, prev);
    heads_at = __ballot_sync(~0u, have && (!below || prev_b != p.b || prev_x != p.x));
  }
  // as many rows at once as have threads for their heads
  int row_threads = 32;
  while (row_threads < a.part_heads * kQuads && row_threads < kWarps * 32) row_threads *= 2;
  const int row_tid = tid & (row_threads - 1), my_turn = tid / row_threads, turns = kWarps * 32 / row_threads;
  // a slot of what goes on in other CTAs, by its place in global memory: 0 begun
  // before, 1 begun here (all parts of its query heads alike)
  int open[2] = {-1, -1};
  for (int turn = 0; heads_at; ++turn) {
    const int s = __ffs(heads_at) - 1;
    heads_at &= heads_at - 1;
    const uint32_t behind = heads_at ? ~0u << (__ffs(heads_at) - 1) : 0u;  // slots of later rows
    const uint32_t parts = held & ~behind & (~0u << s);
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
            v[x] = *reinterpret_cast<const float4*>(part_o(slot) + o_at<kBits, D>(h, d));
          }
        }
        sum.add(ml, v);
      }
      if (whole) {
        store_joined<kBits>(a, D, p.b, first + h, d, sum);
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
        constexpr int kThreads = kWarps * 32;
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
            store_joined<kBits>(a, D, p.b, first + h, d, sum[z]);
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

template <int kBits, int D, int NT, bool kSide, typename U>
cudaError_t launch(const ArgsOf<kBits>& a, int sms, cudaStream_t stream) {
  using C = DecodeCfg<kBits, D, NT>;
  static_assert(C::kCtasPerSm * (C::kSmemBytes + sizeof(DecodeShared<C::kWarps, NT>) + (kBits < 16 ? C::kWarps : 1) * C::kHeads * 16 + 1024) <= 233472, "shared memory of an SM");
  cudaError_t e = set_smem_limit_once<decode_kernel<kBits, D, NT, kSide, U>>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_overlapped(decode_kernel<kBits, D, NT, kSide, U>, dim3(sms * C::kCtasPerSm), C::kWarps * 32,
                           C::kSmemBytes, stream, a);
}

template <int kBits, int D, typename U>
cudaError_t launch_by_heads(const ArgsOf<kBits>& a, int sms, cudaStream_t stream) {
  if constexpr (kBits < 16) {
    if (a.mates > 1) return a.part_heads <= 8 ? launch<kBits, D, 1, true, U>(a, sms, stream) : launch<kBits, D, 2, true, U>(a, sms, stream);
  }
  if (a.together > 1) return launch<kBits, D, 2, true, U>(a, sms, stream);
  return a.part_heads <= 8 ? launch<kBits, D, 1, false, U>(a, sms, stream) : launch<kBits, D, 2, false, U>(a, sms, stream);
}

template <int kBits>
cudaError_t launch_by_size(const ArgsOf<kBits>& a, int sms, cudaStream_t stream, bool wide = false) {
  // the units of B full table rows
  constexpr int kTile = DecodeCfg<kBits, 128, 1>::kTile;
  static_assert(kTile == DecodeCfg<kBits, 64, 2>::kTile, "tiles go by the bits alone");
  const int64_t most = int64_t(a.B) * (int64_t(a.max_pages) * a.div.d / kTile + 1 + kRowUnits<kBits>);
  if (wide || most > UINT32_MAX / (a.Hkv * a.passes))
    return a.D == 128 ? launch_by_heads<kBits, 128, uint64_t>(a, sms, stream) : launch_by_heads<kBits, 64, uint64_t>(a, sms, stream);
  return a.D == 128 ? launch_by_heads<kBits, 128, uint32_t>(a, sms, stream) : launch_by_heads<kBits, 64, uint32_t>(a, sms, stream);
}

}  // namespace
}  // namespace jfa
