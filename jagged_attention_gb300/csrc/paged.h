// paged.h -- parameter blocks and launchers of the rotary and paged-cache
// kernels (internal), and the index arithmetic that host and device share.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace jfa {

// These kernels are launched before the one ahead of them in the stream has quite
// ended: they are set up while its last writes settle, and wait for those before
// they touch memory.  Back to back that takes 0.2 to 0.5 us off a call (letting go
// of the next kernel earlier, while this one still runs, gains nothing more).  As a
// kernel so begins before its inputs are final, nothing is read through the
// non-coherent cache.
#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_launch_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Adds one to a counter, releasing this thread's view of memory and acquiring the
// others': what was there before.
__device__ __forceinline__ int arrive(int* counter) {
  int was;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(was) : "l"(counter) : "memory");
  return was;
}
// Whether the caller is the last of `count` at a counter, which starts again then.
// A barrier before orders the other threads' writes, one behind their reads.
__device__ __forceinline__ bool last_of(int* counter, int count) {
  if (arrive(counter) != count - 1) return false;
  *counter = 0;
  return true;
}
template <typename K, typename... A>
cudaError_t launch_overlapped(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

// Bits of a pager's status word (JFA_PAGER_* in jfa.h).
enum PagerBits : int { kPagerNoPages = 1, kPagerBadLength = 2, kPagerBadPage = 4 };

// n / d for 0 <= n < 2^31 and a divisor fixed at creation: with 2^(s-1) < d <= 2^s
// and m = floor(2^(31+s) / d) + 1, m d = 2^(31+s) + e with 0 < e <= 2^s, so that
// n m / 2^(31+s) exceeds n / d by n e / (d 2^(31+s)) < 1 / d: the floors agree.
struct PageDiv {
  uint32_t mul;
  int shift;  // 31 + s
  int d;
  __host__ __device__ int quot(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
  }
};
inline PageDiv make_page_div(int d) {
  int s = 0;
  while ((int64_t(1) << s) < d) ++s;
  return {static_cast<uint32_t>((uint64_t(1) << (31 + s)) / static_cast<uint64_t>(d) + 1), 31 + s, d};
}

constexpr int kMaxPairs = 64;  // rotary pairs of a head (D <= 128)

// The rotation a handle holds: turn fractions and axes of its pairs.
struct Turns {
  uint64_t turn[kMaxPairs];  // inv_freq / (2 pi) in units of 2^-64
  uint8_t axis[kMaxPairs];
  int pairs;  // 0: nothing turns
  bool interleaved;
};

// One tensor of rows going through the row kernel.  Distances in elements.
struct RowJob {
  const void* in;
  void* out;
  int64_t in_row, out_row;
  int64_t out_page, out_head;  // out_page: scattered rows only
  int heads;
  bool f32, scatter, rotate;
};

struct RowsArgs {
  RowJob job[3];  // heads 0: unused
  int heads;      // of all jobs
  int D;
  int64_t rows;
  const int32_t* positions;
  int64_t pos_row, pos_axis;
  bool inverse;
  const int32_t* slots;  // scattered rows: slot of each row, negative: left out
  int64_t num_slots;
  PageDiv div;
  int* status;
  Turns turns;
};

// Where the scale bytes of a cache of 8 or 4 bits are, and their distances in bytes.
struct Scales {
  uint8_t *k, *v;
  int64_t page, row, head;
};

// Jobs 0 and 1 scatter K and V as codes (coded.cuh), their `out` and its distances in
// bytes.
struct CodedRowsArgs : RowsArgs {
  Scales scales;
};
cudaError_t launch_rows(const RowsArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_rows_coded(const CodedRowsArgs& a, int bits, int sms, cudaStream_t stream);

struct GatherArgs {
  int B, Hkv, D, bits;
  int max_pages;
  int64_t num_pages, rows;
  PageDiv div;
  const unsigned char *k, *v;  // pages, their distances in bytes
  int64_t page, row, head;
  Scales scales;
  const int32_t *table, *starts, *offsets;  // starts may be null: 0
  int64_t table_row;
  uint16_t *k_out, *v_out;
  int64_t k_row, v_row;  // elements from row to row
  int* status;
};
cudaError_t launch_gather(const GatherArgs& a, int sms, cudaStream_t stream);

struct TablesArgs {
  int B, max_pages;
  int64_t num_pages, rows;
  PageDiv div;
  const int32_t *lens, *delta, *n_free;
  int32_t *lens_out, *table, *free_list, *n_free_out, *slots, *positions, *row_offsets;
  int64_t table_row;
  int* status;
  int* counter;  // CTAs that are done; zero between launches
};
cudaError_t launch_tables(const TablesArgs& a, int sms, cudaStream_t stream);

struct DecodeArgs {
  int B, H, Hkv, D;
  int group;                                // H / Hkv
  int parts, together, passes, part_heads;  // QueryParts
  int64_t num_pages;
  int max_pages;
  PageDiv div;
  const uint16_t* q;
  int64_t q_row;
  const uint16_t *k, *v;   // or codes, whose distances count bytes
  int64_t page, row, head;
  const int32_t *table, *lens;
  int64_t table_row;
  float scale;
  uint16_t* out;
  float* lse;
  int* status;
  int* counters;             // arrivals at the parts of split rows; zero between launches
  float *part_ml, *part_o;   // what CTAs leave of split rows
};
struct CodedDecodeArgs : DecodeArgs {
  Scales scales;
  int mates;            // key/value heads that go side by side, 1 where none do,
  uint32_t mates_units; // if the requests have so many units,
  uint32_t far_units;   // and with so many their lines are not marked to leave L2 first
};
// A key/value head's query heads in parts of at most 16: `together` of them (1, 2,
// 4 or 8) side by side in a CTA, in `passes` over the cache.
struct QueryParts {
  int parts, together, passes, part_heads;
};
QueryParts query_parts(int group);
// Key/value heads that may go side by side over a cache of so many bits, 1 where none do.
int decode_mates(int bits, int D, int Hkv, const QueryParts& parts);

// Workspace of a decode launch: counters (int), part_ml and part_o (float).
struct DecodeSpace {
  int counters;
  int64_t part_ml, part_o;
};
DecodeSpace decode_space(int bits, int D, int Hkv, const QueryParts& parts, int sms);
cudaError_t launch_decode(const DecodeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_decode_coded(const DecodeArgs& a, const Scales& scales, int bits, int sms, cudaStream_t stream);

}  // namespace jfa
