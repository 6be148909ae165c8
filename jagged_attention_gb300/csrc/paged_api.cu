// paged_api.cu -- the C ABI of the rotary and paged-cache operators declared
// in include/jfa.h: argument checks, handles and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <new>

#include "jfa.h"
#include "paged.h"

struct jfa_rotary {
  int D;
  jfa::Turns turns;
};

struct jfa_pager {
  int max_seqs, max_pages, H, Hkv, D, bits, device, sms;
  jfa::QueryParts parts;
  int64_t num_pages;
  jfa::PageDiv div;
  int *d_status, *d_counters;  // in the caller's block, as the rest
  float *d_part_ml, *d_part_o;
};

namespace {

static_assert(JFA_PAGER_NO_PAGES == jfa::kPagerNoPages && JFA_PAGER_BAD_LENGTH == jfa::kPagerBadLength &&
                  JFA_PAGER_BAD_PAGE == jfa::kPagerBadPage,
              "status bits");

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// floor(x * 2^64 / (2 pi) + 1/2) modulo 2^64 for a finite |x| < 2^31, from the
// binary digits of 1 / (2 pi): x = m 2^e with |m| < 2^53, and m times the 192
// leading digits, shifted to the place of the 64 fraction bits.
uint64_t turn_fraction(double x) {
  // 1 / (2 pi) = 0.15915494309189533576888376337251... in base 2^64
  static const uint64_t kDigits[3] = {0x28BE60DB9391054Aull, 0x7F09D5F47D4D3770ull, 0x36D8A5664F10E410ull};
  int e = 0;
  const double f = std::frexp(std::fabs(x), &e);               // f in [1/2, 1)
  const uint64_t m = static_cast<uint64_t>(std::ldexp(f, 53));  // x = m 2^(e - 53)
  if (m == 0) return 0;
  // the product of m and the digits: four words, the first above the point
  uint64_t w[4];
  unsigned __int128 carry = 0;
  for (int i = 2; i >= 0; --i) {
    carry += static_cast<unsigned __int128>(m) * kDigits[i];
    w[i + 1] = static_cast<uint64_t>(carry);
    carry >>= 64;
  }
  w[0] = static_cast<uint64_t>(carry);
  // value = (w0 . w1 w2 w3) * 2^(e - 53); wanted: its first 64 fraction bits, rounded
  const int shift = e - 53;  // -1127 .. -22
  const int down = -shift;   // fraction word = bits of w at 64 fraction places, shifted right by `down`
  auto word = [&](int i) { return i < 0 || i > 3 ? uint64_t(0) : w[i]; };
  const int whole = down / 64, part = down % 64;
  // fraction word after the shift: bits from words 1 - whole and before
  uint64_t value = word(1 - whole) >> part;
  if (part) value |= word(-whole) << (64 - part);
  const uint64_t round = part ? (word(1 - whole) >> (part - 1)) & 1 : (word(2 - whole) >> 63) & 1;
  value += round;
  return x < 0 ? ~value + 1 : value;
}

int check_device(const jfa_pager* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return JFA_ERR_CUDA;
  return dev == p->device ? JFA_OK : JFA_ERR_INVALID_ARG;
}

// SMs of the current device, JFA_ERR_UNSUPPORTED where this library does not run on it.
int sm_count(int* sms) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 0: not asked yet; what a device is does not change
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return JFA_ERR_CUDA;
  if (dev < kDevices && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return JFA_OK;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return JFA_ERR_CUDA;
  if (major != 10 || minor != 3) return JFA_ERR_UNSUPPORTED;  // built for sm_103a only
  if (dev < kDevices) known[dev].store(*sms, std::memory_order_relaxed);
  return JFA_OK;
}

// One tensor of `heads` heads a row, `row` elements from row to row.
int check_rows(const void* p, int64_t row, int heads, int D, bool f32) {
  if (!p || row < int64_t(heads) * D) return JFA_ERR_INVALID_ARG;
  if (!aligned(p, 16) || row % (f32 ? 4 : 8) != 0) return JFA_ERR_ALIGNMENT;
  return JFA_OK;
}

// Whether p and q overlap nowhere: `rows` rows of n bf16 values each, p's one behind
// the other and q's q_row >= n values apart.
bool apart(const void* p, const void* q, int64_t rows, int64_t n, int64_t q_row) {
  using Wide = unsigned __int128;
  const Wide at = reinterpret_cast<uintptr_t>(p), from = reinterpret_cast<uintptr_t>(q);
  return at + 2 * Wide(rows) * n <= from || from + 2 * (Wide(rows - 1) * q_row + n) <= at;
}

// Whether two outputs of `rows` rows of n bf16 values overlap nowhere: apart as a whole, or
// side by side in rows the same distance apart (of a fused tensor, say).
bool side_by_side(const void* p, int64_t p_row, const void* q, int64_t q_row, int64_t rows, int64_t n) {
  using Wide = unsigned __int128;
  const Wide a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  if (a + 2 * (Wide(rows - 1) * p_row + n) <= b || b + 2 * (Wide(rows - 1) * q_row + n) <= a) return true;
  if (p_row != q_row) return false;
  const Wide row = 2 * Wide(p_row), d = (a < b ? b - a : a - b) % row;
  return d >= 2 * Wide(n) && d + 2 * Wide(n) <= row;
}

int check_pages(const jfa_pages* g) {
  if (!g || !g->k || !g->v || g->page < 0 || g->row < 0 || g->head < 0) return JFA_ERR_INVALID_ARG;
  if (!aligned(g->k, 16) || !aligned(g->v, 16) || g->page % 8 || g->row % 8 || g->head % 8)
    return JFA_ERR_ALIGNMENT;
  return JFA_OK;
}

// Pages and scales of a cache of `bits` bits.  Codes are copied 16 bytes at a time,
// scale bytes a row's head at a time.
int check_cache(const jfa_pager* p, const jfa_pages* g, const jfa_scales* s) {
  if ((p->bits < 16) != (s != nullptr)) return JFA_ERR_INVALID_ARG;
  if (int rc = check_pages(g)) return rc;
  if (p->bits == 16) return JFA_OK;
  if (!s->k || !s->v || s->page < 0 || s->row < 0 || s->head < 0) return JFA_ERR_INVALID_ARG;
  if (g->page % 16 || g->row % 16 || g->head % 16) return JFA_ERR_ALIGNMENT;
  const int n = p->bits == 8 ? 1 : p->D / 16;
  if (!aligned(s->k, n) || !aligned(s->v, n) || s->page % n || s->row % n || s->head % n) return JFA_ERR_ALIGNMENT;
  return JFA_OK;
}
jfa::Scales scales_of(const jfa_scales* s) {
  if (!s) return {};
  return {static_cast<uint8_t*>(s->k), static_cast<uint8_t*>(s->v), s->page, s->row, s->head};
}

// A pager's block: status word, counters, then what split rows leave.
struct Block {
  size_t counters, part_ml, part_o, bytes;
  jfa::QueryParts parts;
};
Block block_of(int bits, int H, int Hkv, int D, int sms) {
  Block k;
  k.parts = jfa::query_parts(H / Hkv);
  const jfa::DecodeSpace n = jfa::decode_space(bits, D, Hkv, k.parts, sms);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  k.counters = 256;
  k.part_ml = up(k.counters + n.counters * sizeof(int));
  k.part_o = up(k.part_ml + n.part_ml * sizeof(float));
  k.bytes = up(k.part_o + n.part_o * sizeof(float));
  return k;
}
// Bits of a pager with these flags, 0: no such flags.
int bits_of(unsigned flags) {
  return flags == 0 ? 16 : flags == JFA_PAGER_8BIT ? 8 : flags == JFA_PAGER_4BIT ? 4 : 0;
}
int check_heads(int H, int Hkv, int D) {
  if (Hkv < 1 || H < Hkv || H % Hkv) return JFA_ERR_INVALID_ARG;
  return (D != 64 && D != 128) || H > 65535 ? JFA_ERR_UNSUPPORTED : JFA_OK;
}

jfa::RowJob dense_job(const void* in, int64_t in_row, void* out, int64_t out_row, int heads, int D,
                      bool f32, bool rotate) {
  return {in, out, in_row, out_row, 0, D, heads, f32, false, rotate};
}

// rows of one launch: the grid's first dimension holds 2^31 - 1 blocks of at least 8 rows
constexpr int64_t kMaxRows = int64_t(1) << 33;

}  // namespace

extern "C" {

int jfa_rotary_turns(const double* inv_freq_host, int pairs, uint64_t* turns_out) {
  if (!inv_freq_host || !turns_out || pairs < 0) return JFA_ERR_INVALID_ARG;
  for (int i = 0; i < pairs; ++i)
    if (!(std::fabs(inv_freq_host[i]) < 2147483648.0)) return JFA_ERR_INVALID_ARG;  // NaN too
  for (int i = 0; i < pairs; ++i) turns_out[i] = turn_fraction(inv_freq_host[i]);
  return JFA_OK;
}

int jfa_rotary_create(const double* inv_freq_host, const int32_t* axis_host, int pairs, int D,
                      unsigned flags, jfa_rotary_t* out) {
  if (!out || !inv_freq_host || !axis_host || (flags & ~JFA_ROTARY_INTERLEAVED)) return JFA_ERR_INVALID_ARG;
  *out = nullptr;
  if (D != 64 && D != 128) return JFA_ERR_UNSUPPORTED;
  if (pairs < 8 || 2 * pairs > D || pairs % 8) return JFA_ERR_INVALID_ARG;
  for (int i = 0; i < pairs; ++i)
    if (axis_host[i] < 0 || axis_host[i] > 3) return JFA_ERR_INVALID_ARG;
  jfa_rotary r{};
  r.D = D;
  if (int rc = jfa_rotary_turns(inv_freq_host, pairs, r.turns.turn)) return rc;
  for (int i = 0; i < pairs; ++i) r.turns.axis[i] = static_cast<uint8_t>(axis_host[i]);
  r.turns.pairs = pairs;
  r.turns.interleaved = (flags & JFA_ROTARY_INTERLEAVED) != 0;
  *out = new (std::nothrow) jfa_rotary(r);
  return *out ? JFA_OK : JFA_ERR_WORKSPACE;
}

int jfa_rotary_destroy(jfa_rotary_t rotary) {
  if (!rotary) return JFA_ERR_INVALID_ARG;
  delete rotary;
  return JFA_OK;
}

int jfa_rotate(jfa_rotary_t rotary, const int32_t* positions, int64_t pos_row, int64_t pos_axis,
               int64_t rows, unsigned flags, const void* x, int64_t x_row, void* x_out,
               int64_t x_out_row, int x_heads, const void* y, int64_t y_row, void* y_out,
               int64_t y_out_row, int y_heads, void* stream) {
  if (!rotary || rows < 0 || rows >= kMaxRows || pos_row < 0 || pos_axis < 0 ||
      (flags & ~(JFA_ROTATE_INVERSE | JFA_ROTATE_X_FP32 | JFA_ROTATE_Y_FP32)) || x_heads < 1 ||
      y_heads < 0 || x_heads > INT_MAX - y_heads)
    return JFA_ERR_INVALID_ARG;
  if (rows == 0) return JFA_OK;
  if (!positions || (y_heads == 0) != (y == nullptr)) return JFA_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return JFA_ERR_ALIGNMENT;
  const int D = rotary->D;
  const bool x32 = flags & JFA_ROTATE_X_FP32, y32 = flags & JFA_ROTATE_Y_FP32;
  if (int rc = check_rows(x, x_row, x_heads, D, x32)) return rc;
  if (int rc = check_rows(x_out, x_out_row, x_heads, D, x32)) return rc;
  if (y) {
    if (int rc = check_rows(y, y_row, y_heads, D, y32)) return rc;
    if (int rc = check_rows(y_out, y_out_row, y_heads, D, y32)) return rc;
  }
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  jfa::RowsArgs a{};
  a.job[0] = dense_job(x, x_row, x_out, x_out_row, x_heads, D, x32, true);
  if (y) a.job[1] = dense_job(y, y_row, y_out, y_out_row, y_heads, D, y32, true);
  a.heads = x_heads + y_heads;
  a.D = D;
  a.rows = rows;
  a.positions = positions;
  a.pos_row = pos_row;
  a.pos_axis = pos_axis;
  a.inverse = flags & JFA_ROTATE_INVERSE;
  a.turns = rotary->turns;
  return jfa::launch_rows(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

size_t jfa_pager_block_bytes_ex(int H, int Hkv, int D, unsigned flags) {
  int sms = 0;
  if (!bits_of(flags) || check_heads(H, Hkv, D) != JFA_OK || sm_count(&sms) != JFA_OK) return 0;
  return block_of(bits_of(flags), H, Hkv, D, sms).bytes;
}

size_t jfa_pager_block_bytes(int H, int Hkv, int D) {
  size_t most = 0;
  for (unsigned flags : {0u, JFA_PAGER_8BIT, JFA_PAGER_4BIT}) most = std::max(most, jfa_pager_block_bytes_ex(H, Hkv, D, flags));
  return most;
}

int jfa_pager_create(int max_seqs, int max_pages, int64_t num_pages, int page_size, int H, int Hkv,
                     int D, void* block, size_t block_bytes, void* stream, jfa_pager_t* out) {
  return jfa_pager_create_ex(max_seqs, max_pages, num_pages, page_size, H, Hkv, D, 0, block, block_bytes, stream, out);
}

int jfa_pager_create_ex(int max_seqs, int max_pages, int64_t num_pages, int page_size, int H, int Hkv,
                        int D, unsigned flags, void* block, size_t block_bytes, void* stream, jfa_pager_t* out) {
  if (!out) return JFA_ERR_INVALID_ARG;
  *out = nullptr;
  const int bits = bits_of(flags);
  if (!bits) return JFA_ERR_INVALID_ARG;
  if (max_seqs < 1 || max_pages < 1 || num_pages < 1 || page_size < 1) return JFA_ERR_INVALID_ARG;
  if (int rc = check_heads(H, Hkv, D)) return rc;
  if (max_seqs > JFA_PAGER_MAX_SEQS || num_pages > INT_MAX ||
      (int64_t(max_pages) + 1) * page_size > INT_MAX || (num_pages + 1) * page_size > INT_MAX)
    return JFA_ERR_UNSUPPORTED;
  if (!aligned(block, 256)) return JFA_ERR_ALIGNMENT;
  int sms = 0, dev = 0;
  if (int rc = sm_count(&sms)) return rc;
  if (cudaGetDevice(&dev) != cudaSuccess) return JFA_ERR_CUDA;
  const Block k = block_of(bits, H, Hkv, D, sms);
  if (!block || block_bytes < k.bytes) return JFA_ERR_WORKSPACE;
  auto* base = static_cast<unsigned char*>(block);
  if (cudaMemsetAsync(base, 0, k.part_ml, static_cast<cudaStream_t>(stream)) != cudaSuccess) return JFA_ERR_CUDA;
  auto* p = new (std::nothrow) jfa_pager;
  if (!p) return JFA_ERR_WORKSPACE;
  p->max_seqs = max_seqs;
  p->max_pages = max_pages;
  p->H = H;
  p->Hkv = Hkv;
  p->D = D;
  p->bits = bits;
  p->device = dev;
  p->sms = sms;
  p->parts = k.parts;
  p->num_pages = num_pages;
  p->div = jfa::make_page_div(page_size);
  p->d_status = reinterpret_cast<int*>(base);
  p->d_counters = reinterpret_cast<int*>(base + k.counters);
  p->d_part_ml = reinterpret_cast<float*>(base + k.part_ml);
  p->d_part_o = reinterpret_cast<float*>(base + k.part_o);
  *out = p;
  return JFA_OK;
}

int jfa_pager_destroy(jfa_pager_t pager) {
  if (!pager) return JFA_ERR_INVALID_ARG;
  delete pager;
  return JFA_OK;
}

int jfa_pager_status(jfa_pager_t pager, void* stream, int* raw) {
  if (!pager) return JFA_ERR_INVALID_ARG;
  if (int rc = check_device(pager)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int word = 0;
  if (cudaMemcpyAsync(&word, pager->d_status, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return JFA_ERR_CUDA;
  if (raw) *raw = word;
  if (word == 0) return JFA_OK;
  if (cudaMemsetAsync(pager->d_status, 0, sizeof(int), s) != cudaSuccess) return JFA_ERR_CUDA;
  return JFA_ERR_PAGES;
}

int jfa_paged_tables(jfa_pager_t pager, int B, const int32_t* lens, const int32_t* delta,
                     int32_t* lens_out, int32_t* table, int64_t table_row, int32_t* free_list,
                     const int32_t* n_free, int32_t* n_free_out, int64_t rows, int32_t* slots,
                     int32_t* positions, int32_t* row_offsets, void* stream) {
  if (!pager || B < 1 || B > pager->max_seqs || rows < 0 || rows > INT_MAX) return JFA_ERR_INVALID_ARG;
  if (!lens || !delta || !lens_out || !table || !free_list || !n_free || !n_free_out || !row_offsets ||
      (rows > 0 && (!slots || !positions)) || table_row < pager->max_pages)
    return JFA_ERR_INVALID_ARG;
  if (lens_out == delta || n_free_out == lens_out) return JFA_ERR_INVALID_ARG;  // read or written by others meanwhile
  const void* ptrs[] = {lens, delta, lens_out, table, free_list, n_free, n_free_out, slots, positions, row_offsets};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return JFA_ERR_ALIGNMENT;
  if (int rc = check_device(pager)) return rc;
  jfa::TablesArgs a{};
  a.B = B;
  a.max_pages = pager->max_pages;
  a.num_pages = pager->num_pages;
  a.rows = rows;
  a.div = pager->div;
  a.lens = lens;
  a.delta = delta;
  a.n_free = n_free;
  a.lens_out = lens_out;
  a.table = table;
  a.free_list = free_list;
  a.n_free_out = n_free_out;
  a.slots = slots;
  a.positions = positions;
  a.row_offsets = row_offsets;
  a.table_row = table_row;
  a.status = pager->d_status;
  a.counter = pager->d_status + 16;  // in the block's first 256 bytes, as the status word
  return jfa::launch_tables(a, pager->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

int jfa_paged_append(jfa_pager_t pager, int64_t rows, const void* k, int64_t k_row, const void* v,
                     int64_t v_row, const int32_t* slots, const jfa_pages* pages,
                     jfa_rotary_t rotary, const int32_t* positions, int64_t pos_row,
                     int64_t pos_axis, const void* q, int64_t q_row, void* q_out, int64_t q_out_row,
                     void* stream) {
  return jfa_paged_append_ex(pager, rows, k, k_row, v, v_row, slots, pages, nullptr, rotary, positions, pos_row,
                             pos_axis, q, q_row, q_out, q_out_row, stream);
}

int jfa_paged_append_ex(jfa_pager_t pager, int64_t rows, const void* k, int64_t k_row, const void* v,
                        int64_t v_row, const int32_t* slots, const jfa_pages* pages,
                        const jfa_scales* scales, jfa_rotary_t rotary, const int32_t* positions,
                        int64_t pos_row, int64_t pos_axis, const void* q, int64_t q_row, void* q_out,
                        int64_t q_out_row, void* stream) {
  if (!pager || rows < 0 || rows >= kMaxRows || pos_row < 0 || pos_axis < 0) return JFA_ERR_INVALID_ARG;
  if (!rotary && (positions || q || q_out)) return JFA_ERR_INVALID_ARG;
  if (rotary && rotary->D != pager->D) return JFA_ERR_INVALID_ARG;
  if (rows == 0) return JFA_OK;
  if (!slots || (rotary && !positions) || (q == nullptr) != (q_out == nullptr)) return JFA_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(positions, 4)) return JFA_ERR_ALIGNMENT;
  const int D = pager->D;
  if (int rc = check_rows(k, k_row, pager->Hkv, D, false)) return rc;
  if (int rc = check_rows(v, v_row, pager->Hkv, D, false)) return rc;
  if (int rc = check_cache(pager, pages, scales)) return rc;
  if (q) {
    if (int rc = check_rows(q, q_row, pager->H, D, false)) return rc;
    if (int rc = check_rows(q_out, q_out_row, pager->H, D, false)) return rc;
  }
  if (int rc = check_device(pager)) return rc;
  jfa::CodedRowsArgs a{};
  a.job[0] = {k, pages->k, k_row, pages->row, pages->page, pages->head, pager->Hkv, false, true, rotary != nullptr};
  a.job[1] = {v, pages->v, v_row, pages->row, pages->page, pages->head, pager->Hkv, false, true, false};
  a.scales = scales_of(scales);
  if (q) a.job[2] = dense_job(q, q_row, q_out, q_out_row, pager->H, D, false, true);
  a.heads = 2 * pager->Hkv + (q ? pager->H : 0);
  a.D = D;
  a.rows = rows;
  a.positions = positions;
  a.pos_row = pos_row;
  a.pos_axis = pos_axis;
  a.slots = slots;
  a.num_slots = pager->num_pages * pager->div.d;
  a.div = pager->div;
  a.status = pager->d_status;
  if (rotary) a.turns = rotary->turns;
  const auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pager->bits == 16 ? jfa::launch_rows(a, pager->sms, s) : jfa::launch_rows_coded(a, pager->bits, pager->sms, s);
  return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

int jfa_paged_decode(jfa_pager_t pager, int B, const void* q, int64_t q_row, const jfa_pages* pages,
                     const int32_t* table, int64_t table_row, const int32_t* lens, float scale,
                     void* out, float* lse, void* stream) {
  return jfa_paged_decode_ex(pager, B, q, q_row, pages, nullptr, table, table_row, lens, scale, out, lse, stream);
}

int jfa_paged_decode_ex(jfa_pager_t pager, int B, const void* q, int64_t q_row, const jfa_pages* pages,
                        const jfa_scales* scales, const int32_t* table, int64_t table_row,
                        const int32_t* lens, float scale, void* out, float* lse, void* stream) {
  if (!pager || B < 1 || B > pager->max_seqs) return JFA_ERR_INVALID_ARG;
  if (!(std::fabs(scale) < 0x1p127f)) return JFA_ERR_INVALID_ARG;  // times log2 e it is finite; NaN too
  if (!table || !lens || !out || !lse || table_row < pager->max_pages) return JFA_ERR_INVALID_ARG;
  if (int rc = check_rows(q, q_row, pager->H, pager->D, false)) return rc;
  if (int rc = check_cache(pager, pages, scales)) return rc;
  if (pager->div.d > 1 && (pages->row > UINT32_MAX || (scales && scales->row > UINT32_MAX))) return JFA_ERR_UNSUPPORTED;
  if (!aligned(out, 16) || !aligned(lse, 16) || !aligned(table, 4) || !aligned(lens, 4)) return JFA_ERR_ALIGNMENT;
  // a row of out may be written while another CTA still reads its query
  if (!apart(out, q, B, int64_t(pager->H) * pager->D, q_row)) return JFA_ERR_INVALID_ARG;
  if (int rc = check_device(pager)) return rc;
  jfa::DecodeArgs a{};
  a.B = B;
  a.H = pager->H;
  a.Hkv = pager->Hkv;
  a.D = pager->D;
  a.group = pager->H / pager->Hkv;
  a.parts = pager->parts.parts;
  a.together = pager->parts.together;
  a.passes = pager->parts.passes;
  a.part_heads = pager->parts.part_heads;
  a.num_pages = pager->num_pages;
  a.max_pages = pager->max_pages;
  a.div = pager->div;
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row;
  a.k = static_cast<const uint16_t*>(pages->k);
  a.v = static_cast<const uint16_t*>(pages->v);
  a.page = pages->page;
  a.row = pages->row;
  a.head = pages->head;
  a.table = table;
  a.table_row = table_row;
  a.lens = lens;
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = pager->d_status;
  a.counters = pager->d_counters;
  a.part_ml = pager->d_part_ml;
  a.part_o = pager->d_part_o;
  const auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pager->bits == 16 ? jfa::launch_decode(a, pager->sms, s)
                                          : jfa::launch_decode_coded(a, scales_of(scales), pager->bits, pager->sms, s);
  return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

int jfa_paged_gather(jfa_pager_t pager, int B, const jfa_pages* pages, const jfa_scales* scales,
                     const int32_t* table, int64_t table_row, const int32_t* starts,
                     const int32_t* offsets, int64_t rows, void* k_out, int64_t k_row, void* v_out,
                     int64_t v_row, void* stream) {
  if (!pager || B < 1 || B > pager->max_seqs || rows < 0 || rows > INT_MAX) return JFA_ERR_INVALID_ARG;
  if (!offsets) return JFA_ERR_INVALID_ARG;
  if (!aligned(offsets, 4)) return JFA_ERR_ALIGNMENT;
  jfa::GatherArgs a{};
  a.B = B;
  a.bits = pager->bits;
  a.rows = rows;
  a.offsets = offsets;
  a.status = pager->d_status;
  const auto s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // whether the offsets say so too
    if (int rc = check_device(pager)) return rc;
    return jfa::launch_gather(a, pager->sms, s) == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
  }
  if (!table || table_row < pager->max_pages) return JFA_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(starts, 4)) return JFA_ERR_ALIGNMENT;
  if (int rc = check_cache(pager, pages, scales)) return rc;
  if (int rc = check_rows(k_out, k_row, pager->Hkv, pager->D, false)) return rc;
  if (int rc = check_rows(v_out, v_row, pager->Hkv, pager->D, false)) return rc;
  if (!side_by_side(k_out, k_row, v_out, v_row, rows, int64_t(pager->Hkv) * pager->D)) return JFA_ERR_INVALID_ARG;
  if (int rc = check_device(pager)) return rc;
  const int unit = pager->bits == 16 ? 2 : 1;  // bytes of an element of the pages
  a.Hkv = pager->Hkv;
  a.D = pager->D;
  a.max_pages = pager->max_pages;
  a.num_pages = pager->num_pages;
  a.div = pager->div;
  a.k = static_cast<const unsigned char*>(pages->k);
  a.v = static_cast<const unsigned char*>(pages->v);
  a.page = pages->page * unit;
  a.row = pages->row * unit;
  a.head = pages->head * unit;
  a.scales = scales_of(scales);
  a.table = table;
  a.starts = starts;
  a.table_row = table_row;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.k_row = k_row;
  a.v_row = v_row;
  return jfa::launch_gather(a, pager->sms, s) == cudaSuccess ? JFA_OK : JFA_ERR_CUDA;
}

}  // extern "C"
