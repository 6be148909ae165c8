// decode_coded.cu -- attention over a cache of 8 or 4 bits: how its launches differ.
#include <algorithm>

#include "decode_kernel.cuh"

namespace jfa {

namespace {

// Memory gives 128 bytes at a time, and gives 256 in a row faster.  Rows of neighbouring
// heads that lie within so much are read side by side, by warps of one CTA, where there is
// enough to read; in between the lines are in L2.  That halves the warps along a row and
// doubles the parts that CTAs join, which a single row feels most: just above the bounds it
// loses up to 3%, batches gain or lose nothing there.
//   rows of 64 and 32 bytes: 96 requests up to 32768 rows, 8 heads: 4 bits of 128 values 391
//   us, one head after the other 592; 8 bits of 64 values 288 and 542; 128 mixed requests,
//   126 MB, 40.4 and 42.9, 96, 95 MB, 33.5 and 34.7, 64, 64 MB, 27.2 and 27.5, 32, 34 MB, 20.9
//   and 18.8; one of 524288 rows of 4 heads, 302 MB, 75.3 and 86.2, of 262144, 151 MB, 48.1
//   and 46.9, of 131072, 76 MB, 32.5 and 29.8.
//   rows of 128 bytes: the full cache of 8 bits 541 us and 604 (of one GPU; of another 539
//   and 546), 512 mixed requests, 0.9 GB, 147 and 159, 128, 224 MB, 45 either way; one of
//   524288 rows, 541 MB, 90.4 and 89.1, of 131072, 135 MB, 34.1 and 29.7.
constexpr int kLineMb = 80, kPairMb = 256;

// Where so much is read as comes and goes in L2 meanwhile, 4-bit lines are not marked to
// leave first, or their second reader might miss them: the full cache 391 us, marked 398;
// 256 mixed requests, 250 MB, 69.9 and 67.9.  Of 8 bits they always are (not 549, marked 541).
constexpr int kFarMb = 512;

constexpr int kCodedTile = DecodeCfg<8, 128, 1>::kTile;
static_assert(kCodedTile == DecodeCfg<4, 128, 1>::kTile, "units of either");

}  // namespace

cudaError_t launch_decode_coded(const DecodeArgs& given, const Scales& scales, int bits, int sms, cudaStream_t stream) {
  CodedDecodeArgs a{given, scales, 1, 0, 0};
  const int row_bytes = a.D * bits / 8;
  const int mates = decode_mates(bits, a.D, a.Hkv, {a.parts, a.together, a.passes, a.part_heads});
  if (mates > 1 && a.head == row_bytes) {
    const int64_t unit = int64_t(2) * row_bytes * kCodedTile * a.Hkv;  // bytes of a tile of all heads
    auto units = [&](int mb) { return static_cast<uint32_t>((int64_t(mb) << 20) / unit); };
    a.mates = mates;
    a.mates_units = units(row_bytes < 128 ? kLineMb : kPairMb);
    a.far_units = bits == 4 ? units(kFarMb) : UINT32_MAX;
  }
  // whether 32 bits hold offsets as the kernel counts them
  const int n = bits == 8 ? 1 : a.D / kBlock;
  auto beyond = [&](int64_t page, int64_t row, int64_t head, int unit) {
    using Wide = __int128;
    return ((a.num_pages - 1) * Wide(page) + (a.div.d - 1) * Wide(row) + (a.Hkv - 1) * Wide(head)) / unit > UINT32_MAX;
  };
  const bool wide = beyond(a.page, a.row, a.head, 16) || beyond(a.scales.page, a.scales.row, a.scales.head, n);
  return bits == 8 ? launch_by_size<8>(a, sms, stream, wide) : launch_by_size<4>(a, sms, stream, wide);
}

}  // namespace jfa
