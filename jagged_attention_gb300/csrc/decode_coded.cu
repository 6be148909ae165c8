// decode_coded.cu -- attention over a cache of 8 or 4 bits.
#include "decode_kernel.cuh"

namespace jfa {

cudaError_t launch_decode_coded(const DecodeArgs& given, int sms, cudaStream_t stream) {
  DecodeArgs a = given;
  // Rows of neighbouring heads that share lines of 128 bytes, which is what memory gives
  // at once, are read side by side: 4 bits, 64 heads on 8 of 128, rows outside heads, TODO.
  const int row_bytes = a.D * a.bits / 8, mates = 128 / row_bytes;
  if (a.parts == 1 && mates > 1 && a.head == row_bytes && a.Hkv % mates == 0) {
    a.together = mates;
    a.vheads = a.Hkv / mates;
  }
  // whether 32 bits hold offsets as the kernel counts them
  const int n = a.bits == 8 ? 1 : a.D / kBlock;
  auto beyond = [&](int64_t page, int64_t row, int64_t head, int unit) {
    using Wide = __int128;
    return ((a.num_pages - 1) * Wide(page) + (a.div.d - 1) * Wide(row) + (a.Hkv - 1) * Wide(head)) / unit > UINT32_MAX;
  };
  const bool wide = beyond(a.page, a.row, a.head, 16) || beyond(a.scales.page, a.scales.row, a.scales.head, n);
  return a.bits == 8 ? launch_by_size<8>(a, sms, stream, wide) : launch_by_size<4>(a, sms, stream, wide);
}

}  // namespace jfa
