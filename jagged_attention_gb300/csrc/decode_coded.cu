// decode_coded.cu -- attention over a cache of 8 or 4 bits.
#include "decode_kernel.cuh"

namespace jfa {

constexpr int kLineMb = 96, kMatesMb = 2048, kFarMb = 512;

cudaError_t launch_decode_coded(const DecodeArgs& given, int sms, cudaStream_t stream) {
  DecodeArgs a = given;
  // Rows of neighbouring heads are read side by side where there is enough to read: TODO.
  const int row_bytes = a.D * a.bits / 8, mates = row_bytes < 128 ? 128 / row_bytes : 2;
  const int64_t least = int64_t(row_bytes < 128 ? kLineMb : kMatesMb) << 20;
  if (a.parts == 1 && a.head == row_bytes && a.Hkv % mates == 0) {
    a.mates = mates;
    const int64_t unit = 2 * row_bytes * (a.bits == 8 ? 32 : 64) * a.Hkv;  // of all heads
    a.mates_units = static_cast<uint32_t>(least / unit);
    a.far_units = static_cast<uint32_t>((int64_t(kFarMb) << 20) / unit);
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
