// decode.cu -- attention over a cache of bf16 rows, and what calls of any cache need.
#include <algorithm>

#include "decode_kernel.cuh"

namespace jfa {

namespace {

template <int kBits>
int ctas_per_sm(int D, int heads) {
  if (D == 64) return heads == 8 ? DecodeCfg<kBits, 64, 1>::kCtasPerSm : DecodeCfg<kBits, 64, 2>::kCtasPerSm;
  return heads == 8 ? DecodeCfg<kBits, 128, 1>::kCtasPerSm : DecodeCfg<kBits, 128, 2>::kCtasPerSm;
}

}  // namespace

// Rows below 128 bytes: as many as fill them; else two.
int decode_mates(int bits, int D, int Hkv, const QueryParts& parts) {
  const int row_bytes = D * bits / 8, mates = row_bytes < 128 ? 128 / row_bytes : 2;
  return bits < 16 && parts.parts == 1 && Hkv % mates == 0 ? mates : 1;
}

DecodeSpace decode_space(int bits, int D, int Hkv, const QueryParts& parts, int sms) {
  const int heads = parts.part_heads <= 8 ? 8 : 16;
  const int ctas = sms * (bits == 16 ? ctas_per_sm<16>(D, heads) : bits == 8 ? ctas_per_sm<8>(D, heads) : ctas_per_sm<4>(D, heads));
  // a counter for the row that begins in a CTA's share, two for groups that a CTA
  // leads; two places for each CTA and part
  const int64_t places = int64_t(ctas) * 2 * std::max(parts.together, decode_mates(bits, D, Hkv, parts));
  return {3 * ctas, places * heads * 2, places * heads * D};
}

QueryParts query_parts(int group) {
  QueryParts k{1, 1, 1, group};
  while (k.together < kMostTogether && k.together * kMostHeads < group) k.together *= 2;
  k.passes = (group + kMostHeads * k.together - 1) / (kMostHeads * k.together);
  k.parts = k.passes * k.together;
  k.part_heads = (group + k.parts - 1) / k.parts;  // above 8 where there are parts
  return k;
}

cudaError_t launch_decode(const DecodeArgs& a, int sms, cudaStream_t stream) { return launch_by_size<16>(a, sms, stream); }

}  // namespace jfa
