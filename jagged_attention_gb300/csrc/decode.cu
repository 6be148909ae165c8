// decode.cu -- attention over a cache of bf16 rows, and what calls of any cache need.
#include <algorithm>

#include "decode_kernel.cuh"

namespace jfa {

DecodeSpace decode_space(int D, const QueryParts& parts, int sms) {
  const int heads = parts.part_heads <= 8 ? 8 : 16;
  const int ctas = sms * kMostCtasPerSm;  // one block for any number of bits
  // a counter for the row that begins in a CTA's share, two for groups that a CTA
  // leads; two places for each CTA and part
  const int64_t places = int64_t(ctas) * 2 * std::max(parts.together, parts.parts == 1 ? kMostMates : 1);
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
