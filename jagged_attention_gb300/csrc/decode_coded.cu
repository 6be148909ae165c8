// decode_coded.cu -- attention over a cache of 8 or 4 bits.
#include "decode_kernel.cuh"

namespace jfa {

cudaError_t launch_decode_coded(const DecodeArgs& a, int sms, cudaStream_t stream) {
  return a.bits == 8 ? launch_by_size<8>(a, sms, stream) : launch_by_size<4>(a, sms, stream);
}

}  // namespace jfa
