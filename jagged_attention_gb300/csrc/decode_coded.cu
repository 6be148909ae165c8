// decode_coded.cu -- attention of one new token per request over a cache of 8 or 4 bits.
//
// A block for each request and query head; its warps take rows in turn, a lane D / 32
// neighbouring values of each, with the running maximum and sum of a softmax in fp32,
// and join in shared memory.
#include "coded.cuh"
#include "kernels.h"
#include "paged.h"

namespace jfa {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int kBits, int N>  // N values of a lane
__device__ __forceinline__ void values(const unsigned char* codes, const uint8_t* scales, int lane, float (&x)[N]) {
  if (kBits == 8) {
    const float by = power_value(*scales);
    uint32_t w = N == 4 ? reinterpret_cast<const uint32_t*>(codes)[lane] : reinterpret_cast<const uint16_t*>(codes)[lane];
    uint32_t h[2];
    halves_of_e4m3x4(w, h[0], h[1]);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 f = floats_of(h[i]);
      x[2 * i] = f.x * by;
      x[2 * i + 1] = f.y * by;
    }
  } else {
    const float by = scale_value(scales[lane * N / kBlock]);
    uint32_t w = N == 4 ? reinterpret_cast<const uint16_t*>(codes)[lane] : codes[lane];
    uint32_t h[4];
    halves_of_e2m1x8(w, h);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 f = floats_of(h[i]);
      x[2 * i] = f.x * by;
      x[2 * i + 1] = f.y * by;
    }
  }
}

template <int kBits, int D>
__global__ void __launch_bounds__(kWarps * 32) decode_coded_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int N = D / 32;
  __shared__ float sh_m[kWarps], sh_l[kWarps], sh_o[kWarps][D];
  wait_for_launch_before();
  const int b = blockIdx.x, h = blockIdx.y, kv = h / a.group, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int len = a.lens[b];
  if (len < 0 || len > a.max_pages * a.div.d) {
    if (threadIdx.x == 0) atomicOr(a.status, kPagerBadLength);
    len = 0;
  }
  float q[N], o[N] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    q[i] = __uint_as_float(static_cast<uint32_t>(a.q[b * a.q_row + int64_t(h) * D + lane * N + i]) << 16);
  for (int t = warp; t < len; t += kWarps) {
    const int i = a.div.quot(t), page = a.table[b * a.table_row + i], in_page = t - i * a.div.d;
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, kPagerBadPage);
      continue;
    }
    const int64_t at = page * a.page + in_page * a.row + kv * a.head;
    const int64_t scales = page * a.scales.page + in_page * a.scales.row + kv * a.scales.head;
    float k[N], v[N], s = 0.f;
    values<kBits>(reinterpret_cast<const unsigned char*>(a.k) + at, a.scales.k + scales, lane, k);
    values<kBits>(reinterpret_cast<const unsigned char*>(a.v) + at, a.scales.v + scales, lane, v);
#pragma unroll
    for (int i = 0; i < N; ++i) s += q[i] * k[i];
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) s += __shfl_xor_sync(~0u, s, x);
    s *= a.scale * kLog2e;
    const float up = fmaxf(m, s), ref = up == -INFINITY ? 0.f : up;
    const float keep = fast_exp2(m - ref), p = fast_exp2(s - ref);
    m = up;
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * keep + p * v[i];
  }
  if (lane == 0) sh_m[warp] = m, sh_l[warp] = l;
#pragma unroll
  for (int i = 0; i < N; ++i) sh_o[warp][lane * N + i] = o[i];
  __syncthreads();
  float top = -INFINITY, sum = 0.f, got = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  const int d = threadIdx.x;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float by = fast_exp2(sh_m[w] - ref);
    sum += by * sh_l[w];
    if (d < D) got += by * sh_o[w][d];
  }
  if (d < D) a.out[(int64_t(b) * a.H + h) * D + d] = static_cast<uint16_t>(pack_bf16x2(sum == 0.f ? 0.f : got / sum, 0.f));
  if (d == 0) a.lse[int64_t(h) * a.B + b] = len == 0 ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

}  // namespace

cudaError_t launch_decode_coded(const DecodeArgs& a, int, cudaStream_t stream) {
  auto* kernel = a.bits == 8 ? (a.D == 128 ? decode_coded_kernel<8, 128> : decode_coded_kernel<8, 64>)
                             : (a.D == 128 ? decode_coded_kernel<4, 128> : decode_coded_kernel<4, 64>);
  return launch_overlapped(kernel, dim3(a.B, a.H), kWarps * 32, 0, stream, a);
}

}  // namespace jfa
