// W4A16: products of few activation rows with 4-bit weights that carry one
// scale (and optionally one zero point) per group of inputs.
//
//   y[m,n] = sum_g s[n,g] * ( sum_{k in g} (u[n,k] - z[n,g]) x[m,k] ) + b[n]
#include "qvla_common.cuh"
#include "qvla_internal.h"

namespace qvla {
namespace {

// ------------------------------------------------------------------- pack
// One warp per group of one row: min and max, scale rounded to its stored
// type, codes by IEEE division with the rounded scale (so that the codes are
// the nearest to what the product will use).
template <typename S>
__global__ void __launch_bounds__(256) pack_w4g_kernel(const float* __restrict__ W, int64_t groups,
                                                       int group, uint8_t* __restrict__ wq,
                                                       S* __restrict__ scale,
                                                       uint8_t* __restrict__ zero) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (i >= groups) return;
  const float* w = W + i * group;
  float lo = 0.f, hi = 0.f;
  for (int k = lane; k < group; k += 32) {
    lo = fminf(lo, w[k]);
    hi = fmaxf(hi, w[k]);
  }
  for (int d = 16; d; d >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
  }
  const float s0 = zero ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
  S stored;
  float s;
  if constexpr (sizeof(S) == 2) {
    stored = __float2bfloat16_rn(s0);
    s = __bfloat162float(stored);
  } else {
    stored = s = s0;
  }
  int z = 0;
  if (zero && s > 0.f) z = static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f));
  auto code = [&](float v) -> unsigned {
    if (!(s > 0.f)) return 0u;
    const float r = rintf(__fdiv_rn(v, s));
    if (zero) return static_cast<unsigned>(fminf(fmaxf(r + z, 0.f), 15.f));
    return static_cast<unsigned>(static_cast<int>(fminf(fmaxf(r, -7.f), 7.f))) & 15u;
  };
  uint8_t* out = wq + i * group / 2;
  for (int j = lane; j < group / 2; j += 32)
    out[j] = static_cast<uint8_t>(code(w[2 * j]) | code(w[2 * j + 1]) << 4);
  if (lane == 0) {
    scale[i] = stored;
    if (zero) zero[i] = static_cast<uint8_t>(z);
  }
}

// ---------------------------------------------------------------- product
__device__ __forceinline__ float load_f32(const void* p, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// One warp per weight row, eight activation rows at a time: a lane takes eight
// codes (one word) of every 256, which lie in one group.
__global__ void __launch_bounds__(256) gemv_kernel(GemvArgs a) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int groups = a.K / a.group;
  for (int m0 = 0; m0 < a.M; m0 += 8) {
    const int mc = min(8, a.M - m0);
    float acc[8] = {};
    for (int k = lane * 8; k < a.K; k += 256) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(
          a.wq + static_cast<int64_t>(n) * (a.K / 2) + k / 2);
      const int64_t gi = static_cast<int64_t>(n) * groups + k / a.group;
      const float s = load_f32(a.scale, gi, a.sdt == QVLA_DTYPE_F32);
      const int z = a.zero ? a.zero[gi] & 15 : 8;
      const uint32_t u = a.zero ? w : w ^ 0x88888888u;
      for (int m = 0; m < mc; ++m) {
        float part = 0.f;
        for (int j = 0; j < 8; ++j)
          part += static_cast<float>(static_cast<int>(u >> (4 * j) & 15u) - z) *
                  load_f32(a.x, static_cast<int64_t>(m0 + m) * a.ldx + k + j,
                           a.xdt == QVLA_DTYPE_F32);
        acc[m] += s * part;
      }
    }
    for (int m = 0; m < mc; ++m) {
      float v = acc[m];
      for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      if (lane == 0) {
        if (a.bias) v += a.bias[n];
        const int64_t o = static_cast<int64_t>(m0 + m) * a.ldy + n;
        if (a.ydt == QVLA_DTYPE_F32)
          static_cast<float*>(a.y)[o] = v;
        else
          static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
      }
    }
  }
}

}  // namespace

cudaError_t launch_pack_w4g(const float* W, int N, int K, int group, qvla_dtype sdt, uint8_t* wq,
                            void* scale, uint8_t* zero, cudaStream_t s) {
  const int64_t groups = static_cast<int64_t>(N) * (K / group);
  const unsigned grid = static_cast<unsigned>((groups + 7) / 8);
  if (sdt == QVLA_DTYPE_F32)
    pack_w4g_kernel<<<grid, 256, 0, s>>>(W, groups, group, wq, static_cast<float*>(scale), zero);
  else
    pack_w4g_kernel<<<grid, 256, 0, s>>>(W, groups, group, wq, static_cast<__nv_bfloat16*>(scale),
                                         zero);
  return cudaGetLastError();
}

cudaError_t launch_w4a16_gemv(const GemvArgs& a, cudaStream_t stream) {
  gemv_kernel<<<(a.N + 7) / 8, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace qvla
