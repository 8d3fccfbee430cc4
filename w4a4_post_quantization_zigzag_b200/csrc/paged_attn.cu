// Attention of one new token per sequence over a paged key/value cache.
//
//   o = sum_t p_t v_t,  p = softmax over the visible t of scale * q . k_t
#include "qvla_common.cuh"
#include "qvla_internal.h"

namespace qvla {
namespace {

constexpr int kWarps = 8;

// Sequence length as the kernel uses it: 0 (and the error bit) if it is
// outside its page table.
QVLA_DEVICE int checked_len(const PagedAttnArgs& a, int b, unsigned int* err) {
  const int n = a.seq_lens[b];
  if (n >= 0 && n <= static_cast<int64_t>(a.max_pages) * a.cache.page_size) return n;
  report(err, QVLA_DEVERR_CACHE_RANGE);
  return 0;
}

// One CTA per sequence and query head; a warp takes every eighth token, its
// lanes split the head's values.
__global__ void __launch_bounds__(32 * kWarps) attn_kernel(const __grid_constant__ PagedAttnArgs a,
                                                           unsigned int* err) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
  const int b = blockIdx.y, h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.cache.dim, hk = h / (a.Hq / a.cache.heads);
  const int n = checked_len(a, b, err);
  const int64_t hidden_end = a.window ? static_cast<int64_t>(n) - a.window : 0;  // first visible of the window
  float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < 8; ++i) {
    const int d = lane + 32 * i;
    const int64_t at = b * a.ldq + static_cast<int64_t>(h) * D + d;
    q[i] = d < D ? (a.qdt == QVLA_DTYPE_F32 ? static_cast<const float*>(a.q)[at]
                                            : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]))
                 : 0.f;
  }
  for (int t = warp; t < n; t += kWarps) {
    if (t >= a.sinks && t < hidden_end) continue;
    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + t / a.cache.page_size];
    if (page < 0 || page >= a.cache.pages) {
      if (lane == 0) report(err, QVLA_DEVERR_CACHE_RANGE);
      continue;
    }
    const int tok = t % a.cache.page_size;
    const int64_t at = page * a.cache.page_stride + tok * a.cache.token_stride + hk * a.cache.head_stride;
    float ks = 1.f, vs = 1.f;
    if (a.cache.bits == 8) {
      const int64_t sat = page * a.cache.s_page_stride + tok * a.cache.s_token_stride + hk * a.cache.s_head_stride;
      ks = a.cache.k_scale[sat];
      vs = a.cache.v_scale[sat];
    }
    auto value = [&](const void* base, int d) -> float {
      if (d >= D) return 0.f;
      return a.cache.bits == 8 ? static_cast<float>(static_cast<const int8_t*>(base)[at + d])
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at + d]);
    };
    float s = 0.f;
    for (int i = 0; i < 8; ++i) s += q[i] * value(a.cache.k, lane + 32 * i);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= ks * a.scale;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float keep = expf(m - base), p = expf(s - base);
    m = mn;
    l = l * keep + p;
    for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + p * vs * value(a.cache.v, lane + 32 * i);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int i = 0; i < 8; ++i) so[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float mx = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w]);
  const float base = mx == -INFINITY ? 0.f : mx;
  for (int w = 0; w < kWarps; ++w) total += sl[w] * expf(sm[w] - base);
  const int d = threadIdx.x;
  if (d < D) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += so[w][d] * expf(sm[w] - base);
    v = total == 0.f ? 0.f : v / total;
    const int64_t at = b * a.ldo + static_cast<int64_t>(h) * D + d;
    if (a.qdt == QVLA_DTYPE_F32)
      static_cast<float*>(a.out)[at] = v;
    else
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  }
  if (a.lse && d == 0)
    a.lse[static_cast<int64_t>(b) * a.Hq + h] = total == 0.f ? -INFINITY : base + logf(total);
}

}  // namespace

size_t paged_attn_ws_bytes(int Hq, int heads, int dim) { return 16; }

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  attn_kernel<<<dim3(a.Hq, a.B), 32 * kWarps, 0, stream>>>(a, err);
  return cudaGetLastError();
}

}  // namespace qvla
