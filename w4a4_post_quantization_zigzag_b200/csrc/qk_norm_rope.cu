// RMS norm of query and key heads with the position rotation, keys and values
// written to the paged cache, in one pass over the rows of the q, k, v linears.
//
//   h' = h * w / sqrt(mean(h^2) + eps);  (a, b) -> (a c - b s, b c + a s)
#include "qvla_common.cuh"
#include "qvla_internal.h"

namespace qvla {
namespace {

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeFreqs freqs,
                                                         int half, int64_t total,
                                                         float* __restrict__ table) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t p = i / half;
  const int j = static_cast<int>(i - p * half);
  double s, c;
  sincos(static_cast<double>(p) * freqs.f[j], &s, &c);
  table[p * 2 * half + j] = static_cast<float>(c);
  table[p * 2 * half + half + j] = static_cast<float>(s);
}

struct Vec8 {
  float v[8];
};

template <typename X>
QVLA_DEVICE Vec8 load8(const X* p) {
  Vec8 r;
  if constexpr (sizeof(X) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = __uint_as_float(u[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    r = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  return r;
}

QVLA_DEVICE uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename X>
QVLA_DEVICE void store8(X* p, const Vec8& r) {
  if constexpr (sizeof(X) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(r.v[0], r.v[1]), pack_bf16(r.v[2], r.v[3]), pack_bf16(r.v[4], r.v[5]),
                   pack_bf16(r.v[6], r.v[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
  }
}

// 8-bit code of x / s, as the 8-bit activation quantiser rounds it.
QVLA_DEVICE uint32_t code8(float x, float s) {
  if (!(s > 0.f)) return 0u;
  return static_cast<uint32_t>(
             static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x, s)), -128.f), 127.f))) & 255u;
}

QVLA_DEVICE void store_codes(int8_t* p, const Vec8& r, float s) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = code8(r.v[4 * i], s) | code8(r.v[4 * i + 1], s) << 8 | code8(r.v[4 * i + 2], s) << 16 |
           code8(r.v[4 * i + 3], s) << 24;
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// One CTA per token.  A head's row of D values belongs to LPR = 4, 8 or 16
// lanes of a warp; a lane holds two chunks of eight values that hold whole
// rotation pairs (for separate halves: chunk j and chunk j + rot/16 of the
// row), so norm, rotation and stores need no exchange but the sum of squares
// (and the maximum, for 8-bit codes).  A lane writes only what it read, so
// q_out and k_out may be the inputs.
template <typename X, int LPR>
__global__ void __launch_bounds__(256) norm_rope_kernel(const __grid_constant__ NormRopeArgs a,
                                                        unsigned int* err) {
  const int t = blockIdx.x;
  const int sub = threadIdx.x % LPR, items = a.D / 16;
  const bool on = sub < items;
  const int pairs = a.rot / 16;            // lanes whose chunks are rotated
  const bool turn = sub < pairs;
  // the two chunks of this lane (in units of eight values)
  int c0 = 2 * sub, c1 = 2 * sub + 1;
  if (turn && !a.interleaved) {
    c0 = sub;
    c1 = sub + pairs;
  }
  bool bad = false;
  Vec8 cs, sn;
  if (a.table) {
    const int p = a.positions[t];
    bad = p < 0 || p >= a.P;
    if (!bad && on && turn) {
      const float* row = a.table + static_cast<int64_t>(p) * a.rot + sub * 8;
      cs = load8(row);
      sn = load8(row + a.rot / 2);
    }
  }
  int64_t slot_off = -1, scale_off = 0;
  if (a.has_cache) {
    const int s = a.slots[t];
    const int page = s / a.cache.page_size, tok = s - page * a.cache.page_size;
    if (s >= 0 && page >= a.cache.pages) {
      if (threadIdx.x == 0) report(err, QVLA_DEVERR_CACHE_RANGE);
    } else if (s >= 0 && !bad) {
      slot_off = page * a.cache.page_stride + tok * a.cache.token_stride;
      scale_off = page * a.cache.s_page_stride + tok * a.cache.s_token_stride;
    }
  }
  if (bad && threadIdx.x == 0) report(err, QVLA_DEVERR_CACHE_RANGE);

  const int heads = a.Hq + a.Hkv + (a.has_cache ? a.Hkv : 0);
  for (int h0 = 0; h0 < heads; h0 += blockDim.x / LPR) {   // whole warps stay together
    const int h = h0 + static_cast<int>(threadIdx.x) / LPR;
    const bool live = on && h < heads;
    const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;    // query, key, value
    const int hh = kind == 0 ? h : kind == 1 ? h - a.Hq : h - a.Hq - a.Hkv;
    Vec8 x0 = {}, x1 = {};
    if (live) {
      const void* base = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
      const int64_t ld = kind == 0 ? a.ldq : kind == 1 ? a.ldk : a.ldv;
      const X* row = static_cast<const X*>(base) + t * ld + static_cast<int64_t>(hh) * a.D;
      x0 = load8(row + c0 * 8);
      x1 = load8(row + c1 * 8);
    }
    const float* w = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x0.v[i] * x0.v[i] + x1.v[i] * x1.v[i];
#pragma unroll
    for (int d = LPR / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if (live && w) {
      const float r = 1.f / sqrtf(ss / static_cast<float>(a.D) + a.eps);
      const Vec8 w0 = load8(w + c0 * 8), w1 = load8(w + c1 * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x0.v[i] = x0.v[i] * r * w0.v[i];
        x1.v[i] = x1.v[i] * r * w1.v[i];
      }
    }
    if (live && turn && kind < 2 && !bad) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p0 = x0.v[2 * i], q0 = x0.v[2 * i + 1], p1 = x1.v[2 * i], q1 = x1.v[2 * i + 1];
          x0.v[2 * i] = p0 * cs.v[i] - q0 * sn.v[i];
          x0.v[2 * i + 1] = q0 * cs.v[i] + p0 * sn.v[i];
          x1.v[2 * i] = p1 * cs.v[4 + i] - q1 * sn.v[4 + i];
          x1.v[2 * i + 1] = q1 * cs.v[4 + i] + p1 * sn.v[4 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = x0.v[i], q = x1.v[i];
          x0.v[i] = p * cs.v[i] - q * sn.v[i];
          x1.v[i] = q * cs.v[i] + p * sn.v[i];
        }
      }
    }
    if (bad) x0 = x1 = Vec8{};
    if (live && kind < 2) {
      void* base = kind == 0 ? a.q_out : a.k_out;
      if (base) {
        X* row = static_cast<X*>(base) + t * (kind == 0 ? a.ldqo : a.ldko) + static_cast<int64_t>(hh) * a.D;
        store8(row + c0 * 8, x0);
        store8(row + c1 * 8, x1);
      }
    }
    if (kind == 0 || slot_off < 0) {
      if (a.cache.bits != 8) continue;
    }
    const int64_t at = slot_off + hh * a.cache.head_stride;
    if (a.cache.bits == 8) {
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fmaxf(fabsf(x0.v[i]), fabsf(x1.v[i])));
#pragma unroll
      for (int d = LPR / 2; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      if (live && kind > 0 && slot_off >= 0) {
        const float s = __fdiv_rn(mx, 127.f);
        int8_t* row = static_cast<int8_t*>(kind == 1 ? a.cache.k : a.cache.v) + at;
        store_codes(row + c0 * 8, x0, s);
        store_codes(row + c1 * 8, x1, s);
        if (sub == 0)
          (kind == 1 ? a.cache.k_scale : a.cache.v_scale)[scale_off + hh * a.cache.s_head_stride] = s;
      }
    } else if (live) {
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(kind == 1 ? a.cache.k : a.cache.v) + at;
      store8(row + c0 * 8, x0);
      store8(row + c1 * 8, x1);
    }
  }
}

template <typename X, int LPR>
cudaError_t launch_typed(const NormRopeArgs& a, cudaStream_t stream) {
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  const int64_t heads = static_cast<int64_t>(a.Hq) + a.Hkv + (a.has_cache ? a.Hkv : 0);
  const int64_t lanes = (heads * LPR + 31) / 32 * 32;
  norm_rope_kernel<X, LPR><<<a.T, static_cast<int>(lanes < 256 ? lanes : 256), 0, stream>>>(a, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const RopeFreqs& freqs, int half, int P, float* table,
                              cudaStream_t s) {
  const int64_t total = static_cast<int64_t>(P) * half;
  rope_table_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, s>>>(freqs, half, total, table);
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  const bool f32 = a.xdt == QVLA_DTYPE_F32;
  if (a.D <= 64) return f32 ? launch_typed<float, 4>(a, stream) : launch_typed<__nv_bfloat16, 4>(a, stream);
  if (a.D <= 128) return f32 ? launch_typed<float, 8>(a, stream) : launch_typed<__nv_bfloat16, 8>(a, stream);
  return f32 ? launch_typed<float, 16>(a, stream) : launch_typed<__nv_bfloat16, 16>(a, stream);
}

}  // namespace qvla
