// RMS norm of query and key heads with the position rotation, keys and values
// written to the paged cache, in one pass over the rows of the q, k, v linears.
//
//   h' = h * w / sqrt(mean(h^2) + eps);  (a, b) -> (a c - b s, b c + a s)
#include "qvla_common.cuh"
#include "qvla_internal.h"

#include <algorithm>

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

QVLA_DEVICE Vec8 load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
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

// Raw chunk of eight values as it is loaded (a pass ahead of its use).
template <typename X>
struct Raw8 {
  uint4 v[sizeof(X) == 2 ? 1 : 2];
};
template <typename X>
QVLA_DEVICE Raw8<X> load_raw(const X* p) {
  Raw8<X> r;
  r.v[0] = reinterpret_cast<const uint4*>(p)[0];
  if constexpr (sizeof(X) == 4) r.v[1] = reinterpret_cast<const uint4*>(p)[1];
  return r;
}
template <typename X>
QVLA_DEVICE Vec8 widen(const Raw8<X>& w) {
  Vec8 r;
  const uint32_t u[4] = {w.v[0].x, w.v[0].y, w.v[0].z, w.v[0].w};
  if constexpr (sizeof(X) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = __uint_as_float(u[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const uint4 h = w.v[sizeof(X) == 2 ? 0 : 1];
    const uint32_t q[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[i] = __uint_as_float(u[i]);
      r.v[4 + i] = __uint_as_float(q[i]);
    }
  }
  return r;
}

// A token's rows (query, key, value heads) are dealt to `share` warps, which
// go on to further tokens.
struct RowShare {
  int share;           // warps of a token
  int passes;          // passes of 32 / LPR rows that one of them takes
  int64_t items;       // T * share
};

// Bound by reading the rows and writing them back.  A head's row of D values
// belongs to LPR = 4, 8 or 16 lanes of a warp; a lane holds two chunks of eight
// values that hold whole rotation pairs (for separate halves: chunk j and chunk
// j + rot/16 of the row), so norm, rotation and stores need no exchange but the
// sum of squares (and the maximum, for 8-bit codes).  A lane writes only what it
// read, so q_out and k_out may be the inputs.  The next pass's rows are loaded
// before this pass's are worked on: with 24 warps on an SM that keeps 48 KB on
// the way.
template <typename X, int LPR>
__global__ void __launch_bounds__(256, sizeof(X) == 2 ? 3 : 2)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ RowShare sh,
                     unsigned int* err) {
  constexpr int kRows = 32 / LPR;          // rows of a pass
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPR;
  const bool on = sub < a.D / 16;
  const int pairs = a.rot / 16;            // lanes whose chunks are rotated
  const bool turn = sub < pairs;
  // the two chunks of this lane (in units of eight values)
  int c0 = 2 * sub, c1 = 2 * sub + 1;
  if (turn && !a.interleaved) {
    c0 = sub;
    c1 = sub + pairs;
  }
  const int heads = a.Hq + a.Hkv + (a.has_cache ? a.Hkv : 0);
  const float inv_dim = 1.f / static_cast<float>(a.D);
  pdl_launch_dependents();
  pdl_wait();

  // row h of token t: query, key or value head; its place in the inputs
  struct Place {
    int kind, head;          // 0 query, 1 key, 2 value, 3 none
    const X* x;
  };
  auto place = [&](int t, int h) -> Place {
    Place p;
    p.kind = !on || h >= heads ? 3 : h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
    p.head = h - (p.kind == 0 ? 0 : p.kind == 1 ? a.Hq : a.Hq + a.Hkv);
    const void* base = p.kind == 0 ? a.q : p.kind == 1 ? a.k : a.v;
    const int64_t ld = p.kind == 0 ? a.ldq : p.kind == 1 ? a.ldk : a.ldv;
    p.x = static_cast<const X*>(base) + t * ld + static_cast<int64_t>(p.head) * a.D;
    return p;
  };

  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); item < sh.items; item += step) {
    const int t = static_cast<int>(item / sh.share), part = static_cast<int>(item - static_cast<int64_t>(t) * sh.share);
    const int h0 = part * sh.passes * kRows + lane / LPR;
    const int pos = a.table ? a.positions[t] : 0;
    const int s = a.has_cache ? a.slots[t] : -1;
    Place now = place(t, h0);
    Raw8<X> r0 = {}, r1 = {};
    if (now.kind < 3) {
      r0 = load_raw(now.x + c0 * 8);
      r1 = load_raw(now.x + c1 * 8);
    }
    const bool bad = a.table && (pos < 0 || pos >= a.P);
    Vec8 cs = {}, sn = {};
    if (a.table && !bad && on && turn) {
      const float* row = a.table + static_cast<int64_t>(pos) * a.rot + sub * 8;
      cs = load8(row);
      sn = load8(row + a.rot / 2);
    }
    int64_t slot_off = -1, scale_off = 0;
    if (s >= 0) {
      const int page = s / a.cache.page_size, tok = s - page * a.cache.page_size;
      if (page < a.cache.pages && !bad) {
        slot_off = page * a.cache.page_stride + tok * a.cache.token_stride;
        scale_off = page * a.cache.s_page_stride + tok * a.cache.s_token_stride;
      }
      if (page >= a.cache.pages && part == 0 && lane == 0) report(err, QVLA_DEVERR_CACHE_RANGE);
    }
    if (bad && part == 0 && lane == 0) report(err, QVLA_DEVERR_CACHE_RANGE);

#pragma unroll 1
    for (int i = 0; i < sh.passes; ++i) {
      Vec8 x0 = widen<X>(r0), x1 = widen<X>(r1);
      const Place at = now;
      if (i + 1 < sh.passes) {
        now = place(t, h0 + (i + 1) * kRows);
        if (now.kind < 3) {
          r0 = load_raw(now.x + c0 * 8);
          r1 = load_raw(now.x + c1 * 8);
        } else {
          r0 = r1 = Raw8<X>{};
        }
      }
      const float* w = at.kind == 0 ? a.q_norm : at.kind == 1 ? a.k_norm : nullptr;
      if (a.q_norm || a.k_norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x0.v[j], x0.v[j], fmaf(x1.v[j], x1.v[j], ss));
#pragma unroll
        for (int d = LPR / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if (at.kind < 2 && w) {
          const float r = 1.f / sqrtf(fmaf(ss, inv_dim, a.eps));
          const Vec8 w0 = load8(w + c0 * 8), w1 = load8(w + c1 * 8);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x0.v[j] = x0.v[j] * r * w0.v[j];
            x1.v[j] = x1.v[j] * r * w1.v[j];
          }
        }
      }
      if (at.kind < 2 && turn && !bad) {
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p0 = x0.v[2 * j], q0 = x0.v[2 * j + 1], p1 = x1.v[2 * j], q1 = x1.v[2 * j + 1];
            x0.v[2 * j] = p0 * cs.v[j] - q0 * sn.v[j];
            x0.v[2 * j + 1] = q0 * cs.v[j] + p0 * sn.v[j];
            x1.v[2 * j] = p1 * cs.v[4 + j] - q1 * sn.v[4 + j];
            x1.v[2 * j + 1] = q1 * cs.v[4 + j] + p1 * sn.v[4 + j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float p = x0.v[j], q = x1.v[j];
            x0.v[j] = p * cs.v[j] - q * sn.v[j];
            x1.v[j] = q * cs.v[j] + p * sn.v[j];
          }
        }
      }
      if (bad) x0 = x1 = Vec8{};
      if (at.kind < 2) {
        void* base = at.kind == 0 ? a.q_out : a.k_out;
        if (base) {
          X* row = static_cast<X*>(base) + t * (at.kind == 0 ? a.ldqo : a.ldko) + static_cast<int64_t>(at.head) * a.D;
          store8(row + c0 * 8, x0);
          store8(row + c1 * 8, x1);
        }
      }
      if (!a.has_cache) continue;
      const bool store = (at.kind == 1 || at.kind == 2) && slot_off >= 0;
      const int64_t to = slot_off + at.head * a.cache.head_stride;
      if (a.cache.bits == 8) {
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(fabsf(x0.v[j]), fabsf(x1.v[j])));
#pragma unroll
        for (int d = LPR / 2; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        if (store) {
          const float q = __fdiv_rn(mx, 127.f);
          int8_t* row = static_cast<int8_t*>(at.kind == 1 ? a.cache.k : a.cache.v) + to;
          store_codes(row + c0 * 8, x0, q);
          store_codes(row + c1 * 8, x1, q);
          if (sub == 0)
            (at.kind == 1 ? a.cache.k_scale : a.cache.v_scale)[scale_off + at.head * a.cache.s_head_stride] = q;
        }
      } else if (store) {
        __nv_bfloat16* row = static_cast<__nv_bfloat16*>(at.kind == 1 ? a.cache.k : a.cache.v) + to;
        store8(row + c0 * 8, x0);
        store8(row + c1 * 8, x1);
      }
    }
  }
}

template <typename X, int LPR>
cudaError_t launch_typed(const NormRopeArgs& a, cudaStream_t stream) {
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int resident = sms * (sizeof(X) == 2 ? 3 : 2);             // CTAs at once
  const int heads = a.Hq + a.Hkv + (a.has_cache ? a.Hkv : 0);
  const int passes = (heads + 32 / LPR - 1) / (32 / LPR);
  // with fewer tokens than warps, several warps share a token
  RowShare sh;
  const int want = static_cast<int>(std::min<int64_t>(passes, std::max<int64_t>(1, 8ll * resident / a.T)));
  sh.passes = (passes + want - 1) / want;
  sh.share = (passes + sh.passes - 1) / sh.passes;
  sh.items = static_cast<int64_t>(a.T) * sh.share;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((sh.items + 7) / 8, resident)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<X, LPR>, a, sh, err);
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
