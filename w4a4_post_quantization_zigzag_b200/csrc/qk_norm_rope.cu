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

// The larger of two magnitudes; NaN if one is.
QVLA_DEVICE float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 8-bit code of x / s, as the 8-bit activation quantiser rounds it; 0 if s is not
// above 0 (a row of zeros, or one that has no 8-bit form).
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

// A token's heads go by in passes of 32 / LPR rows: query passes, key passes,
// value passes.  `share` warps take `each` passes of a token, and go on to
// further tokens.
struct RowShare {
  int query, key, all;     // passes before the key's, before the value's, of a token
  int share, each;
  int64_t items;           // T * share
};

// Where a lane's values lie in a row, and what its token says.
template <typename X>
struct Lane {
  int c0, c1;              // its two chunks
  int row;                 // its row of a pass
  bool on, turn;           // it has values, they are rotated
  int pos;
  bool bad;                // position outside the table
  int64_t slot_off, scale_off;   // of the token's slot; slot_off < 0: nothing is written
};

// Mean of the squares of the row that LPR lanes hold.
template <int LPR>
QVLA_DEVICE float mean_square(const Vec8& x0, const Vec8& x1, int D) {
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(x0.v[j], x0.v[j], fmaf(x1.v[j], x1.v[j], ss));
#pragma unroll
  for (int d = LPR / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  return ss / static_cast<float>(D);
}
constexpr uint32_t kLeastMean = 0x0d800000u, kMostMean = 0x71800000u;   // bits of 2^-100 and 2^100
constexpr float kShrink = 8.07793567e-28f;                              // 2^-90

// Passes [lo, hi) of one kind of head (0 query, 1 key, 2 value) of a token.
// With norm weight w and r = 1 / sqrt(mean + eps), pairs become
//   (a, b) -> r (a (w_a c) - b (w_b s)),  r (b (w_b c) + a (w_a s)):
// four coefficients a pair, formed once here.
template <typename X, int LPR, bool INTER, int KIND>
QVLA_DEVICE void some_heads(const NormRopeArgs& a, const Lane<X>& ln, int t, int lo, int hi) {
  if (lo >= hi) return;
  constexpr int kRows = 32 / LPR;
  const int H = KIND == 0 ? a.Hq : a.Hkv;
  int h = lo * kRows + ln.row;
  const X* x = (KIND == 0   ? static_cast<const X*>(a.q) + t * a.ldq
                : KIND == 1 ? static_cast<const X*>(a.k) + t * a.ldk
                            : static_cast<const X*>(a.v) + t * a.ldv) +
               h * a.D;
  X* out = KIND == 0   ? static_cast<X*>(a.q_out) + t * a.ldqo + h * a.D
           : KIND == 1 ? static_cast<X*>(a.k_out) + t * a.ldko + h * a.D
                       : nullptr;
  const bool to_out = KIND == 0 || (KIND == 1 && a.k_out != nullptr);
  const bool to_cache = KIND > 0 && a.has_cache && ln.slot_off >= 0;
  int64_t at = ln.slot_off + h * a.cache.head_stride, scale_at = ln.scale_off + h * a.cache.s_head_stride;
  const float* w = KIND == 0 ? a.q_norm : KIND == 1 ? a.k_norm : nullptr;
  Raw8<X> r0 = {}, r1 = {};
  if (ln.on && h < H) {
    r0 = load_raw(x + ln.c0);
    r1 = load_raw(x + ln.c1);
  }
  Vec8 p0, p1, q0, q1;
  if constexpr (KIND < 2) {
    if (w && ln.on) {
      p0 = load8(w + ln.c0);
      p1 = load8(w + ln.c1);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p0.v[j] = p1.v[j] = 1.f;
    }
    if (ln.turn && !ln.bad) {
      const float* row = a.table + static_cast<int64_t>(ln.pos) * a.rot + (threadIdx.x % LPR) * 8;
      const Vec8 cs = load8(row), sn = load8(row + a.rot / 2);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (INTER) {
          q0.v[j] = p0.v[j ^ 1] * (j & 1 ? sn.v[j / 2] : -sn.v[j / 2]);
          q1.v[j] = p1.v[j ^ 1] * (j & 1 ? sn.v[4 + j / 2] : -sn.v[4 + j / 2]);
        } else {
          q0.v[j] = -p1.v[j] * sn.v[j];
          q1.v[j] = p0.v[j] * sn.v[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p0.v[j] *= cs.v[INTER ? j / 2 : j];
        p1.v[j] *= cs.v[INTER ? 4 + j / 2 : j];
      }
    }
  }
#pragma unroll 1
  for (int i = lo; i < hi; ++i) {
    const bool live = ln.on && h < H;
    Vec8 x0 = widen<X>(r0), x1 = widen<X>(r1);
    h += kRows;
    x += kRows * a.D;
    if (i + 1 < hi && ln.on && h < H) {
      r0 = load_raw(x + ln.c0);
      r1 = load_raw(x + ln.c1);
    } else {
      r0 = r1 = Raw8<X>{};
    }
    if constexpr (KIND < 2) {
      float r = 1.f;
      if (w) {
        float mean = mean_square<LPR>(x0, x1, a.D) + a.eps;
        // Squares that fp32 does not hold (a row of values past 2^50 or, with no
        // eps to speak of, below 2^-50, NaN too): once more at another power of two.
        if (__any_sync(0xffffffffu, __float_as_uint(mean) - kLeastMean > kMostMean - kLeastMean)) {
          const float by = mean > __uint_as_float(kMostMean)    ? kShrink
                           : mean < __uint_as_float(kLeastMean) ? 1.f / kShrink
                                                                : 1.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x0.v[j] *= by;
            x1.v[j] *= by;
          }
          mean = mean_square<LPR>(x0, x1, a.D) + a.eps * by * by;
        }
        r = rsqrtf(mean);
      }
      if (ln.bad) {
        x0 = x1 = Vec8{};
      } else if (ln.turn) {
        const Vec8 y0 = x0, y1 = x1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x0.v[j] = fmaf(y0.v[j], p0.v[j], (INTER ? y0.v[j ^ 1] : y1.v[j]) * q0.v[j]) * r;
          x1.v[j] = fmaf(y1.v[j], p1.v[j], (INTER ? y1.v[j ^ 1] : y0.v[j]) * q1.v[j]) * r;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x0.v[j] = x0.v[j] * p0.v[j] * r;
          x1.v[j] = x1.v[j] * p1.v[j] * r;
        }
      }
      if (to_out) {
        if (live) {
          store8(out + ln.c0, x0);
          store8(out + ln.c1, x1);
        }
        out += kRows * a.D;
      }
    }
    if constexpr (KIND > 0) {
      if (!to_cache) continue;               // the same for the whole warp
      if (a.cache.bits == 8) {
        float mx = 0.f;
        if (live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) mx = max_or_nan(mx, max_or_nan(fabsf(x0.v[j]), fabsf(x1.v[j])));
        }
#pragma unroll
        for (int d = LPR / 2; d; d >>= 1) mx = max_or_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        if (live) {
          // an infinity or a NaN in the row: its scale says so, for no code can
          const float s = mx < INFINITY ? __fdiv_rn(mx, 127.f) : __uint_as_float(0x7fc00000u);
          int8_t* row = static_cast<int8_t*>(KIND == 1 ? a.cache.k : a.cache.v) + at;
          store_codes(row + ln.c0, x0, s);
          store_codes(row + ln.c1, x1, s);
          if (threadIdx.x % LPR == 0) (KIND == 1 ? a.cache.k_scale : a.cache.v_scale)[scale_at] = s;
        }
        scale_at += kRows * a.cache.s_head_stride;
      } else if (live) {
        __nv_bfloat16* row = static_cast<__nv_bfloat16*>(KIND == 1 ? a.cache.k : a.cache.v) + at;
        store8(row + ln.c0, x0);
        store8(row + ln.c1, x1);
      }
      at += kRows * a.cache.head_stride;
    }
  }
}

// CTAs of 256 threads per SM: with three, at 80 registers, the coefficients spill
// (16381 x 48 heads of 128: 94 against 85 us); rows two or more passes ahead
// change nothing there (85 to 88 us).  With two, bf16 rows spill 4 bytes at most,
// fp32 rows, twice as wide, 24 to 52.
constexpr int kResident = 2;

// Bound by the rows on the way from memory, of which registers hold too few to
// fill it (16 KB an SM; DRAM is half busy).  A head's row of D values
// belongs to LPR = 4, 8 or 16 lanes of a warp; a lane holds two chunks of eight
// values that hold whole rotation pairs (for separate halves: chunk j and chunk
// j + rot/16 of the row), so norm, rotation and stores need no exchange but the
// sum of squares (and the maximum, for 8-bit codes).  A lane writes only what it
// read, so q_out and k_out may be the inputs.  The next pass's rows are loaded
// before this pass's are worked on.  16381 tokens of 32 + 8 + 8 heads of 128:
// 85 us for 411 MB read and written, 4.8 TB/s (73 % of the copy rate of large
// buffers; a plain device copy of 206 MB ran at 3.0); into an 8-bit cache 114 us,
// the maximum, divisions and codes of every key and value.  8000 such tokens in
// fp32: 72 us for 365 MB, 86 into an 8-bit cache.  1024 tokens of 8 + 1 + 1 heads
// of 256: 5.0 us (8 bits: 7.8), one token 2.5: the launch and one trip to memory.
template <typename X, int LPR, bool INTER>
__global__ void __launch_bounds__(256, kResident)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ RowShare sh,
                     unsigned int* err) {
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  Lane<X> ln;
  ln.on = sub < a.D / 16;
  ln.turn = sub < a.rot / 16;
  ln.row = lane / LPR;
  ln.c0 = 16 * sub;
  ln.c1 = 16 * sub + 8;
  if (ln.turn && !INTER) {
    ln.c0 = 8 * sub;
    ln.c1 = 8 * sub + a.rot / 2;
  }
  pdl_launch_dependents();
  pdl_wait();
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); item < sh.items; item += step) {
    const int t = sh.share == 1 ? static_cast<int>(item) : static_cast<int>(item / sh.share);
    const int lo = static_cast<int>(item - static_cast<int64_t>(t) * sh.share) * sh.each;
    const int hi = min(lo + sh.each, sh.all);
    ln.pos = a.table ? a.positions[t] : 0;
    const int s = a.has_cache ? a.slots[t] : -1;
    ln.bad = a.table && (ln.pos < 0 || ln.pos >= a.P);
    ln.slot_off = -1;
    ln.scale_off = 0;
    bool outside = ln.bad;
    if (s >= 0) {
      const int page = s / a.cache.page_size, tok = s - page * a.cache.page_size;
      outside |= page >= a.cache.pages;
      if (!outside) {
        ln.slot_off = page * a.cache.page_stride + tok * a.cache.token_stride;
        ln.scale_off = page * a.cache.s_page_stride + tok * a.cache.s_token_stride;
      }
    }
    if (outside && lo == 0 && lane == 0) report(err, QVLA_DEVERR_CACHE_RANGE);
    some_heads<X, LPR, INTER, 0>(a, ln, t, lo, min(hi, sh.query));
    some_heads<X, LPR, INTER, 1>(a, ln, t, max(lo - sh.query, 0), min(hi, sh.key) - sh.query);
    some_heads<X, LPR, INTER, 2>(a, ln, t, max(lo - sh.key, 0), hi - sh.key);
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
  const int64_t resident = sms * kResident;
  constexpr int kRows = 32 / LPR;
  RowShare sh;
  sh.query = (a.Hq + kRows - 1) / kRows;
  sh.key = sh.query + (a.Hkv + kRows - 1) / kRows;
  sh.all = sh.key + (a.has_cache ? (a.Hkv + kRows - 1) / kRows : 0);
  // with fewer tokens than warps, several warps share a token
  const int want = static_cast<int>(std::min<int64_t>(sh.all, std::max<int64_t>(1, 8 * resident / a.T)));
  sh.each = (sh.all + want - 1) / want;
  sh.share = (sh.all + sh.each - 1) / sh.each;
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
  if (a.interleaved) return cudaLaunchKernelEx(&cfg, norm_rope_kernel<X, LPR, true>, a, sh, err);
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<X, LPR, false>, a, sh, err);
}

}  // namespace

cudaError_t launch_rope_table(const RopeFreqs& freqs, int half, int P, float* table,
                              cudaStream_t s) {
  const int64_t total = static_cast<int64_t>(P) * half;
  // a launch that returns its own status, not an error that an earlier call left
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((total + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, freqs, half, total, table);
}

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  const bool f32 = a.xdt == QVLA_DTYPE_F32;
  if (a.D <= 64) return f32 ? launch_typed<float, 4>(a, stream) : launch_typed<__nv_bfloat16, 4>(a, stream);
  if (a.D <= 128) return f32 ? launch_typed<float, 8>(a, stream) : launch_typed<__nv_bfloat16, 8>(a, stream);
  return f32 ? launch_typed<float, 16>(a, stream) : launch_typed<__nv_bfloat16, 16>(a, stream);
}

}  // namespace qvla
