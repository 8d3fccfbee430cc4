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
// Bound by reading the codes once.  A warp multiplies 32 weight rows with 8 MT
// activation rows on the warp-level tensor cores: the codes become exact bf16
// values (u - z) in registers, x enters as bf16 (fp32 x as three bf16 parts
// whose sum is x), every product is exact, a group's sum is fp32 and is scaled
// once.  The order of K inside an MMA is free as long as both operands agree,
// so a lane takes the codes as they lie in memory, eight per 32-bit word, and
// the activations as 16-byte loads.
//
// A CTA has WR x WK warps: WR bands of 32 rows, K dealt to WK warps in chunks
// of 256 (one 128-byte line of codes per row), and with few rows also to the
// KC CTAs of a cluster; partial sums meet in shared memory (and the cluster's)
// in a fixed order.  CTAs stay and walk over the bands, and each warp's ring
// of code chunks (cp.async, three stages) runs on across them.
constexpr int kChunk = 256;           // K of a ring stage
constexpr int kStages = 3;
constexpr int kStageBytes = 32 * kChunk / 2;
constexpr int kMaxWarps = 8;

struct GemvShape {
  int WR, WK, KC;
};

QVLA_DEVICE void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
QVLA_DEVICE void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
QVLA_DEVICE uint32_t sub2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes j and j + 4 of a word, as bf16 values less z: 128 + u is the bf16 with
// u in its low mantissa bits (`flip` holds 0x4300 and, for two's complement,
// the bit that turns a code into code + 8); `zero` is 128 + z twice.
QVLA_DEVICE void expand(uint32_t w, uint32_t flip, uint32_t zero, uint32_t (&e)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) e[j] = sub2((w >> (4 * j) & 0x000f000fu) ^ flip, zero);
}
// The bf16 values below two fp32 values (cut, not rounded: no value overflows)
// side by side, and what they leave.
QVLA_DEVICE uint32_t take2(float& lo, float& hi) {
  const uint32_t a = __float_as_uint(lo) & 0xffff0000u, b = __float_as_uint(hi) & 0xffff0000u;
  lo -= __uint_as_float(a);
  hi -= __uint_as_float(b);
  return a >> 16 | b;
}
QVLA_DEVICE float scale_at(const GemvArgs& a, int64_t i) {
  return a.sdt == QVLA_DTYPE_F32 ? static_cast<const float*>(a.scale)[i]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(a.scale)[i]);
}

// Scales and zero points of one row's chunk.
template <int NG>
struct RowGroups {
  float s[NG];
  uint32_t z[NG];        // 128 + z as two bf16
};

template <int NG>
QVLA_DEVICE void load_groups(const GemvArgs& a, int n, int c, RowGroups<NG>& r) {
  const int groups = a.K / a.group;
  const int64_t at = static_cast<int64_t>(n) * groups + c * NG;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    r.s[j] = 0.f;
    r.z[j] = a.zero ? 0x43004300u : 0x43084308u;
  }
  if (n >= a.N) return;
  if (groups % NG == 0) {
    // every row's chunk is whole and starts at a multiple of its size
    if (a.sdt == QVLA_DTYPE_F32) {
      const float* p = static_cast<const float*>(a.scale) + at;
      if constexpr (NG >= 4) {
#pragma unroll
        for (int j = 0; j < NG; j += 4) {
          const float4 v = *reinterpret_cast<const float4*>(p + j);
          r.s[j] = v.x, r.s[j + 1] = v.y, r.s[j + 2] = v.z, r.s[j + 3] = v.w;
        }
      } else if constexpr (NG == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        r.s[0] = v.x, r.s[1] = v.y;
      } else {
        r.s[0] = *p;
      }
    } else {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.scale) + at;
      if constexpr (NG >= 2) {
        uint32_t w[NG / 2];
        if constexpr (NG == 8)
          *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (NG == 4)
          *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        else
          w[0] = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
        for (int j = 0; j < NG / 2; ++j) {
          r.s[2 * j] = __uint_as_float(w[j] << 16);
          r.s[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      } else {
        r.s[0] = __bfloat162float(*p);
      }
    }
    if (a.zero) {
      const uint8_t* p = a.zero + at;
      uint64_t w;
      if constexpr (NG == 8)
        w = *reinterpret_cast<const uint64_t*>(p);
      else if constexpr (NG == 4)
        w = *reinterpret_cast<const uint32_t*>(p);
      else if constexpr (NG == 2)
        w = *reinterpret_cast<const uint16_t*>(p);
      else
        w = *p;
#pragma unroll
      for (int j = 0; j < NG; ++j)
        r.z[j] = 0x43004300u + (static_cast<uint32_t>(w >> (8 * j)) & 15u) * 0x10001u;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NG; ++j)
    if (c * NG + j < groups) {
      r.s[j] = scale_at(a, at + j);
      if (a.zero) r.z[j] = 0x43004300u + (a.zero[at + j] & 15u) * 0x10001u;
    }
}

// Eight activations of a row in the order of expand(): XP parts of the pairs
// (0, 4), (1, 5), (2, 6), (3, 7).
template <int XP>
struct Acts {
  uint32_t p[XP][4];
};
template <int XP>
QVLA_DEVICE Acts<XP> load_acts(const void* x, int64_t at, bool in) {
  Acts<XP> r = {};
  if (!in) return r;
  if constexpr (XP == 1) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at);
    r.p[0][0] = __byte_perm(v.x, v.z, 0x5410);
    r.p[0][1] = __byte_perm(v.x, v.z, 0x7632);
    r.p[0][2] = __byte_perm(v.y, v.w, 0x5410);
    r.p[0][3] = __byte_perm(v.y, v.w, 0x7632);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    float4 lo = q[0], hi = q[1];
#pragma unroll
    for (int p = 0; p < XP; ++p) {
      r.p[p][0] = take2(lo.x, hi.x);
      r.p[p][1] = take2(lo.y, hi.y);
      r.p[p][2] = take2(lo.z, hi.z);
      r.p[p][3] = take2(lo.w, hi.w);
    }
  }
  return r;
}

// 16-byte unit of a row in its 128-byte line of a stage: lanes that read 4, 8
// or 16 bytes of 8, 4 or 2 rows at once meet no bank twice (the row's three
// low bits, reversed).
QVLA_DEVICE int unit_at(int row, int unit) {
  return unit ^ ((row & 1) << 2 | (row & 2) | (row >> 2 & 1));
}

template <int G, int MT, int XP>
__global__ void __launch_bounds__(32 * kMaxWarps, MT <= 2 ? 2 : 1)
    gemv_kernel(const __grid_constant__ GemvArgs a, const __grid_constant__ GemvShape sh) {
  constexpr int kSeg = G < 128 ? G : 128;      // K of one lane quad's load
  constexpr int kWords = kSeg / 32;            // words of eight codes per lane and load
  constexpr int NG = kChunk / G;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int wk = warp % sh.WK, wr = warp / sh.WK, W = sh.WK * sh.WR;
  const int kc = sh.KC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
  float* red = reinterpret_cast<float*>(smem + W * kStages * kStageBytes);   // [W][8 MT][33]
  constexpr int kRed = 8 * MT * 33;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int first = kc * sh.WK + wk, stride = sh.KC * sh.WK;
  const int per_tile = first < chunks ? (chunks - first + stride - 1) / stride : 0;
  const int tiles = (a.N + 32 * sh.WR - 1) / (32 * sh.WR);
  const int tile0 = blockIdx.x / sh.KC, tile_step = gridDim.x / sh.KC;
  const int my_tiles = tile0 < tiles ? (tiles - tile0 + tile_step - 1) / tile_step : 0;
  const int total = per_tile * my_tiles;
  const int m0 = blockIdx.y * 8 * MT;
  const int64_t pitch = a.K / 2;

  // the first lines of codes start for L2 before the previous kernel's end
  for (int i = 0; i < kStages - 1 && i < per_tile; ++i) {
    const int64_t n = (static_cast<int64_t>(tile0) * sh.WR + wr) * 32 + lane;
    if (total && n < a.N)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.wq + n * pitch + (first + i * stride) * 128));
  }
  pdl_launch_dependents();
  pdl_wait();

  int f_tile = tile0, f_i = 0;                 // next chunk to fetch
  auto fetch = [&](int stage) {
    const int c = first + f_i * stride;
    const int unit = lane & 7, r0 = lane >> 3;
    const int64_t n0 = (static_cast<int64_t>(f_tile) * sh.WR + wr) * 32 + r0;
    const bool col = c * 128 + unit * 16 < pitch;
    const uint8_t* src = a.wq + n0 * pitch + c * 128 + unit * 16;
    const uint32_t dst = ring + stage * kStageBytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = r0 + 4 * i;
      const bool in = col && n0 + 4 * i < a.N;
      cp_async16(dst + row * 128 + unit_at(row, unit) * 16, in ? src + 4 * i * pitch : a.wq, in);
    }
    if (++f_i == per_tile) {
      f_i = 0;
      f_tile += tile_step;
    }
  };
  int fetched = 0;
  for (int s = 0; s < kStages - 1; ++s) {
    if (fetched < total) {
      fetch(s);
      ++fetched;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const uint32_t flip = a.zero ? 0x43004300u : 0x43084308u;
  RowGroups<NG> next;
  if (total) load_groups<NG>(a, (tile0 * sh.WR + wr) * 32 + lane, first, next);

  int stage = 0;
  for (int tile = tile0; tile < tiles; tile += tile_step) {
    float acc[2][MT][4] = {};
    const int n_band = (tile * sh.WR + wr) * 32;
#pragma unroll 1
    for (int i = 0; i < per_tile; ++i) {
      const int c = first + i * stride;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      if (fetched < total) {
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        ++fetched;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      const RowGroups<NG> rg = next;
      if (i + 1 < per_tile)
        load_groups<NG>(a, n_band + lane, c + stride, next);
      else if (tile + tile_step < tiles)
        load_groups<NG>(a, ((tile + tile_step) * sh.WR + wr) * 32 + lane, first, next);
      const uint32_t base = ring + stage * kStageBytes;
      // fp32 x: the products of its first part apart from those of the rest
      float part[XP > 1 ? 2 : 1][2][MT][4] = {};
#pragma unroll
      for (int seg = 0; seg < kChunk / kSeg; ++seg) {
        const int grp = seg * kSeg / G;
        // codes of rows g, g + 8 of both halves of the band
        uint32_t w[4][kWords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = g + 8 * r;
          const int byte = seg * (kSeg / 2) + t * 4 * kWords;
          const uint32_t at = base + row * 128 + unit_at(row, byte >> 4) * 16 + (byte & 15);
          if constexpr (kWords == 4) {
            const uint4 v = lds128(at);
            w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
          } else if constexpr (kWords == 2) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[r][0]), "=r"(w[r][1]) : "r"(at) : "memory");
          } else {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[r][0]) : "r"(at) : "memory");
          }
        }
        uint32_t z[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          z[r] = a.zero ? __shfl_sync(0xffffffffu, rg.z[grp], g + 8 * r) : 0x43084308u;
        const int k0 = c * kChunk + seg * kSeg + t * 8 * kWords;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          uint32_t e[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) expand(w[r][j], flip, z[r], e[r]);
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            const int m = m0 + n * 8 + g;
            const Acts<XP> b = load_acts<XP>(a.x, static_cast<int64_t>(m) * a.ldx + k0 + 8 * j,
                                             m < a.M && k0 + 8 * j < a.K);
#pragma unroll
            for (int p = 0; p < XP; ++p)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float (&to)[4] = part[p > 0][h][n];
                mma(to, e[2 * h][0], e[2 * h + 1][0], e[2 * h][1], e[2 * h + 1][1], b.p[p][0], b.p[p][1]);
                mma(to, e[2 * h][2], e[2 * h + 1][2], e[2 * h][3], e[2 * h + 1][3], b.p[p][2], b.p[p][3]);
              }
          }
        }
        if ((seg + 1) * kSeg % G == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float s0 = __shfl_sync(0xffffffffu, rg.s[grp], g + 16 * h);
            const float s1 = __shfl_sync(0xffffffffu, rg.s[grp], g + 16 * h + 8);
#pragma unroll
            for (int q = XP > 1 ? 1 : 0; q >= 0; --q)
#pragma unroll
              for (int n = 0; n < MT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  acc[h][n][j] = fmaf(j < 2 ? s0 : s1, part[q][h][n][j], acc[h][n][j]);
                  part[q][h][n][j] = 0.f;
                }
          }
        }
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    // ---- the band's sums: over the WK warps, then over the cluster
    float* mine = red + warp * kRed;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mine[(n * 8 + 2 * t + (j & 1)) * 33 + 16 * h + g + (j >> 1) * 8] = acc[h][n][j];
    if (sh.KC > 1)
      cluster_sync();
    else
      __syncthreads();
    const int cols = min(8 * MT, a.M - m0);
    for (int x = threadIdx.x + kc * blockDim.x; x < sh.WR * 32 * cols; x += blockDim.x * sh.KC) {
      const int row = x % 32, band = x / 32 % sh.WR, col = x / 32 / sh.WR;
      const int n = (tile * sh.WR + band) * 32 + row;
      const float* at = red + band * sh.WK * kRed + col * 33 + row;
      float v = 0.f;
      if (sh.KC == 1) {
        for (int k = 0; k < sh.WK; ++k) v += at[k * kRed];
      } else {
        for (int r = 0; r < sh.KC; ++r) {
          const uint32_t far = map_shared_rank(smem_u32(at), r);
          for (int k = 0; k < sh.WK; ++k) {
            float f;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(far + k * kRed * 4) : "memory");
            v += f;
          }
        }
      }
      if (n < a.N) {
        if (a.bias) v += a.bias[n];
        const int64_t o = static_cast<int64_t>(m0 + col) * a.ldy + n;
        if (a.ydt == QVLA_DTYPE_F32)
          static_cast<float*>(a.y)[o] = v;
        else
          static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
      }
    }
    // the partial sums may be overwritten (or their CTA leave) after this
    if (sh.KC > 1)
      cluster_sync();
    else
      __syncthreads();
  }
}

// Warps, bands and cluster of a launch, from N and K alone, so that a row's
// result does not depend on the batch.  The model: an SM moves a 4 KB chunk in
// about 90 ns, a warp needs about 1 us for its first chunk and 0.25 us for
// each further one, a cluster's exchange costs about 1 us.
GemvShape gemv_shape(int N, int K, int sms) {
  const int chunks = (K + kChunk - 1) / kChunk;
  GemvShape best = {1, 1, 1};
  double best_t = 1e30;
  for (int KC = 1; KC <= 8; KC *= 2)
    for (int WK = 1; WK <= 8; WK *= 2)
      for (int WR = 1; WR * WK <= kMaxWarps; WR *= 2) {
        if (KC * WK > chunks && KC * WK > 1) continue;
        const int W = WR * WK;
        if (W < 4 && chunks >= 4) continue;
        const int64_t ctas = static_cast<int64_t>((N + 32 * WR - 1) / (32 * WR)) * KC;
        const int64_t slots = static_cast<int64_t>(sms) * (16 / W);
        if (KC > 1 && ctas > slots) continue;
        const int64_t each = (chunks + KC * WK - 1) / (KC * WK);      // chunks of a warp and band
        const double passes = static_cast<double>((ctas + slots - 1) / slots);
        const double busy = static_cast<double>((ctas + sms - 1) / sms) * W * each * 0.09;
        const double wait = 1.0 + 0.25 * (passes * each - 1) + 0.2 * passes + (KC > 1 ? 1.0 : 0.0);
        const double time = (busy > wait ? busy : wait) + 0.05 * passes + 0.01 * WK;
        if (time < best_t) {
          best_t = time;
          best = {WR, WK, KC};
        }
      }
  return best;
}

int sm_count() {
  static std::atomic<int> sms[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = sms[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) sms[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int G, int MT, int XP>
cudaError_t run_gemv(const GemvArgs& a, cudaStream_t stream) {
  auto kernel = gemv_kernel<G, MT, XP>;
  constexpr int most = kMaxWarps * (kStages * kStageBytes + 8 * MT * 33 * 4);
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms == 0) return cudaErrorUnknown;
  const GemvShape sh = gemv_shape(a.N, a.K, sms);
  const int W = sh.WR * sh.WK;
  const int64_t tiles = (a.N + 32 * sh.WR - 1) / (32 * sh.WR);
  const int64_t slots = static_cast<int64_t>(sms) * (16 / W);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * sh.KC <= slots ? tiles * sh.KC : slots),
                     (a.M + 8 * MT - 1) / (8 * MT));
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = W * (kStages * kStageBytes + 8 * MT * 33 * 4);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (sh.KC > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = sh.KC;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, a, sh);
}

template <int G>
cudaError_t run_group(const GemvArgs& a, cudaStream_t stream) {
  if (a.xdt == QVLA_DTYPE_F32)
    return a.M <= 8 ? run_gemv<G, 1, 3>(a, stream) : run_gemv<G, 2, 3>(a, stream);
  if (a.M <= 8) return run_gemv<G, 1, 1>(a, stream);
  return a.M <= 16 ? run_gemv<G, 2, 1>(a, stream) : run_gemv<G, 4, 1>(a, stream);
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
  switch (a.group) {
    case 32: return run_group<32>(a, stream);
    case 64: return run_group<64>(a, stream);
    case 128: return run_group<128>(a, stream);
    default: return run_group<256>(a, stream);
  }
}

}  // namespace qvla
