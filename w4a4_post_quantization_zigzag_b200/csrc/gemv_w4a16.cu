// W4A16: products of few activation rows with 4-bit weights that carry one
// scale (and optionally one zero point) per group of inputs.
//
//   y[m,n] = sum_g s[n,g] * ( sum_{k in g} (u[n,k] - z[n,g]) x[m,k] ) + b[n]
#include "qvla_common.cuh"
#include "qvla_internal.h"

#include <algorithm>
#include <type_traits>

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
  const float span = hi - lo;                  // past the largest float: its half over 7.5
  const float s0 = !zero            ? __fdiv_rn(fmaxf(hi, -lo), 7.f)
                   : span < INFINITY ? __fdiv_rn(span, 15.f)
                                     : __fdiv_rn(0.5f * hi - 0.5f * lo, 7.5f);
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
// Bound by reading the codes once, so the work per code has to be small.  Two
// kernels share the way the codes come and how work is dealt; one multiplies
// in integers and serves one and two activation rows, the other in bf16 and
// serves more.  (2048 -> 131072, groups of 128: one row 24.7 us in integers,
// 5.7 TB/s, against 34.5 in bf16, two rows 25.0 against 34.8, three, which
// would be two passes in integers, 51 against 35; sixteen rows 46.8 us, 3.2
// TB/s.  Groups of 32: one row 49 against 53 us.  Where the codes fit the SMs
// at once there is little between them: 4096 -> 4096, one row 5.5 against 5.2,
// two 6.2 against 5.3 us.  fp32 rows of 2048 -> 131072: one 24.8 us, four 48,
// sixteen 170, in three parts.)  One and two rows of a large matrix are bound by
// memory (87 % of the copy rate; groups below 128 by the scaling of each group);
// more rows by the warps' instructions and their latencies, about 820 per 32 x
// 256 codes at sixteen rows, half of them to expand the codes; small matrices
// by the launch and one trip to memory (1024 -> 4096: 3.8 us).  Past sixteen rows
// every sixteen read and expand all codes again (64 rows of 2048 -> 131072: 188
// us; 50 of 1024 -> 4096: 10.3).  The kernels of sixteen rows spill at 128
// registers: bf16 x 4 to 36 bytes, fp32 x up to 108.
//
// A warp multiplies bands of 32 weight rows.  A CTA has WR x WK warps: WR
// groups that take bands in turn, K dealt to the WK warps of a group in chunks
// of 256 (one 128-byte line of codes per row), and with few rows also to the
// KC CTAs of a cluster; partial sums meet in shared memory in a fixed order.
// Each warp feeds itself: one lane asks TMA for 32 rows x 128 bytes per chunk
// into the warp's own ring, which runs on across bands.
constexpr int kChunk = 256;           // K of a ring stage
constexpr int kStageBytes = 32 * kChunk / 2;
constexpr int kMaxWarps = 16;
constexpr int kStages = 3;
constexpr int kMaxSmem = 226 * 1024;

struct GemvShape {
  int WR, WK, KC;
  int stages;            // of each warp's ring
  int rows;              // activation rows of a pass
};

// What both kernels know about a warp's share of the work.
struct Share {
  int wk, wr, kc;        // this warp's place
  int first, stride, per_band;     // its chunks of K
  int band0, band_step, bands;     // its bands
  int total;             // chunks in all
  QVLA_DEVICE Share(const GemvArgs& a, const GemvShape& sh, int warp) {
    wk = warp % sh.WK;
    wr = warp / sh.WK;
    kc = sh.KC > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int chunks = (a.K + kChunk - 1) / kChunk;
    first = kc * sh.WK + wk;
    stride = sh.KC * sh.WK;
    per_band = first < chunks ? (chunks - first + stride - 1) / stride : 0;
    // bands are dealt to CTAs (clusters) one by one, a CTA's to its WR groups
    bands = (a.N + 31) / 32;
    const int step = gridDim.x / sh.KC;
    band0 = blockIdx.x / sh.KC + wr * step;
    band_step = step * sh.WR;
    total = band0 < bands ? per_band * ((bands - band0 + band_step - 1) / band_step) : 0;
  }
};

// A warp's ring of code chunks.
struct Ring {
  uint8_t* mem;
  uint64_t* bars;
  int stages, fetched, f_band, f_i;
  int stage;
  uint32_t phase;
  bool ok;               // no wait has expired; else where one did:
  int lost_stage;
  uint32_t lost_phase;

  // Before the previous kernel's end: barriers, and the first codes on their
  // way to L2.
  QVLA_DEVICE void open(uint8_t* m, uint64_t* b, int s, const Share& w, const CUtensorMap& codes, int lane) {
    mem = m;
    bars = b;
    stages = s;
    fetched = f_i = stage = 0;
    f_band = w.band0;
    phase = 0;
    ok = true;
    lost_stage = 0;
    lost_phase = 0;
    if (lane == 0) {
      for (int i = 0; i < stages; ++i) mbar_init(&bars[i], 1);
      fence_mbar_init();
      for (int i = 0; i < stages && i < w.per_band && w.total; ++i)
        tma_prefetch_l2_2d(&codes, (w.first + i * w.stride) * (kChunk / 2), w.band0 * 32);
    }
    __syncwarp();
  }
  QVLA_DEVICE void fetch(int to, const Share& w, const CUtensorMap& codes, int lane) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[to], kStageBytes);
      tma_load_2d(mem + to * kStageBytes, &codes, &bars[to], (w.first + f_i * w.stride) * (kChunk / 2),
                  f_band * 32);
    }
    ++fetched;
    if (++f_i == w.per_band) {
      f_i = 0;
      f_band += w.band_step;
    }
  }
  QVLA_DEVICE void fill(const Share& w, const CUtensorMap& codes, int lane) {
    for (int s = 0; s < stages - 1; ++s)
      if (fetched < w.total) fetch(s, w, codes, lane);
  }
  // Waits for the next chunk and asks for the one that takes the place of the
  // last (every lane has read that when all have come here).
  QVLA_DEVICE void next(const Share& w, const CUtensorMap& codes, int lane, unsigned int* err) {
    if (ok) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[stage], phase, err));
      if (!ok) {
        lost_stage = stage;
        lost_phase = phase;
      }
    }
    if (ok && fetched < w.total) fetch(stage == 0 ? stages - 1 : stage - 1, w, codes, lane);
  }
  QVLA_DEVICE void done() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // After an expired wait: one more limit for the copies in flight to land.
  QVLA_DEVICE void close(int lane, unsigned int* err) {
    if (!ok && lane == 0)
      for (int s = 0; s < stages; ++s) mbar_wait(&bars[s], lost_phase ^ (s < lost_stage), err);
  }
};

// The MMA's row g is row rho(g) of eight: with TMA's 128-byte swizzle, lanes
// that read 4, 8 or 16 bytes of 8, 4 or 2 rows at once then meet no bank twice.
QVLA_DEVICE int rho_of(int g) { return (g & 1) << 2 | (g & 2) | (g >> 2 & 1); }

// Words of eight codes of rows rho + 8 r in segment `seg` of a stage: kWords
// words per lane quad member t.
template <int kSeg, int kWords>
QVLA_DEVICE void load_codes(uint32_t stage, int seg, int rho, int t, uint32_t (&w)[4][kWords]) {
  const int byte = seg * (kSeg / 2) + t * 4 * kWords;
  const uint32_t at = stage + rho * 128 + ((byte >> 4) ^ rho) * 16 + (byte & 15);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t from = at + r * 1024;
    if constexpr (kWords == 4) {
      const uint4 v = lds128(from);
      w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
    } else if constexpr (kWords == 2) {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[r][0]), "=r"(w[r][1]) : "r"(from) : "memory");
    } else {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[r][0]) : "r"(from) : "memory");
    }
  }
}

// Scales and zero points of one row's chunk, as they lie in memory: loaded a
// chunk ahead and converted where they are used, so that no warp waits for the
// load itself.
template <int NG>
struct RawGroups {
  uint32_t s[NG];            // fp32 bits, or bf16 two to a word
  uint32_t z[(NG + 3) / 4];  // bytes
};
template <int NG>
struct RowGroups {
  float s[NG];
  float z[NG];
};

template <int NG, bool ZERO>
QVLA_DEVICE void load_groups(const GemvArgs& a, int n, int c, RawGroups<NG>& r) {
  const int groups = a.K / a.group;
  const int64_t at = static_cast<int64_t>(n) * groups + c * NG;
  if (groups % NG == 0) {
    // every row's chunk is whole and starts at a multiple of its size
    if (a.sdt == QVLA_DTYPE_F32) {
      const uint32_t* p = static_cast<const uint32_t*>(a.scale) + at;
      if constexpr (NG >= 4) {
#pragma unroll
        for (int j = 0; j < NG; j += 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(p + j);
          r.s[j] = v.x, r.s[j + 1] = v.y, r.s[j + 2] = v.z, r.s[j + 3] = v.w;
        }
      } else if constexpr (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.s[0] = v.x, r.s[1] = v.y;
      } else {
        r.s[0] = *p;
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(a.scale) + at;
      if constexpr (NG == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r.s[0] = v.x, r.s[1] = v.y, r.s[2] = v.z, r.s[3] = v.w;
      } else if constexpr (NG == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.s[0] = v.x, r.s[1] = v.y;
      } else if constexpr (NG == 2) {
        r.s[0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        r.s[0] = *p;
      }
    }
    if constexpr (ZERO) {
      const uint8_t* p = a.zero + at;
      if constexpr (NG == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.z[0] = v.x, r.z[1] = v.y;
      } else if constexpr (NG == 4) {
        r.z[0] = *reinterpret_cast<const uint32_t*>(p);
      } else if constexpr (NG == 2) {
        r.z[0] = *reinterpret_cast<const uint16_t*>(p);
      } else {
        r.z[0] = *p;
      }
    }
    return;
  }
  r = RawGroups<NG>{};
#pragma unroll
  for (int j = 0; j < NG; ++j)
    if (c * NG + j < groups) {
      if (a.sdt == QVLA_DTYPE_F32)
        r.s[j] = static_cast<const uint32_t*>(a.scale)[at + j];
      else
        r.s[j / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(a.scale)[at + j]) << (16 * (j & 1));
      if constexpr (ZERO) r.z[j / 4] |= static_cast<uint32_t>(a.zero[at + j]) << (8 * (j & 3));
    }
}

template <int NG, bool ZERO>
QVLA_DEVICE RowGroups<NG> convert_groups(const GemvArgs& a, const RawGroups<NG>& r) {
  RowGroups<NG> g = {};
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    if (a.sdt == QVLA_DTYPE_F32)
      g.s[j] = __uint_as_float(r.s[j]);
    else
      g.s[j] = __uint_as_float(j & 1 ? r.s[j / 2] & 0xffff0000u : r.s[j / 2] << 16);
    if constexpr (ZERO) g.z[j] = static_cast<float>(r.z[j >> 2] >> (8 * (j & 3)) & 15u);
  }
  return g;
}

QVLA_DEVICE void store_y(const GemvArgs& a, int m, int n, float v) {
  if (a.bias) v += a.bias[n];
  const int64_t o = static_cast<int64_t>(m) * a.ldy + n;
  if (a.ydt == QVLA_DTYPE_F32)
    static_cast<float*>(a.y)[o] = v;
  else
    static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
}

// ---- the end of a band: y[m] of weight row `lane`, for each of the pass's
// rows, summed over the WK warps, then over the cluster, and stored.
// red [W][rows][32], far [KC][rows][32].
template <int kRows>
QVLA_DEVICE void finish_band(const GemvArgs& a, const GemvShape& sh, const Share& w, int band, int warp, int lane,
                             int m0, int rows, const float (&y)[kRows], float* red, float* far) {
  const int row = band * 32 + lane;
  if (sh.WK == 1 && sh.KC == 1) {
#pragma unroll
    for (int m = 0; m < kRows; ++m)
      if (m < rows && row < a.N) store_y(a, m0 + m, row, y[m]);
    return;
  }
  if (sh.WK > 1) {
#pragma unroll
    for (int m = 0; m < kRows; ++m)
      if (m < rows) red[(warp * sh.rows + m) * 32 + lane] = y[m];
    named_barrier(1 + w.wr, 32 * sh.WK);
  }
  uint32_t to = 0;
  if (sh.KC > 1) {
    // one band per cluster (WR = 1): each CTA's sums go to the first one
    to = map_shared_rank(smem_u32(far + w.kc * sh.rows * 32), 0);
    cluster_wait();
  }
  if (sh.WK > 1) {
    for (int m = w.wk; m < rows; m += sh.WK) {
      float v = 0.f;
      for (int k = 0; k < sh.WK; ++k) v += red[((w.wr * sh.WK + k) * sh.rows + m) * 32 + lane];
      if (sh.KC > 1)
        st_shared_cluster_f32(to + (m * 32 + lane) * 4, v);
      else if (row < a.N)
        store_y(a, m0 + m, row, v);
    }
  } else {
#pragma unroll
    for (int m = 0; m < kRows; ++m)
      if (m < rows) st_shared_cluster_f32(to + (m * 32 + lane) * 4, y[m]);
  }
  if (sh.KC > 1) {
    cluster_sync();
    if (w.kc == 0)
      for (int m = w.wk; m < rows; m += sh.WK) {
        float v = 0.f;
        for (int r = 0; r < sh.KC; ++r) v += far[(r * sh.rows + m) * 32 + lane];
        if (row < a.N) store_y(a, m0 + m, row, v);
      }
  } else if (band + w.band_step < w.bands) {
    named_barrier(1 + w.wr, 32 * sh.WK);       // the sums may be overwritten after this
  }
}

// A warp's tile [8][32] of sums (columns x weight rows), transposed from the
// MMA's lanes: the lane's own weight row of each column.
QVLA_DEVICE void turn_tile(float* tile, const float (&lo)[4], const float (&hi)[4], int rho, int t, int lane,
                           float (&v)[8]) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    tile[(2 * t + (j & 1)) * 32 + ((rho + (j >> 1) * 8) ^ 8 * t)] = lo[j];
    tile[(2 * t + (j & 1)) * 32 + ((16 + rho + (j >> 1) * 8) ^ 8 * t)] = hi[j];
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = tile[q * 32 + (lane ^ 8 * (q / 2))];
}

// ============================================================ one or two rows
// Within a group, an activation row is a row of integers X = rint(x 2^e), e set
// by the group's largest |x|: 24 bits for bf16 x, 32 for fp32 x, split into
// ND = 3 or 4 signed bytes, X = sum_j 2^(8j) d_j.  Each byte plane is a column
// of the right operand (six or eight of the MMA's eight for two rows).  The
// codes become bytes by a mask and a shift, eight codes in three instructions;
// sum u d is exact in 32 bits; once per group it is scaled by s 2^(8j - e) and
// added in fp32, and at the end a row's planes are added, the smallest first.
//
// What rounding x to its group's grid costs: at most 2^-23 (bf16) or 2^-30
// (fp32) of the group's largest |x| per element, what an fp32 sum that holds
// that element may lose with every addition; for a bf16 maximum in the last
// 1/128 below a power of two, whose top byte has to hold 127 and a carry, 1.01
// times that.  bf16 values within 2^14 of the largest, and fp32 values within
// 2^6, are not rounded at all.  The grid is never finer than 2^-145 (the factor
// of the lowest byte is a float), which groups below 2^-123 (bf16) or 2^-116
// (fp32) meet.
//
// The planes are laid out in shared memory once per CTA, while the first codes
// come.

// D = A B + C, 16 x 8 x 32, signed bytes, 32-bit sums.
QVLA_DEVICE void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with every sum starting at c0.
QVLA_DEVICE void mma_s8_from(int (&c)[4], int c0, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0));
}

QVLA_DEVICE float pow2(int e) {                // 2^e for e in [-149, 127]
  return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                   : __uint_as_float(1u << (e + 149));
}

// One lane's eight activations (chunk octet `lane`) as byte planes.  `mag` is
// the largest |x| of the group (bits); returns e, the group's exponent.
// planes[j] = {bytes of x 0, 2, 4, 6, bytes of x 1, 3, 5, 7}: the order in
// which a code word's masks give the codes.
template <int ND>
QVLA_DEVICE int byte_planes(const float (&x)[8], uint32_t mag, uint2 (&planes)[ND]) {
  // ND = 3: the top byte holds 127 2^16 + ...: the last 1/128 below a power of
  // two takes the next exponent
  const int p = static_cast<int>((mag + (ND == 3 ? 0x10000u : 0u)) >> 23) - 127;
  const int e = min((ND == 3 ? 22 : 29) - p, 145);
  const float f0 = pow2(e >> 1), f1 = pow2(e - (e >> 1));
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    constexpr uint32_t bias = ND == 3 ? 0x00808080u : 0x80808080u;
    const int X = mag < 0x7f800000u ? __float2int_rn(x[i] * f0 * f1) : 0;
    b[i] = (static_cast<uint32_t>(X) + bias) ^ bias;       // two's complement bytes with carries
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo01 = __byte_perm(b[h], b[h + 2], 0x5140);       // bytes 0, 0, 1, 1
    const uint32_t lo23 = __byte_perm(b[h + 4], b[h + 6], 0x5140);
    const uint32_t hi01 = __byte_perm(b[h], b[h + 2], 0x7362);       // bytes 2, 2, 3, 3
    const uint32_t hi23 = __byte_perm(b[h + 4], b[h + 6], 0x7362);
    uint32_t w[4] = {__byte_perm(lo01, lo23, 0x5410), __byte_perm(lo01, lo23, 0x7632),
                     __byte_perm(hi01, hi23, 0x5410), __byte_perm(hi01, hi23, 0x7632)};
#pragma unroll
    for (int j = 0; j < ND; ++j) (h ? planes[j].y : planes[j].x) = w[j];
  }
  return e;
}

// Shared memory: rings, byte planes, their factors (and sums, with zero
// points), a transposing tile per warp, sums of the WK warps and of the cluster.
struct PlaneLayout {
  int slots, cols, pairs;
  uint32_t planes, factors, tile, red, far, bytes;
};

__host__ __device__ inline PlaneLayout plane_layout(const GemvShape& sh, int K, int G, int ND, bool zero) {
  PlaneLayout l;
  const int W = sh.WR * sh.WK, chunks = (K + kChunk - 1) / kChunk;
  l.slots = (chunks + sh.KC * sh.WK - 1) / (sh.KC * sh.WK) * sh.WK;
  l.cols = sh.rows * ND;
  l.pairs = (l.cols + 1) / 2;
  l.planes = W * sh.stages * kStageBytes;
  l.factors = l.planes + l.slots * kChunk * l.cols;
  l.tile = l.factors + l.slots * (kChunk / G) * l.pairs * (zero ? 16 : 8);
  l.tile = (l.tile + 15) & ~15u;
  l.red = l.tile + W * 1024;
  l.far = l.red + (sh.WK > 1 ? W * sh.rows * 128 : 0);
  l.bytes = l.far + (sh.KC > 1 ? sh.KC * sh.rows * 128 : 0) + 1024;   // + alignment of the rings
  return l;
}

// Rows past N are computed from the zeros that TMA fills in, columns past the
// last plane repeat it; neither is stored, and rows and columns of the product
// do not mix.  K ends with a group, so the last chunk's loop just ends early.
template <int G, int ND, bool ZERO>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
    gemv_planes_kernel(const __grid_constant__ GemvArgs a, const __grid_constant__ GemvShape sh,
                       const __grid_constant__ CUtensorMap codes, unsigned int* err) {
  constexpr int kSeg = G < 128 ? G : 128;      // K of one lane quad's load
  constexpr int kSegs = kChunk / kSeg;
  constexpr int kWords = kSeg / 32;            // words of eight codes per lane and load
  constexpr int NG = kChunk / G;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kMaxWarps][kStages];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, rho = rho_of(g);
  const Share w(a, sh, warp);
  const int m0 = blockIdx.y * sh.rows, rows = min(sh.rows, a.M - m0), cols = rows * ND;
  const PlaneLayout at = plane_layout(sh, a.K, G, ND, ZERO);
  uint8_t* planes = smem + at.planes;
  // [slot][NG][pair of columns]: their factors and, with zero points, sums
  float* factors = reinterpret_cast<float*>(smem + at.factors);
  constexpr int kPair = ZERO ? 4 : 2;
  float* tile = reinterpret_cast<float*>(smem + at.tile) + warp * 256;
  Ring ring;
  ring.open(smem + warp * sh.stages * kStageBytes, bars[warp], sh.stages, w, codes, lane);
  if (sh.KC > 1) cluster_arrive_relaxed();     // every CTA of the cluster runs before any writes to another
  pdl_launch_dependents();
  pdl_wait();
  ring.fill(w, codes, lane);
  RawGroups<NG> next = {};
  if (w.total) load_groups<NG, ZERO>(a, min(w.band0 * 32 + lane, a.N - 1), w.first, next);

  // ---- the byte planes of x: the chunks of this warp's share of K, dealt to
  // the WR warps that use them; slot i WK + wk is chunk first + i stride
  using X = std::conditional_t<ND == 3, uint4, float4>;
  constexpr int kVecs = ND == 3 ? 1 : 2, kBatch = ND == 3 ? 4 : 2;
  const int units = w.per_band * rows;
  for (int u0 = w.wr; u0 < units; u0 += sh.WR * kBatch) {
    X raw[kBatch][kVecs];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int u = u0 + q * sh.WR, i = u / rows, k = (w.first + i * w.stride) * kChunk + lane * 8;
      const int64_t src = static_cast<int64_t>(m0 + u - i * rows) * a.ldx + k;
#pragma unroll
      for (int h = 0; h < kVecs; ++h) {
        raw[q][h] = X{};
        if (u < units && k < a.K)
          raw[q][h] = ND == 3 ? *reinterpret_cast<const X*>(static_cast<const __nv_bfloat16*>(a.x) + src)
                              : reinterpret_cast<const X*>(static_cast<const float*>(a.x) + src)[h];
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int u = u0 + q * sh.WR;
      if (u >= units) break;
      const int i = u / rows, m = u - i * rows;
      float x[8];
      if constexpr (ND == 3) {
        const uint32_t h[4] = {raw[q][0].x, raw[q][0].y, raw[q][0].z, raw[q][0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[2 * j] = __uint_as_float(h[j] << 16);
          x[2 * j + 1] = __uint_as_float(h[j] & 0xffff0000u);
        }
      } else {
        const X v = raw[q][0], w = raw[q][kVecs - 1];
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
      }
      uint32_t mag = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mag = max(mag, __float_as_uint(x[j]) & 0x7fffffffu);
#pragma unroll
      for (int d = 1; d < G / 8; d <<= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, d));
      uint2 pl[ND];
      const int e = byte_planes<ND>(x, mag, pl);
      // this lane's octet is word j of quad lane y in segment seg
      const int seg = lane / (kSeg / 8), y = lane % (kSeg / 8) / kWords, j = lane % kWords;
      const int slot = i * sh.WK + w.wk, grp = lane / (G / 8);
      uint8_t* chunk = planes + static_cast<size_t>(slot) * kChunk * at.cols;
      const bool bad = mag >= 0x7f800000u;
#pragma unroll
      for (int p = 0; p < ND; ++p) {
        const int col = m * ND + p;
        if constexpr (kWords == 1)
          *reinterpret_cast<uint2*>(chunk + (seg * at.cols + col) * 32 + y * 8) = pl[p];
        else
          *reinterpret_cast<uint2*>(chunk + ((seg * (kWords / 2) + j / 2) * at.cols + col) * 64 + y * 16 +
                                    j % 2 * 8) = pl[p];
        int sum = 0;
        if constexpr (ZERO) {
          sum = __dp4a(static_cast<int>(pl[p].x), 0x01010101, __dp4a(static_cast<int>(pl[p].y), 0x01010101, 0));
#pragma unroll
          for (int d = 1; d < G / 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        }
        if (lane % (G / 8) == 0) {
          // two's complement codes enter as 16 times their value
          float* to = factors + ((slot * NG + grp) * at.pairs + col / 2) * kPair + col % 2;
          to[0] = bad ? __uint_as_float(0x7fc00000u) : pow2(8 * p - e - (ZERO ? 0 : 4));
          if constexpr (ZERO) to[2] = static_cast<float>(sum);
        }
      }
    }
  }
  if (sh.WR > 1)
    __syncthreads();
  else
    __syncwarp();

  // this lane's column as operand, its pair of columns as result
  const int col_b = min(g, cols - 1) * (kWords == 1 ? 32 : 64) + t * (kWords == 1 ? 8 : 16);
  const int pair_c = min(t, at.pairs - 1) * kPair;
  constexpr uint32_t mask = ZERO ? 0x0f0f0f0fu : 0xf0f0f0f0u;
  for (int band = w.band0; band < w.bands; band += w.band_step) {
    float acc[2][4] = {};
#pragma unroll 1
    for (int i = 0; i < w.per_band; ++i) {
      const int c = w.first + i * w.stride, slot = i * sh.WK + w.wk;
      ring.next(w, codes, lane, err);
      const RowGroups<NG> rg = convert_groups<NG, ZERO>(a, next);
      if (i + 1 < w.per_band)
        load_groups<NG, ZERO>(a, min(band * 32 + lane, a.N - 1), c + w.stride, next);
      else if (band + w.band_step < w.bands)
        load_groups<NG, ZERO>(a, min((band + w.band_step) * 32 + lane, a.N - 1), w.first, next);
      const uint32_t stage = smem_u32(ring.mem) + ring.stage * kStageBytes;
      const uint8_t* chunk = planes + static_cast<size_t>(slot) * kChunk * at.cols;
      int part[2][4];
#pragma unroll
      for (int seg = 0; seg < kSegs; ++seg) {
        if (c * kChunk + seg * kSeg >= a.K) break;
        const int grp = seg * kSeg / G;
        uint32_t u[4][kWords];
        load_codes<kSeg, kWords>(stage, seg, rho, t, u);
#pragma unroll
        for (int j2 = 0; j2 < (kWords + 1) / 2; ++j2) {
          uint32_t b[2][2];
          if constexpr (kWords == 1) {
            const uint2 v = *reinterpret_cast<const uint2*>(chunk + seg * at.cols * 32 + col_b);
            b[0][0] = v.x, b[0][1] = v.y;
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(
                chunk + (seg * (kWords / 2) + j2) * at.cols * 64 + col_b);
            b[0][0] = v.x, b[0][1] = v.y, b[1][0] = v.z, b[1][1] = v.w;
          }
#pragma unroll
          for (int jj = 0; jj < (kWords == 1 ? 1 : 2); ++jj) {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t v = u[r][2 * j2 + jj];
              lo[r] = (ZERO ? v : v << 4) & mask;
              hi[r] = (ZERO ? v >> 4 : v) & mask;
            }
            // a sum that starts at the bits of 1.5 2^23 ends as the bits of
            // 1.5 2^23 + itself (|sum| <= 256 * 128 * 128)
            const bool opens = seg * kSeg % G == 0 && j2 == 0 && jj == 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (opens)
                mma_s8_from(part[h], 0x4b400000, lo[2 * h], lo[2 * h + 1], hi[2 * h], hi[2 * h + 1], b[jj][0],
                            b[jj][1]);
              else
                mma_s8(part[h], lo[2 * h], lo[2 * h + 1], hi[2 * h], hi[2 * h + 1], b[jj][0], b[jj][1]);
            }
          }
        }
        if ((seg + 1) * kSeg % G == 0) {
          const float* fp = factors + (slot * NG + grp) * at.pairs * kPair + pair_c;
          const float2 f = *reinterpret_cast<const float2*>(fp);
          float2 sum = {};
          if constexpr (ZERO) sum = *reinterpret_cast<const float2*>(fp + 2);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float s = __shfl_sync(0xffffffffu, rg.s[grp], rho + 16 * h + 8 * r);
              float v0 = __int_as_float(part[h][2 * r]) - 12582912.f;
              float v1 = __int_as_float(part[h][2 * r + 1]) - 12582912.f;
              if constexpr (ZERO) {                      // exact: below 2^22
                const float z = __shfl_sync(0xffffffffu, rg.z[grp], rho + 16 * h + 8 * r);
                v0 = fmaf(-z, sum.x, v0);
                v1 = fmaf(-z, sum.y, v1);
              }
              acc[h][2 * r] = fmaf(v0 * s, f.x, acc[h][2 * r]);
              acc[h][2 * r + 1] = fmaf(v1 * s, f.y, acc[h][2 * r + 1]);
            }
        }
      }
      ring.done();
    }
    float v[8], y[2] = {};
    turn_tile(tile, acc[0], acc[1], rho, t, lane, v);
#pragma unroll
    for (int q = 0; q < 2 * ND; ++q) y[q / ND] += v[q];
    finish_band(a, sh, w, band, warp, lane, m0, rows, y, reinterpret_cast<float*>(smem + at.red),
                reinterpret_cast<float*>(smem + at.far));
  }
  ring.close(lane, err);
}

// ============================================================== three and more
// The codes become exact bf16 values (u - z) in registers, x enters as bf16
// (fp32 x as three bf16 parts whose sum is x, down to 2^-133), every product is exact, a
// group's sum is fp32 and is scaled once.  The order of K inside an MMA is free
// as long as both operands agree, so a lane takes the codes as they lie in
// memory, eight per 32-bit word, and meets them with activations in that order.

QVLA_DEVICE void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from a zero sum.
QVLA_DEVICE void mma_bf16_from0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// Eight activations of a row in the order of expand(): XP parts of the pairs
// (0, 4), (1, 5), (2, 6), (3, 7).
template <int XP>
struct Acts {
  uint32_t p[XP][4];
};
template <int XP, typename X>
QVLA_DEVICE Acts<XP> load_acts(const X* x) {
  Acts<XP> r;
  const uint4 v = reinterpret_cast<const uint4*>(x)[0];
  if constexpr (XP == 1) {
    r.p[0][0] = __byte_perm(v.x, v.z, 0x5410);
    r.p[0][1] = __byte_perm(v.x, v.z, 0x7632);
    r.p[0][2] = __byte_perm(v.y, v.w, 0x5410);
    r.p[0][3] = __byte_perm(v.y, v.w, 0x7632);
  } else {
    const uint4 u = reinterpret_cast<const uint4*>(x)[1];
    float lo[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
    float hi[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
#pragma unroll
    for (int p = 0; p < XP; ++p)
#pragma unroll
      for (int j = 0; j < 4; ++j) r.p[p][j] = take2(lo[j], hi[j]);
  }
  return r;
}

// Shared memory: rings, a transposing tile per warp, sums of the WK warps and
// of the cluster, the activations in operand order if they are staged.
struct PartLayout {
  uint32_t tile, red, far, acts, bytes;
};

__host__ __device__ inline PartLayout part_layout(const GemvShape& sh, int K, int XP, bool staged) {
  PartLayout l;
  const int W = sh.WR * sh.WK;
  l.tile = W * sh.stages * kStageBytes;
  l.red = l.tile + W * 1024;
  l.far = l.red + (sh.WK > 1 ? W * sh.rows * 128 : 0);
  l.acts = l.far + (sh.KC > 1 ? sh.KC * sh.rows * 128 : 0);
  l.bytes = l.acts + (staged ? K * sh.rows * 2 * XP : 0) + 1024;
  return l;
}

// As above; columns past the last activation row repeat it and are not stored.
template <int G, int MT, int XP, bool STAGED>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
    gemv_parts_kernel(const __grid_constant__ GemvArgs a, const __grid_constant__ GemvShape sh,
                      const __grid_constant__ CUtensorMap codes, unsigned int* err) {
  using X = std::conditional_t<XP == 1, __nv_bfloat16, float>;
  constexpr int kSeg = G < 128 ? G : 128;
  constexpr int kSegs = kChunk / kSeg;
  constexpr int kWords = kSeg / 32;
  constexpr int NG = kChunk / G;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kMaxWarps][kStages];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, rho = rho_of(g);
  const Share w(a, sh, warp);
  const int m0 = blockIdx.y * sh.rows, cols = min(sh.rows, a.M - m0);
  const PartLayout at = part_layout(sh, a.K, XP, STAGED);
  float* tile = reinterpret_cast<float*>(smem + at.tile) + warp * 256;
  uint4* xs = reinterpret_cast<uint4*>(smem + at.acts);
  Ring ring;
  ring.open(smem + warp * sh.stages * kStageBytes, bars[warp], sh.stages, w, codes, lane);
  if (sh.KC > 1) cluster_arrive_relaxed();
  pdl_launch_dependents();
  pdl_wait();
  ring.fill(w, codes, lane);
  const bool zero = a.zero != nullptr;
  const uint32_t flip = zero ? 0x43004300u : 0x43084308u;
  RawGroups<NG> next = {};
  auto load_next = [&](int n, int c) {
    if (zero)
      load_groups<NG, true>(a, min(n, a.N - 1), c, next);
    else
      load_groups<NG, false>(a, min(n, a.N - 1), c, next);
  };
  if (w.total) load_next(w.band0 * 32 + lane, w.first);
  const X* xrow[MT];                           // direct: this lane's place in its activation rows
  int xcol[MT];                                // staged: its columns
#pragma unroll
  for (int n = 0; n < MT; ++n) {
    xcol[n] = min(n * 8 + g, cols - 1);
    xrow[n] = static_cast<const X*>(a.x) + static_cast<int64_t>(m0 + xcol[n]) * a.ldx + t * 8 * kWords;
  }
  if constexpr (STAGED) {
    // 16-byte pieces in the order the lanes read them: [segment, word, part]
    // [column][t], so that the eight lanes of a quarter warp meet no bank twice
    const int pieces = a.K / 8;
    for (int i = threadIdx.x; i < pieces * cols; i += blockDim.x) {
      const int k8 = i % pieces, col = i / pieces;
      const int seg = k8 / (kSeg / 8), q = k8 % (kSeg / 8);
      const Acts<XP> v =
          load_acts<XP>(static_cast<const X*>(a.x) + static_cast<int64_t>(m0 + col) * a.ldx + k8 * 8);
#pragma unroll
      for (int p = 0; p < XP; ++p)
        xs[(((seg * kWords + q % kWords) * XP + p) * cols + col) * 4 + q / kWords] =
            make_uint4(v.p[p][0], v.p[p][1], v.p[p][2], v.p[p][3]);
    }
    __syncthreads();
  }
  for (int band = w.band0; band < w.bands; band += w.band_step) {
    float acc[2][MT][4] = {};
#pragma unroll 1
    for (int i = 0; i < w.per_band; ++i) {
      const int c = w.first + i * w.stride;
      ring.next(w, codes, lane, err);
      const RowGroups<NG> rg = convert_groups<NG, false>(a, next);
      uint32_t zs[(NG + 3) / 4];
#pragma unroll
      for (int j = 0; j < (NG + 3) / 4; ++j) zs[j] = next.z[j];
      if (i + 1 < w.per_band)
        load_next(band * 32 + lane, c + w.stride);
      else if (band + w.band_step < w.bands)
        load_next((band + w.band_step) * 32 + lane, w.first);
      const uint32_t stage = smem_u32(ring.mem) + ring.stage * kStageBytes;
      // fp32 x: its first part's sums apart from the rest's, which the MMA would
      // cut off (a second chain for bf16 x: 54.1 against 50.2 us at 16 rows)
      float part[XP == 1 ? 1 : 2][2][MT][4];
#pragma unroll
      for (int seg = 0; seg < kSegs; ++seg) {
        if (c * kChunk + seg * kSeg >= a.K) break;
        const int grp = seg * kSeg / G;
        uint32_t u[4][kWords];
        load_codes<kSeg, kWords>(stage, seg, rho, t, u);
        uint32_t z[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] = 0x43084308u;
        if (zero) {
          const uint32_t mine = (zs[grp >> 2] >> (8 * (grp & 3)) & 15u) * 0x10001u + 0x43004300u;
#pragma unroll
          for (int r = 0; r < 4; ++r) z[r] = __shfl_sync(0xffffffffu, mine, rho + 8 * r);
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          uint32_t e[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) expand(u[r][j], flip, z[r], e[r]);
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            Acts<XP> b;
            if constexpr (STAGED) {
              const int piece = ((c * kSegs + seg) * kWords + j) * XP;
#pragma unroll
              for (int p = 0; p < XP; ++p) {
                const uint4 v = xs[((piece + p) * cols + xcol[n]) * 4 + t];
                b.p[p][0] = v.x, b.p[p][1] = v.y, b.p[p][2] = v.z, b.p[p][3] = v.w;
              }
            } else {
              b = load_acts<XP>(xrow[n] + c * kChunk + seg * kSeg + 8 * j);
            }
#pragma unroll
            for (int p = 0; p < XP; ++p)
#pragma unroll
              for (int d = 0; d < 2; ++d) {              // the word's two MMAs
                const int q = p > 0;
                const bool opens = seg * kSeg % G == 0 && j == 0 && d == 0 && p < 2;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  if (opens)
                    mma_bf16_from0(part[q][h][n], e[2 * h][2 * d], e[2 * h + 1][2 * d], e[2 * h][2 * d + 1],
                                   e[2 * h + 1][2 * d + 1], b.p[p][2 * d], b.p[p][2 * d + 1]);
                  else
                    mma_bf16(part[q][h][n], e[2 * h][2 * d], e[2 * h + 1][2 * d], e[2 * h][2 * d + 1],
                             e[2 * h + 1][2 * d + 1], b.p[p][2 * d], b.p[p][2 * d + 1]);
                }
              }
          }
        }
        if ((seg + 1) * kSeg % G == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float s0 = __shfl_sync(0xffffffffu, rg.s[grp], rho + 16 * h);
            const float s1 = __shfl_sync(0xffffffffu, rg.s[grp], rho + 16 * h + 8);
#pragma unroll
            for (int q = XP > 1; q >= 0; --q)
#pragma unroll
              for (int n = 0; n < MT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  acc[h][n][j] = fmaf(j < 2 ? s0 : s1, part[q][h][n][j], acc[h][n][j]);
          }
        }
      }
      ring.done();
    }
    float y[8 * MT];
#pragma unroll
    for (int n = 0; n < MT; ++n) {
      float v[8];
      turn_tile(tile, acc[0][n], acc[1][n], rho, t, lane, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) y[n * 8 + q] = v[q];
    }
    finish_band(a, sh, w, band, warp, lane, m0, cols, y, reinterpret_cast<float*>(smem + at.red),
                reinterpret_cast<float*>(smem + at.far));
  }
  ring.close(lane, err);
}

// ============================================================== launches
// Warps, bands and cluster of a launch, from N and K alone (a row's result
// then depends on M only as far as the kernel does).  K is split as far as it
// takes to give every one of 16 warps per SM a piece, first over the warps of a
// CTA (exchange within its shared memory), then over a cluster's CTAs.  Against
// the best of all splits with powers of two this was at most 8 % slower at
// twelve sizes from 256 -> 256 to 2048 -> 131072.
GemvShape gemv_shape(int N, int K, int sms) {
  const int bands = (N + 31) / 32, chunks = (K + kChunk - 1) / kChunk;
  int split = 1;
  while (2 * split <= chunks && 2 * split * bands <= 16 * sms) split *= 2;
  GemvShape s = {};
  s.WK = std::min(split, 8);
  s.KC = std::min(split / s.WK, 8);
  // eight warps a CTA; sixteen where a band has one or eight and there are bands enough
  s.WR = s.KC > 1 ? 1 : std::max(1, (s.WK == 1 || s.WK == 8 ? 16 : 8) / s.WK);
  while (s.WR > 1 && (s.WR - 1) * sms / 2 >= bands) s.WR /= 2;
  s.stages = kStages;
  return s;
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

// CTAs of an SM: what its shared memory and 512 threads of 128 registers hold.
int resident_ctas(const GemvShape& sh, uint32_t smem) {
  return std::max(1, std::min(227 * 1024 / static_cast<int>(smem + 2048), kMaxWarps / (sh.WR * sh.WK)));
}

int64_t wanted_ctas(const GemvShape& sh, int N) {
  return static_cast<int64_t>(((N + 31) / 32 + sh.WR - 1) / sh.WR) * sh.KC;
}

template <typename K>
cudaError_t launch_gemv(K kernel, std::atomic<unsigned long long>& done, const GemvArgs& a, const GemvShape& sh,
                        uint32_t smem, int sms, cudaStream_t stream) {
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap codes;
  if (!encode_map_2d(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq, a.K / 2, a.N, a.K / 2, kChunk / 2, 32,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  const int64_t ctas = wanted_ctas(sh, a.N);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(
                         sh.KC > 1 ? ctas : std::min<int64_t>(ctas, sms * resident_ctas(sh, smem))),
                     (a.M + sh.rows - 1) / sh.rows);
  cfg.blockDim = dim3(32 * sh.WR * sh.WK);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, kernel, a, sh, codes, err);
}

// Gives up ring stages, then bands at a time (neither changes a result), until
// `bytes` of shared memory fit; then the third stage, where without it more
// CTAs are on an SM at once and there are CTAs for them (16384 -> 2048, one
// row: 8.2 against 13.6 us).
template <typename F>
bool make_fit(GemvShape& sh, int N, int sms, F bytes) {
  while (bytes(sh) > kMaxSmem) {
    if (sh.stages > 2)
      --sh.stages;
    else if (sh.WR > 1)
      sh.WR /= 2;
    else
      return false;
  }
  if (sh.stages > 2) {
    GemvShape two = sh;
    two.stages = 2;
    const int now = resident_ctas(sh, bytes(sh));
    if (resident_ctas(two, bytes(two)) > now && wanted_ctas(sh, N) > static_cast<int64_t>(now) * sms) sh = two;
  }
  return true;
}

template <int G, int ND, bool ZERO>
cudaError_t run_planes(const GemvArgs& a, GemvShape sh, int sms, cudaStream_t stream) {
  auto bytes = [&](const GemvShape& s) { return plane_layout(s, a.K, G, ND, ZERO).bytes; };
  sh.rows = a.M;
  const GemvShape whole = sh;
  if (!make_fit(sh, a.N, sms, bytes)) {                  // two rows of the largest K: one pass each
    sh = whole;
    sh.rows = 1;
    while (!make_fit(sh, a.N, sms, bytes)) sh.WK /= 2;   // and with the finest groups fewer warps
  }
  static std::atomic<unsigned long long> done{0};
  return launch_gemv(gemv_planes_kernel<G, ND, ZERO>, done, a, sh, bytes(sh), sms, stream);
}

template <int G, int MT, int XP>
cudaError_t run_parts(const GemvArgs& a, GemvShape sh, int sms, cudaStream_t stream) {
  sh.rows = std::min(a.M, 8 * MT);
  // Operand order is worth its staging where warps take several bands
  // (2048 -> 131072, when measured: 16 rows 56.5 against 67.5 us, 8 rows 39.2
  // against 51.9) or the activations have to be split (1536 -> 6144, seven fp32
  // rows: 9.6 against 12.2 us), and the activations leave room for rings of two
  // stages.  With one band a warp it changes nothing (4096 -> 4096, 16 rows).
  GemvShape st = sh;
  if (sh.KC == 1 && (XP > 1 || wanted_ctas(sh, a.N) > sms)) {
    auto bytes = [&](const GemvShape& s) { return part_layout(s, a.K, XP, true).bytes; };
    while (st.stages > 2 && bytes(st) > kMaxSmem) --st.stages;
    if (bytes(st) <= kMaxSmem) {
      make_fit(st, a.N, sms, bytes);
      static std::atomic<unsigned long long> done{0};
      return launch_gemv(gemv_parts_kernel<G, MT, XP, true>, done, a, st, bytes(st), sms, stream);
    }
  }
  auto bytes = [&](const GemvShape& s) { return part_layout(s, a.K, XP, false).bytes; };
  if (!make_fit(sh, a.N, sms, bytes)) return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done{0};
  return launch_gemv(gemv_parts_kernel<G, MT, XP, false>, done, a, sh, bytes(sh), sms, stream);
}

template <int G>
cudaError_t run_group(const GemvArgs& a, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms == 0) return cudaErrorUnknown;
  const GemvShape sh = gemv_shape(a.N, a.K, sms);
  const bool f32 = a.xdt == QVLA_DTYPE_F32;
  if (a.M <= 2) {
    if (f32) return a.zero ? run_planes<G, 4, true>(a, sh, sms, stream) : run_planes<G, 4, false>(a, sh, sms, stream);
    return a.zero ? run_planes<G, 3, true>(a, sh, sms, stream) : run_planes<G, 3, false>(a, sh, sms, stream);
  }
  if (f32) return a.M <= 8 ? run_parts<G, 1, 3>(a, sh, sms, stream) : run_parts<G, 2, 3>(a, sh, sms, stream);
  return a.M <= 8 ? run_parts<G, 1, 1>(a, sh, sms, stream) : run_parts<G, 2, 1>(a, sh, sms, stream);
}

}  // namespace

cudaError_t launch_pack_w4g(const float* W, int N, int K, int group, qvla_dtype sdt, uint8_t* wq,
                            void* scale, uint8_t* zero, cudaStream_t s) {
  const int64_t groups = static_cast<int64_t>(N) * (K / group);
  // a launch that returns its own status, not an error that an earlier call left
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((groups + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  if (sdt == QVLA_DTYPE_F32)
    return cudaLaunchKernelEx(&cfg, pack_w4g_kernel<float>, W, groups, group, wq, static_cast<float*>(scale), zero);
  return cudaLaunchKernelEx(&cfg, pack_w4g_kernel<__nv_bfloat16>, W, groups, group, wq,
                            static_cast<__nv_bfloat16*>(scale), zero);
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
