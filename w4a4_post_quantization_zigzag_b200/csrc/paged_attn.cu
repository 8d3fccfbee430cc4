// Attention of one new token per sequence over a paged key/value cache.
//
//   o = sum_t p_t v_t,  p = softmax over the visible t of scale * q . k_t
//
// Bound by reading the cache once: a key head's rows serve all query heads of
// its group, which are the columns of two small matrix products per 16 tokens,
//   S^T [16 tokens x heads] = K [16 x D] Q^T [D x heads]
//   O^T [D x heads]        += V^T [D x 16] P^T [16 x heads]
// with tokens (then head values) in the rows of the warp-level MMA, so that a
// group of 8 heads fills its columns.  The running maximum and sum of the
// softmax are per column; the output stays in registers.
//
// Work split.  The visible tokens of all sequences and key heads, in tiles of
// 16, form one line of T tiles that is cut into equal pieces, one per warp of
// a grid that fills the card once: ragged lengths, few heads or one long
// sequence all balance the same way.  A piece may end inside a sequence; what
// a warp holds of an unfinished (sequence, head) is joined first with its
// neighbours in the CTA (shared memory), then across CTAs by a second small
// launch, each in the fixed order of the line.  Hidden tokens of a window are
// not on the line at all, so nothing inside it is masked.
//
// Each warp feeds itself: cp.async of its own tiles into its own ring of
// shared memory, no barrier with other warps before the join.
#include "qvla_common.cuh"
#include "qvla_internal.h"

#include <algorithm>

namespace qvla {
namespace {

constexpr int kMaxCtas = 160;         // at most this many CTAs split the line
constexpr int kSlotHeads = 16;        // statistics per slot (heads of a unit)

// ------------------------------------------------------------- primitives
QVLA_DEVICE void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
QVLA_DEVICE void cp_async4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0)
               : "memory");
}
QVLA_DEVICE void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
QVLA_DEVICE void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
QVLA_DEVICE void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
QVLA_DEVICE void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
QVLA_DEVICE uint32_t movm_t(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// D += A B, 16 x 8 x 16, bf16 in, fp32 sums.
QVLA_DEVICE void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
QVLA_DEVICE float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
QVLA_DEVICE uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The bf16 values below two fp32 values (cut, not rounded: the rest keeps the
// sign and no value overflows), and what they leave.
QVLA_DEVICE uint32_t take2(float& lo, float& hi) {
  const uint32_t a = __float_as_uint(lo) & 0xffff0000u, b = __float_as_uint(hi) & 0xffff0000u;
  lo -= __uint_as_float(a);
  hi -= __uint_as_float(b);
  return a >> 16 | b;
}
// The 8-bit codes in bytes 0 and 2 of w as exact bf16 values: 128 + the low
// seven bits, less 128 or (code negative) 256.
QVLA_DEVICE uint32_t codes2(uint32_t w) {
  const uint32_t a = (w & 0x007f007fu) | 0x43004300u, b = (w & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ---------------------------------------------------------------- line of tiles
struct Span {                        // what the new token of a sequence sees
  int visible, gap;                  // tokens on the line; hidden tokens before token `sinks`
};

QVLA_DEVICE bool good_len(const PagedAttnArgs& a, int n) {
  return n >= 0 && n <= static_cast<int64_t>(a.max_pages) * a.cache.page_size;
}

QVLA_DEVICE Span span_of(const PagedAttnArgs& a, int b) {
  const int n = a.seq_lens[b];
  if (!good_len(a, n)) return {0, 0};
  const int64_t seen = static_cast<int64_t>(a.window) + a.sinks;
  if (a.window == 0 || n <= seen) return {n, 0};
  return {static_cast<int>(seen), static_cast<int>(n - seen)};
}

struct Cursor {
  int b, hu, tile, tiles;
  Span s;
  QVLA_DEVICE void seek(const PagedAttnArgs& a) {      // first sequence from b on with tokens
    for (; b < a.B; ++b) {
      s = span_of(a, b);
      tiles = (s.visible + 15) / 16;
      if (tiles) return;
    }
  }
  QVLA_DEVICE void next(const PagedAttnArgs& a, int HU) {
    if (++tile < tiles) return;
    tile = 0;
    if (++hu < HU) return;
    hu = 0;
    ++b;
    seek(a);
  }
};

// Global scratch: per CTA two joined partial results (0: of a unit that began
// in an earlier CTA, 1: of one that begins here and ends later) and per warp
// one (of a unit that began in an earlier warp).
struct Scratch {
  int4* leader;          // [kMaxCtas]: {b, unit head, last CTA, 1 if slot 1 awaits its join}
  float2* stat;          // [kMaxCtas][2][kSlotHeads] maximum (log2) and sum
  float* o;              // [kMaxCtas][2][heads][DP]
  float* warp_o;         // [kMaxCtas][W][heads][DP]
};

__host__ __device__ constexpr size_t scratch_head_bytes() {
  return kMaxCtas * sizeof(int4) + kMaxCtas * 2 * kSlotHeads * sizeof(float2);
}

template <int HEADS, int DP>
__host__ __device__ Scratch scratch_at(void* ws) {
  Scratch s;
  s.leader = static_cast<int4*>(ws);
  s.stat = reinterpret_cast<float2*>(s.leader + kMaxCtas);
  s.o = reinterpret_cast<float*>(s.stat + kMaxCtas * 2 * kSlotHeads);
  s.warp_o = s.o + static_cast<size_t>(kMaxCtas) * 2 * HEADS * DP;
  return s;
}

template <typename X>
QVLA_DEVICE void store_out(const PagedAttnArgs& a, int b, int h, int d, float v) {
  X* p = static_cast<X*>(a.out) + b * a.ldo + static_cast<int64_t>(h) * a.cache.dim + d;
  if constexpr (sizeof(X) == 2)
    *p = __float2bfloat16_rn(v);
  else
    *p = v;
}

template <typename X>
QVLA_DEVICE void store_out4(const PagedAttnArgs& a, int b, int h, int d, float4 v) {
  X* p = static_cast<X*>(a.out) + b * a.ldo + static_cast<int64_t>(h) * a.cache.dim + d;
  if constexpr (sizeof(X) == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
  else
    *reinterpret_cast<float4*>(p) = v;
}

// log of the sum of exponentials from a maximum in base 2 and the sum.
QVLA_DEVICE float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// The factor that takes a sum relative to maximum m to one relative to M.
QVLA_DEVICE float weight(float m, float M) { return m == -INFINITY ? 0.f : exp2_fast(m - M); }

// DP: head dim rounded up; NT: columns of 8 query heads; QP: bf16 parts of q
// and p (1 for bf16 q, 3 for fp32: their sum is the whole value); BITS of the
// cache; W warps, S stages of one tile each per warp.
template <int DP, int NT, int QP, int BITS, int W, int S>
struct Shape {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kRow = DP * BITS / 8;               // bytes of a token's row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kTile = 16 * kRow;
  static constexpr int kStage = 2 * kTile + (BITS == 8 ? 128 : 0);
  static constexpr int kSmem = W * S * kStage;
  static_assert(S * kStage >= kHeads * DP * 4, "a warp's ring holds its last partial result");
};

template <typename X, int DP, int NT, int QP, int BITS, int W, int S>
__global__ void __launch_bounds__(32 * W, 1)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, unsigned int* err) {
  using Sh = Shape<DP, NT, QP, BITS, W, S>;
  constexpr int kHeads = Sh::kHeads, kChunks = Sh::kChunks, kKs = DP / 16;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int4 meta[W][S];                 // {b, unit head, valid rows | begins << 16 | ends << 17, 0}
  __shared__ int64_t scan[W];
  __shared__ int64_t start_before[W];         // tiles of a head before the sequence
  __shared__ int start_b[W];
  __shared__ int4 slot[W][2];                 // {b (-1: empty), unit head, begins, ends}
  __shared__ float2 slot_stat[W][2][kHeads];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.cache.dim, G = a.Hq / a.cache.heads;
  const int HT = (G + kHeads - 1) / kHeads, HU = a.cache.heads * HT;
  const Scratch ws = scratch_at<kHeads, DP>(a.ws);
  if (threadIdx.x < 2 * W) (&slot[0][0])[threadIdx.x] = make_int4(-1, 0, 0, 0);
  pdl_launch_dependents();
  pdl_wait();

  // ---- the line: tiles of one head before each thread's share of sequences
  const int per = (a.B + 32 * W - 1) / (32 * W);
  const int b_lo = min(static_cast<int>(threadIdx.x) * per, a.B), b_hi = min(b_lo + per, a.B);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += (span_of(a, b).visible + 15) / 16;
  int64_t upto = mine;
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  int64_t before = upto - mine, all = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += scan[w];
    all += scan[w];
  }
  const int64_t T = all * HU;
  const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (T + W - 1) / W));
  const int64_t pieces = static_cast<int64_t>(ctas) * W;
  const bool works = static_cast<int>(blockIdx.x) < ctas;
  if (works) {
    for (int w = 0; w < W; ++w) {
      const int64_t x = (static_cast<int64_t>(blockIdx.x) * W + w) * T / pieces;
      if (x >= before * HU && x < (before + mine) * HU) {
        int64_t at = before;
        int b = b_lo;
        for (;; ++b) {
          const int64_t n = (span_of(a, b).visible + 15) / 16;
          if (x < (at + n) * HU) break;
          at += n;
        }
        start_b[w] = b;
        start_before[w] = at;
      }
    }
  }
  __syncthreads();

  int4 lead = make_int4(0, 0, 0, 0);
  if (works) {
    const int64_t lo = (static_cast<int64_t>(blockIdx.x) * W + warp) * T / pieces;
    const int64_t hi = (static_cast<int64_t>(blockIdx.x) * W + warp + 1) * T / pieces;
    const int count = static_cast<int>(hi - lo);
    const uint32_t ring0 = smem_u32(ring) + warp * S * Sh::kStage;

    Cursor in;
    in.b = count ? start_b[warp] : a.B;
    in.hu = in.tile = in.tiles = 0;
    if (count) {
      in.s = span_of(a, in.b);
      in.tiles = (in.s.visible + 15) / 16;
      const int64_t off = lo - start_before[warp] * HU;
      in.hu = static_cast<int>(off / in.tiles);
      in.tile = static_cast<int>(off - static_cast<int64_t>(in.hu) * in.tiles);
    }

    // ---- feeding: the page of each row is read one tile ahead of its copy
    int row_page = 0, row_tok = 0;
    bool row_in = false;
    auto look_up = [&] {
      const int v = in.tile * 16 + (lane & 15);
      row_in = v < in.s.visible;
      const int t = row_in ? (v >= a.sinks ? v + in.s.gap : v) : 0;
      const int p = t / a.cache.page_size;
      row_tok = t - p * a.cache.page_size;
      row_page = row_in ? a.page_table[static_cast<int64_t>(in.b) * a.max_pages + p] : 0;
    };
    auto feed = [&](int stage) {
      const bool found = row_page >= 0 && row_page < a.cache.pages;
      if (row_in && !found && lane < 16) report(err, QVLA_DEVERR_CACHE_RANGE);
      const bool ok = row_in && found;
      const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const int kh = in.hu / HT;
      const int64_t off = ok ? row_page * a.cache.page_stride + row_tok * a.cache.token_stride +
                                   kh * a.cache.head_stride
                             : 0;
      const uint32_t dst0 = ring0 + stage * Sh::kStage;
      const int chunk = lane % kChunks;
      const bool col = chunk * (128 / BITS) < D;
#pragma unroll
      for (int i = 0; i < kChunks / 2; ++i) {
        const int row = i * (32 / kChunks) + lane / kChunks;
        const int64_t ro = __shfl_sync(0xffffffffu, off, row) * (BITS / 8) + chunk * 16;
        const bool take = col && (mask >> row & 1);
        const int phys = kChunks == 4 ? chunk ^ (row >> 1 & 3) : chunk ^ (row & 7);
        const uint32_t dst = dst0 + row * Sh::kRow + phys * 16;
        cp_async16(dst, static_cast<const uint8_t*>(a.cache.k) + (take ? ro : 0), take);
        cp_async16(dst + Sh::kTile, static_cast<const uint8_t*>(a.cache.v) + (take ? ro : 0), take);
      }
      if constexpr (BITS == 8) {
        const int64_t so = ok ? row_page * a.cache.s_page_stride + row_tok * a.cache.s_token_stride +
                                    kh * a.cache.s_head_stride
                              : 0;
        cp_async4(dst0 + 2 * Sh::kTile + lane * 4, (lane < 16 ? a.cache.k_scale : a.cache.v_scale) + so, ok);
      }
      if (lane == 0)
        meta[warp][stage] = make_int4(in.b, in.hu, static_cast<int>(mask) | (in.tile == 0) << 16 |
                                                       (in.tile == in.tiles - 1) << 17, 0);
    };

    int fed = 0;
    if (count) look_up();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) {
      if (fed < count) {
        feed(s);
        if (++fed < count) {
          in.next(a, HU);
          look_up();
        }
      }
      cp_async_commit();
    }

    // ---- consuming
    const int g = lane >> 2, t4 = lane & 3;      // row and column pair of this lane in an MMA tile
    const float sc = a.scale * 1.44269504088896341f;
    uint32_t qf[QP][NT][kKs][2];
    float o[kKs][NT][4];
    float m[NT][2], l[NT][2];
    bool fresh = true, begun = false;
    int stage = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const int4 mt = meta[warp][stage];
      if (fed < count) {
        feed(stage == 0 ? S - 1 : stage - 1);
        if (++fed < count) {
          in.next(a, HU);
          look_up();
        }
      }
      cp_async_commit();

      const int kh = mt.y / HT, h0 = mt.y % HT * kHeads;         // first head within the group
      if (fresh) {
        fresh = false;
        begun = mt.z >> 16 & 1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bool in_group = h0 + n * 8 + g < G;
          const X* qp = static_cast<const X*>(a.q) + mt.x * a.ldq +
                        static_cast<int64_t>(kh * G + h0 + n * 8 + g) * D;
#pragma unroll
          for (int k = 0; k < kKs; ++k) {
            // the four values of this lane in columns 16k.. of the head; the
            // order inside the sixteen follows that of the keys' registers
            float v[4] = {};
            if (in_group && k * 16 < D) {
              const int d0 = k * 16 + (BITS == 8 ? 4 * t4 : 2 * t4);
              const int d1 = BITS == 8 ? d0 + 2 : d0 + 8;
              if constexpr (sizeof(X) == 2) {
                const uint32_t u0 = *reinterpret_cast<const uint32_t*>(qp + d0);
                const uint32_t u1 = *reinterpret_cast<const uint32_t*>(qp + d1);
                v[0] = __uint_as_float(u0 << 16);
                v[1] = __uint_as_float(u0 & 0xffff0000u);
                v[2] = __uint_as_float(u1 << 16);
                v[3] = __uint_as_float(u1 & 0xffff0000u);
              } else {
                const float2 f0 = *reinterpret_cast<const float2*>(qp + d0);
                const float2 f1 = *reinterpret_cast<const float2*>(qp + d1);
                v[0] = f0.x;
                v[1] = f0.y;
                v[2] = f1.x;
                v[3] = f1.y;
              }
            }
            if constexpr (BITS == 8) {            // even values first, then odd ones
              const float x = v[1];
              v[1] = v[2];
              v[2] = x;
            }
#pragma unroll
            for (int p = 0; p < QP; ++p) {
              qf[p][n][k][0] = take2(v[0], v[1]);
              qf[p][n][k][1] = take2(v[2], v[3]);
            }
          }
          m[n][0] = m[n][1] = -INFINITY;
          l[n][0] = l[n][1] = 0.f;
#pragma unroll
          for (int k = 0; k < kKs; ++k) o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.f;
        }
      }

      const uint32_t kt = ring0 + stage * Sh::kStage, vt = kt + Sh::kTile;
      // S^T = K Q^T, two chains of sums
      float c[NT][4];
      auto scores = [&](auto parts) {
        float c2[2][NT][4] = {};
        if constexpr (BITS == 16) {
          const int row = lane & 15;
          const uint32_t base = kt + row * Sh::kRow;
#pragma unroll
          for (int k = 0; k < kKs; ++k) {
            uint32_t f[4];
            ldsm4(base + ((2 * k + (lane >> 4)) ^ (row & 7)) * 16, f);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < decltype(parts)::value; ++p)
                mma(c2[k & 1][n], f[0], f[1], f[2], f[3], qf[p][n][k][0], qf[p][n][k][1]);
          }
        } else {
          const int row = lane & 15;
          const uint32_t base = kt + row * Sh::kRow;
#pragma unroll
          for (int k = 0; k < kKs; k += 2) {
            const int chunk = k + (lane >> 4);
            const int phys = kChunks == 4 ? chunk ^ (row >> 1 & 3) : chunk ^ (row & 7);
            uint32_t f[4];
            ldsm4(base + phys * 16, f);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a0 = codes2(f[2 * j]), a1 = codes2(f[2 * j + 1]);
              const uint32_t a2 = codes2(f[2 * j] >> 8), a3 = codes2(f[2 * j + 1] >> 8);
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < decltype(parts)::value; ++p)
                  mma(c2[j][n], a0, a1, a2, a3, qf[p][n][k + j][0], qf[p][n][k + j][1]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) c[n][j] = c2[0][n][j] + c2[1][n][j];
      };
      scores(std::integral_constant<int, QP>());
      if constexpr (QP > 1) {
        // an infinite key times a part of q that is 0 is no number: there, q's
        // first part alone (which has its sign) gives the score
        bool nan = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) nan |= c[n][j] != c[n][j];
        if (__any_sync(0xffffffffu, nan)) {
          float whole[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) whole[n][j] = c[n][j];
          scores(std::integral_constant<int, 1>());
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (whole[n][j] == whole[n][j]) c[n][j] = whole[n][j];
        }
      }

      // scale, leave out rows that are not there
      float ks0 = sc, ks1 = sc, vs0 = 1.f, vs1 = 1.f;
      if constexpr (BITS == 8) {
        const float* sp = reinterpret_cast<const float*>(ring + (kt - smem_u32(ring)) + 2 * Sh::kTile);
        ks0 *= sp[g];
        ks1 *= sp[g + 8];
        vs0 = sp[16 + g];
        vs1 = sp[24 + g];
      }
      const bool in0 = mt.z >> g & 1, in1 = mt.z >> (g + 8) & 1;
      bool grew = false;
      float mn[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          c[n][j] = in0 ? c[n][j] * ks0 : -INFINITY;
          c[n][j + 2] = in1 ? c[n][j + 2] * ks1 : -INFINITY;
          float x = fmaxf(c[n][j], c[n][j + 2]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mn[n][j] = fmaxf(m[n][j], x);
          grew |= mn[n][j] > m[n][j];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float keep = weight(m[n][j], mn[n][j]);
            m[n][j] = mn[n][j];
            l[n][j] *= keep;
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
              o[k][n][j] *= keep;
              o[k][n][j + 2] *= keep;
            }
          }
      }
      uint32_t pf[QP][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float base = m[n][j] == -INFINITY ? 0.f : m[n][j];
          c[n][j] = exp2_fast(c[n][j] - base);
          c[n][j + 2] = exp2_fast(c[n][j + 2] - base);
          l[n][j] += c[n][j] + c[n][j + 2];
          if constexpr (BITS == 8) {
            c[n][j] *= vs0;
            c[n][j + 2] *= vs1;
          }
        }
        // tokens to the rows of the second product's right operand; bf16 q
        // rounds p to its own precision, fp32 q takes p whole
        if constexpr (QP == 1) {
          pf[0][n][0] = movm_t(pack2(c[n][0], c[n][1]));
          pf[0][n][1] = movm_t(pack2(c[n][2], c[n][3]));
        } else {
#pragma unroll
          for (int p = 0; p < QP; ++p) {
            pf[p][n][0] = movm_t(take2(c[n][0], c[n][1]));
            pf[p][n][1] = movm_t(take2(c[n][2], c[n][3]));
          }
        }
      }
      // O^T += V^T P^T
      if constexpr (BITS == 16) {
        // matrices: tokens 0-7 and 8-15 of values 0-7, then of values 8-15
        const int row = (lane & 7) + (lane >> 4 & 1) * 8;
        const uint32_t base = vt + row * Sh::kRow;
#pragma unroll
        for (int k = 0; k < kKs; ++k) {
          uint32_t f[4];
          ldsm4_t(base + ((2 * k + (lane >> 3 & 1)) ^ (row & 7)) * 16, f);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < QP; ++p) mma(o[k][n], f[0], f[1], f[2], f[3], pf[p][n][0], pf[p][n][1]);
        }
      } else {
        const int row = lane & 15;
        const uint32_t base = vt + row * Sh::kRow;
#pragma unroll
        for (int k = 0; k < kKs; k += 2) {
          const int chunk = k + (lane >> 4);
          const int phys = kChunks == 4 ? chunk ^ (row >> 1 & 3) : chunk ^ (row & 7);
          uint32_t f[4];
          ldsm4_t(base + phys * 16, f);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a0 = codes2(f[2 * j]), a1 = codes2(f[2 * j] >> 8);
            const uint32_t a2 = codes2(f[2 * j + 1]), a3 = codes2(f[2 * j + 1] >> 8);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < QP; ++p) mma(o[k + j][n], a0, a1, a2, a3, pf[p][n][0], pf[p][n][1]);
          }
        }
      }

      // ---- the unit, or this warp's piece of the line, ends here
      const bool ends = mt.z >> 17 & 1, last = i == count - 1;
      if (ends || last) {
        fresh = true;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            for (int d = 4; d < 32; d <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], d);
        if (last) {
          // every copy has landed and every lane has read its last tile: the
          // ring is free for the partial result
          cp_async_wait<0>();
          __syncwarp();
        }
        const bool whole = begun && ends;
        float* dst = last ? reinterpret_cast<float*>(ring + warp * S * Sh::kStage)
                          : ws.warp_o + (static_cast<size_t>(blockIdx.x) * W + warp) * kHeads * DP;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = n * 8 + 2 * t4 + j;
            const bool in_group = h0 + h < G;
            const int hq = kh * G + h0 + h;
            const float scale_o = whole ? (l[n][j] == 0.f ? 0.f : 1.f / l[n][j]) : 1.f;
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
              const int d0 = k * 16 + (BITS == 8 ? 2 * g : g), d1 = BITS == 8 ? d0 + 1 : d0 + 8;
              // an empty sum stays 0 whatever the values were
              const float v0 = whole && l[n][j] == 0.f ? 0.f : o[k][n][j] * scale_o;
              const float v1 = whole && l[n][j] == 0.f ? 0.f : o[k][n][j + 2] * scale_o;
              if (whole) {
                if (in_group && k * 16 < D) {
                  store_out<X>(a, mt.x, hq, d0, v0);
                  store_out<X>(a, mt.x, hq, d1, v1);
                }
              } else {
                dst[h * DP + d0] = v0;
                dst[h * DP + d1] = v1;
              }
            }
            if (g == 0) {
              if (whole) {
                if (a.lse && in_group) a.lse[static_cast<int64_t>(mt.x) * a.Hq + hq] = lse_of(m[n][j], l[n][j]);
              } else {
                slot_stat[warp][last][h] = make_float2(m[n][j], l[n][j]);
              }
            }
          }
        if (!whole && lane == 0) slot[warp][last] = make_int4(mt.x, mt.y, begun, ends);
      }
      stage = stage == S - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- join the CTA's partial results, unit by unit in the line's order
    const int4* sl = &slot[0][0];
    for (int i = 0; i < 2 * W;) {
      const int4 u = sl[i];
      if (u.x < 0) {
        ++i;
        continue;
      }
      int end = i, j = i + 1;
      for (; j < 2 * W; ++j) {
        if (sl[j].x < 0) continue;
        if (sl[j].x != u.x || sl[j].y != u.y) break;
        end = j;
      }
      const bool ends = sl[end].w, whole = u.z && ends;
      const int which = u.z ? 1 : 0;
      const int kh = u.y / HT, h0 = u.y % HT * kHeads;
      for (int x = threadIdx.x; x < kHeads * DP / 4; x += 32 * W) {
        const int h = x / (DP / 4), d = x % (DP / 4) * 4;
        float M = -INFINITY, L = 0.f;
        for (int k = i; k <= end; ++k)
          if (sl[k].x >= 0) M = fmaxf(M, slot_stat[k >> 1][k & 1][h].x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = i; k <= end; ++k) {
          if (sl[k].x < 0) continue;
          const float2 st = slot_stat[k >> 1][k & 1][h];
          const float w = weight(st.x, M);
          const float* src = (k & 1) ? reinterpret_cast<const float*>(ring + (k >> 1) * S * Sh::kStage)
                                     : ws.warp_o + (static_cast<size_t>(blockIdx.x) * W + (k >> 1)) * kHeads * DP;
          const float4 p = *reinterpret_cast<const float4*>(src + h * DP + d);
          L += st.y * w;
          // a part without weight adds nothing, whatever it holds
          if (st.x != -INFINITY || st.y != 0.f) {
            v.x += p.x * w;
            v.y += p.y * w;
            v.z += p.z * w;
            v.w += p.w * w;
          }
        }
        if (whole) {
          const float r = L == 0.f ? 0.f : 1.f / L;
          if (h0 + h < G && d < D)
            store_out4<X>(a, u.x, kh * G + h0 + h, d,
                          L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                   : make_float4(v.x * r, v.y * r, v.z * r, v.w * r));
          if (d == 0 && a.lse && h0 + h < G)
            a.lse[static_cast<int64_t>(u.x) * a.Hq + kh * G + h0 + h] = lse_of(M, L);
        } else {
          const size_t at = static_cast<size_t>(blockIdx.x) * 2 + which;
          *reinterpret_cast<float4*>(ws.o + (at * kHeads + h) * DP + d) = v;
          if (d == 0) ws.stat[at * kSlotHeads + h] = make_float2(M, L);
        }
      }
      if (u.z && !ends) {
        // begins here, ends in a later CTA: the one that holds the unit's last tile
        lead = make_int4(u.x, u.y, 0, 1);
      }
      i = j;
    }
    if (lead.w && threadIdx.x == 0) {
      // position of the unit's last tile on the line
      int64_t at = 0;
      for (int w = W - 1; w >= 0; --w) {
        // the last warp with work knows the tiles before its first sequence
        const int64_t wl = (static_cast<int64_t>(blockIdx.x) * W + w) * T / pieces;
        const int64_t wh = (static_cast<int64_t>(blockIdx.x) * W + w + 1) * T / pieces;
        if (wl < wh) {
          at = start_before[w];
          for (int b = start_b[w]; b < lead.x; ++b) at += (span_of(a, b).visible + 15) / 16;
          break;
        }
      }
      const int64_t tiles = (span_of(a, lead.x).visible + 15) / 16;
      const int64_t x = at * HU + (static_cast<int64_t>(lead.y) + 1) * tiles - 1;
      lead.z = static_cast<int>(((x + 1) * ctas - 1) / T);
    }
  }
  if (threadIdx.x == 0) ws.leader[blockIdx.x] = lead;

  // ---- sequences without tokens
  for (int b = blockIdx.x + gridDim.x * warp; b < a.B; b += gridDim.x * W) {
    if (span_of(a, b).visible) continue;
    if (lane == 0 && !good_len(a, a.seq_lens[b])) report(err, QVLA_DEVERR_CACHE_RANGE);
    for (int x = lane * 4; x < a.Hq * D; x += 128)
      store_out4<X>(a, b, 0, x, make_float4(0.f, 0.f, 0.f, 0.f));
    if (a.lse)
      for (int h = lane; h < a.Hq; h += 32) a.lse[static_cast<int64_t>(b) * a.Hq + h] = -INFINITY;
  }
}

// Joins the units that span CTAs: a block per (CTA, head) whose CTA began such
// a unit.  Its parts are that CTA's slot 1 and the following CTAs' slot 0.
template <typename X, int DP, int NT>
__global__ void __launch_bounds__(128) paged_attn_join_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int kHeads = 8 * NT, kLanes = DP / 4, kSplit = 128 / kLanes;
  __shared__ float w[kMaxCtas + 1];
  __shared__ float red[2][4];
  __shared__ float4 acc[kSplit][kLanes];
  pdl_wait();
  const Scratch ws = scratch_at<kHeads, DP>(a.ws);
  const int4 lead = ws.leader[blockIdx.x];
  if (!lead.w) return;
  const int h = blockIdx.y, D = a.cache.dim, G = a.Hq / a.cache.heads;
  const int HT = (G + kHeads - 1) / kHeads;
  const int kh = lead.y / HT, hg = lead.y % HT * kHeads + h;
  if (hg >= G) return;
  const int parts = lead.z - blockIdx.x + 1;
  auto at = [&](int i) -> size_t {
    return i == 0 ? static_cast<size_t>(blockIdx.x) * 2 + 1 : static_cast<size_t>(blockIdx.x + i) * 2;
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float M = -INFINITY, L = 0.f;
  for (int i = threadIdx.x; i < parts; i += 128) M = fmaxf(M, ws.stat[at(i) * kSlotHeads + h].x);
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  for (int i = threadIdx.x; i < parts; i += 128) {
    const float2 st = ws.stat[at(i) * kSlotHeads + h];
    const float x = weight(st.x, M);
    // a part without weight is left out (marked by a negative factor)
    w[i] = st.x == -INFINITY && st.y == 0.f ? -1.f : x;
    L += st.y * x;
  }
  for (int d = 16; d; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
  if (lane == 0) red[1][warp] = L;
  __syncthreads();
  L = red[1][0] + red[1][1] + red[1][2] + red[1][3];
  const int d4 = threadIdx.x % kLanes, part0 = threadIdx.x / kLanes;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = part0; i < parts; i += kSplit) {
    const float x = w[i];
    const float4 p = *reinterpret_cast<const float4*>(ws.o + (at(i) * kHeads + h) * DP + d4 * 4);
    if (!(x < 0.f)) {
      v.x += p.x * x;
      v.y += p.y * x;
      v.z += p.z * x;
      v.w += p.w * x;
    }
  }
  acc[part0][d4] = v;
  __syncthreads();
  if (part0 == 0) {
    for (int i = 1; i < kSplit; ++i) {
      const float4 p = acc[i][d4];
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
    const int hq = kh * G + hg;
    const float r = L == 0.f ? 0.f : 1.f / L;
    if (d4 * 4 < D)
      store_out4<X>(a, lead.x, hq, d4 * 4,
                    L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                             : make_float4(v.x * r, v.y * r, v.z * r, v.w * r));
    if (d4 == 0 && a.lse) a.lse[static_cast<int64_t>(lead.x) * a.Hq + hq] = lse_of(M, L);
  }
}

template <typename... A>
cudaError_t launch_pdl(void (*kernel)(A...), dim3 grid, int block, size_t smem, cudaStream_t stream,
                       A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs of the split: one per SM.
int split_ctas() {
  static std::atomic<int> sms[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = sms[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  n = std::min(n, kMaxCtas);
  if (dev < 64) sms[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <typename X, int DP, int NT, int BITS, int W, int S>
cudaError_t run(const PagedAttnArgs& a, cudaStream_t stream) {
  constexpr int QP = sizeof(X) == 2 ? 1 : 3;
  using Sh = Shape<DP, NT, QP, BITS, W, S>;
  auto kernel = paged_attn_kernel<X, DP, NT, QP, BITS, W, S>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  });
  if (e != cudaSuccess) return e;
  unsigned int* err = device_error_word();
  const int ctas = split_ctas();
  if (!err || ctas == 0) return cudaErrorUnknown;
  e = launch_pdl(kernel, dim3(ctas), 32 * W, Sh::kSmem, stream, a, err);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_attn_join_kernel<X, DP, NT>, dim3(ctas, 8 * NT), 128, 0, stream, a);
}

// Warps and stages: the rings of all warps take most of the SM's shared
// memory, so that two tiles of every warp are on the way (at least 128 KB).
template <typename X, int NT>
cudaError_t run_dim(const PagedAttnArgs& a, cudaStream_t stream) {
  const int D = a.cache.dim;
  if (a.cache.bits == 16) {
    if (D <= 64) return run<X, 64, NT, 16, 16, 3>(a, stream);
    if (D <= 128) return run<X, 128, NT, 16, 8, 3>(a, stream);
    return run<X, 256, NT, 16, 4, 3>(a, stream);
  }
  if (D <= 64) return run<X, 64, NT, 8, 16, 4>(a, stream);
  if (D <= 128) return run<X, 128, NT, 8, 16, 3>(a, stream);
  return run<X, 256, NT, 8, 8, 3>(a, stream);
}

// 16 heads a unit when the group has more than 8, unless their registers do
// not fit (fp32 q in three parts at the largest head dim).
bool two_columns(int G, int D, bool f32) { return G > 8 && !(f32 && D > 128); }

}  // namespace

size_t paged_attn_ws_bytes(int Hq, int heads, int dim) {
  const size_t dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  const size_t h = Hq / heads > 8 ? 16 : 8, warps = 16;
  return scratch_head_bytes() + static_cast<size_t>(kMaxCtas) * (2 + warps) * h * dp * sizeof(float);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  const bool f32 = a.qdt == QVLA_DTYPE_F32;
  if (two_columns(a.Hq / a.cache.heads, a.cache.dim, f32))
    return f32 ? run_dim<float, 2>(a, stream) : run_dim<__nv_bfloat16, 2>(a, stream);
  return f32 ? run_dim<float, 1>(a, stream) : run_dim<__nv_bfloat16, 1>(a, stream);
}

}  // namespace qvla
