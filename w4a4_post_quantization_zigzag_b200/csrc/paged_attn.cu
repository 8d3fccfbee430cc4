// Attention of one new token per sequence over a paged key/value cache.
//
//   o = sum_t p_t v_t,  p = softmax over the visible t of scale * q . k_t
//
// Bound by reading the cache once: a key head's rows serve the query heads of
// its group, which are the columns of two small matrix products per 16 tokens,
//   S^T [16 tokens x heads] = K [16 x D] Q^T [D x heads]
//   O^T [D x heads]        += V^T [D x 16] P^T [16 x heads]
// with tokens (then head values) in the rows of the warp-level MMA, so that a
// group of 8 heads fills its columns.  A larger group has 16 columns (fp32 q at
// head dims above 128: 8), and one of more heads than that reads the cache once
// for every 16 (8) of them.  The running maximum and sum of the softmax are per
// column; the output stays in registers.
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
//
// One sequence of 131072 tokens, 32 over 8 heads of 128: 93.5 us, 5.7 TB/s (87 %
// of the copy rate); 32 sequences of up to 8192: 93.4 us (86 %).  With little to
// read the time is a chain of waits (lengths, page numbers, first tiles, the
// join, the second launch): 12.5 us at 1040 tokens and 8 over 1 heads of 256.  An
// 8-bit cache is bound by the instructions that expand its codes: 64 sequences
// of up to 2000 tokens, 32 over 8 heads of 128, take 55 us in 8 bits and 59 in
// bf16 (floors of 21 and 41); with fp32 q, in three parts, 62 and 63.  64 that
// see 2000 tokens of a window in 8 bits, 16 over 2 heads of 64 in fp32: 28.7 us
// for 5 of bytes, 10 of them instructions.
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
// What is left of a probability p after its first part, as a part of its own: never 0
// unless p is, for an infinite value times a part that is 0 is no number.  The
// least it is raised to, 2^-30 p, shows in no sum of fp32; nor does 2^-126, below
// which the exponential is 0.
QVLA_DEVICE float some_left(float left, float p) {
  return fmaxf(left, fminf(p, fmaxf(p * 9.31322575e-10f, 1.17549435e-38f)));
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

// The line's length T cut into equal pieces, one per warp of as many CTAs as
// there is length for: the first `more` pieces have length each + 1.
struct Cut {
  int ctas;
  int64_t each, more;
  int warps;
  QVLA_DEVICE Cut(int64_t T, int W) : warps(W) {
    ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (T + 2 * W - 1) / (2 * W)));
    const int pieces = max(ctas, 1) * W;
    each = T < (1ll << 31) ? static_cast<int>(T) / pieces : T / pieces;
    more = T - each * pieces;
  }
  QVLA_DEVICE int64_t start(int piece) const { return each * piece + min(static_cast<int64_t>(piece), more); }
  // the CTA whose pieces hold place x
  QVLA_DEVICE int owner(int64_t x) const {
    const int64_t big = more * (each + 1);
    const int64_t piece = x < big ? x / (each + 1) : more + (x - big) / each;
    return static_cast<int>(piece / warps);
  }
};

struct Cursor {
  int b, hu, tile, tiles;
  Span s;
  template <int TK>
  QVLA_DEVICE void seek(const PagedAttnArgs& a) {      // first sequence from b on with tokens
    for (; b < a.B; ++b) {
      s = span_of(a, b);
      tiles = (s.visible + TK - 1) / TK;
      if (tiles) return;
    }
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
// (1 for bf16 q, 3 for fp32: their sum is the whole value; p has two parts and
// three); BITS of the cache; W warps, S stages of one tile of TK tokens per warp.
template <int DP, int NT, int QP, int BITS, int W, int S, int TK>
struct Shape {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kRow = DP * BITS / 8;               // bytes of a token's row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kTile = TK * kRow;
  static constexpr int kStage = 2 * kTile + (BITS == 8 ? 8 * TK : 0);
  static constexpr int kSmem = W * S * kStage;
  static_assert(S * kStage >= kHeads * DP * 4, "a warp's ring holds its last partial result");
  static_assert(2 * W <= 32, "a lane for every partial result of a CTA");
};

// 16-byte piece of a row in its tile: eight rows of one piece meet no bank twice.
template <int kChunks>
QVLA_DEVICE int piece_at(int row, int piece) {
  return kChunks == 4 ? piece ^ (row >> 1 & 3) : piece ^ (row & 7);
}

template <typename X, int DP, int NT, int QP, int BITS, int W, int S, int TK>
__global__ void __launch_bounds__(32 * W, 1)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, unsigned int* err) {
  using Sh = Shape<DP, NT, QP, BITS, W, S, TK>;
  constexpr int kHeads = Sh::kHeads, kChunks = Sh::kChunks, kKs = DP / 16, kSub = TK / 16;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int4 meta[W][S];                 // {b, unit head, rows that are there, flags} of each stage
  __shared__ int64_t scan[W];
  __shared__ int64_t start_before[W];         // length of a head's line before the sequence
  __shared__ int start_b[W];
  __shared__ int4 slot[2 * W];                // partial results {b (-1: none), unit head, begins, ends}
  __shared__ float2 slot_stat[2 * W][kHeads];
  __shared__ float slot_weight[2 * W][kHeads];
  __shared__ float2 unit_stat[2 * W][kHeads];
  enum { kBegins = 1, kEnds = 2, kLast = 4 };

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.cache.dim, G = a.Hq / a.cache.heads;
  const int HT = (G + kHeads - 1) / kHeads, HU = a.cache.heads * HT;
  const Scratch ws = scratch_at<kHeads, DP>(a.ws);
  if (threadIdx.x < 2 * W) slot[threadIdx.x] = make_int4(-1, 0, 0, 0);
  pdl_launch_dependents();
  pdl_wait();

  // ---- the line: its length for one head before each thread's share of
  // sequences.  A sequence takes a place per tile and one for its beginning
  // (the query, the end of the unit before), which costs about as much.
  auto length = [&](int b) {
    const int n = (span_of(a, b).visible + TK - 1) / TK;
    return n ? n + 1 : 0;
  };
  const int per = (a.B + 32 * W - 1) / (32 * W);
  const int b_lo = min(static_cast<int>(threadIdx.x) * per, a.B), b_hi = min(b_lo + per, a.B);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += length(b);
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
  const Cut cut(all * HU, W);
  const bool works = static_cast<int>(blockIdx.x) < cut.ctas;
  if (works) {
    for (int w = 0; w < W; ++w) {
      const int64_t x = cut.start(blockIdx.x * W + w);
      if (x >= before * HU && x < (before + mine) * HU) {
        int64_t at = before;
        int b = b_lo;
        for (;; ++b) {
          const int n = length(b);
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
    const int64_t lo = cut.start(blockIdx.x * W + warp);
    int64_t left = cut.start(blockIdx.x * W + warp + 1) - lo;        // places of this piece not fed yet
    const uint32_t ring0 = smem_u32(ring) + warp * S * Sh::kStage;

    Cursor in = {};
    if (left > 0) {
      in.b = start_b[warp];
      in.s = span_of(a, in.b);
      in.tiles = (in.s.visible + TK - 1) / TK;
      const int64_t off = lo - start_before[warp] * HU;
      const int len = in.tiles + 1;
      in.hu = off < (1ll << 31) ? static_cast<int>(off) / len : static_cast<int>(off / len);
      const int r = static_cast<int>(off - static_cast<int64_t>(in.hu) * len);
      in.tile = max(r - 1, 0);
      if (r == 0) --left;
    }

    // ---- feeding.  Two tiles' page numbers are read ahead of the copies.
    struct Row {
      bool valid, in;          // a tile; a row of it for this lane
      int b, hu, flags, page, tok;
    };
    auto look_up = [&]() -> Row {
      Row r = {};
      if (left <= 0) return r;
      r.valid = true;
      r.b = in.b;
      r.hu = in.hu;
      r.flags = (in.tile == 0 ? kBegins : 0) | (in.tile == in.tiles - 1 ? kEnds : 0);
      const int v = in.tile * TK + (lane & (TK - 1));
      r.in = v < in.s.visible;
      if (r.in) {
        const int t = v >= a.sinks ? v + in.s.gap : v;
        const int p = t / a.cache.page_size;
        r.tok = t - p * a.cache.page_size;
        r.page = a.page_table[static_cast<int64_t>(in.b) * a.max_pages + p];
      }
      --left;
      if (++in.tile == in.tiles) {
        in.tile = 0;
        --left;                // the next unit's beginning
        if (++in.hu == HU) {
          in.hu = 0;
          ++in.b;
          if (left > 0) in.template seek<TK>(a);
        }
      }
      if (left <= 0) r.flags |= kLast;
      return r;
    };
    auto feed = [&](const Row& r, int stage) {
      const bool found = r.page >= 0 && r.page < a.cache.pages;
      if (r.in && !found && lane < TK) report(err, QVLA_DEVERR_CACHE_RANGE);
      const bool ok = r.in && found;
      const uint32_t mask = __ballot_sync(0xffffffffu, ok);
      const int kh = r.hu / HT;
      const int64_t off = ok ? r.page * a.cache.page_stride + r.tok * a.cache.token_stride +
                                   kh * a.cache.head_stride
                             : 0;
      const uint32_t dst0 = ring0 + stage * Sh::kStage;
      const int piece = lane % kChunks;
      const bool col = piece * (128 / BITS) < D;
#pragma unroll
      for (int i = 0; i < kChunks * TK / 32; ++i) {
        const int row = i * (32 / kChunks) + lane / kChunks;
        const int64_t ro = __shfl_sync(0xffffffffu, off, row) * (BITS / 8) + piece * 16;
        const bool take = col && (mask >> row & 1);
        const uint32_t dst = dst0 + row * Sh::kRow + piece_at<kChunks>(row, piece) * 16;
        cp_async16(dst, static_cast<const uint8_t*>(a.cache.k) + (take ? ro : 0), take);
        cp_async16(dst + Sh::kTile, static_cast<const uint8_t*>(a.cache.v) + (take ? ro : 0), take);
      }
      if constexpr (BITS == 8) {
        const int64_t so = ok ? r.page * a.cache.s_page_stride + r.tok * a.cache.s_token_stride +
                                    kh * a.cache.s_head_stride
                              : 0;
        const uint32_t to = dst0 + 2 * Sh::kTile + lane * 4;
        if constexpr (TK == 32) {
          cp_async4(to, a.cache.k_scale + so, ok);
          cp_async4(to + 128, a.cache.v_scale + so, ok);
        } else {
          cp_async4(to, (lane < 16 ? a.cache.k_scale : a.cache.v_scale) + so, ok);
        }
      }
      if (lane == 0) meta[warp][stage] = make_int4(r.b, r.hu, static_cast<int>(mask), r.flags);
    };

    int fed = 0;
    Row now = look_up(), then = look_up();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) {
      if (now.valid) {
        feed(now, s);
        ++fed;
        now = then;
        then = look_up();
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
    for (int i = 0; i < fed; ++i) {
      __syncwarp();
      const int4 mt = meta[warp][stage];
      const int kh = mt.y / HT, h0 = mt.y % HT * kHeads;         // first head within the group
      if (fresh) {
        // the columns of Q^T of the unit, in registers, while its first tile comes
        fresh = false;
        begun = mt.w & kBegins;
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
                // a NaN whose bits are all below its first part would become infinite there
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = v[j] == v[j] ? v[j] : __uint_as_float(0x7fc00000u);
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
      cp_async_wait<S - 2>();
      __syncwarp();
      if (now.valid) {
        feed(now, stage == 0 ? S - 1 : stage - 1);
        ++fed;
        now = then;
        then = look_up();
      }
      cp_async_commit();

      const uint32_t kt = ring0 + stage * Sh::kStage, vt = kt + Sh::kTile;
      const int row = lane & 15;
      // S^T = K Q^T, two chains of sums; fp32 q: a third for the parts below its
      // first (the MMA cuts its sums, which costs least where they are small)
      float c[kSub][NT][4];
      auto scores = [&](auto parts) {
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          float c2[QP > 1 ? 3 : 2][NT][4] = {};
          const uint32_t base = kt + (u * 16 + row) * Sh::kRow;
          if constexpr (BITS == 16) {
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
              uint32_t f[4];
              ldsm4(base + piece_at<kChunks>(row, 2 * k + (lane >> 4)) * 16, f);
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < decltype(parts)::value; ++p)
                  mma(c2[p > 0 ? 2 : k & 1][n], f[0], f[1], f[2], f[3], qf[p][n][k][0], qf[p][n][k][1]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < kKs; k += 2) {
              uint32_t f[4];
              ldsm4(base + piece_at<kChunks>(row, k + (lane >> 4)) * 16, f);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t a0 = codes2(f[2 * j]), a1 = codes2(f[2 * j + 1]);
                const uint32_t a2 = codes2(f[2 * j] >> 8), a3 = codes2(f[2 * j + 1] >> 8);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int p = 0; p < decltype(parts)::value; ++p)
                    mma(c2[p > 0 ? 2 : j][n], a0, a1, a2, a3, qf[p][n][k + j][0], qf[p][n][k + j][1]);
              }
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              c[u][n][j] = c2[0][n][j] + c2[1][n][j];
              if constexpr (QP > 1) c[u][n][j] += c2[2][n][j];
            }
        }
      };
      scores(std::integral_constant<int, QP>());
      if constexpr (QP > 1) {
        // an infinite key times a part of q that is 0 is no number: there, q's
        // first part alone (which has its sign) gives the score
        bool nan = false;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) nan |= c[u][n][j] != c[u][n][j];
        if (__any_sync(0xffffffffu, nan)) {
          float whole[kSub][NT][4];
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) whole[u][n][j] = c[u][n][j];
          scores(std::integral_constant<int, 1>());
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (whole[u][n][j] == whole[u][n][j]) c[u][n][j] = whole[u][n][j];
        }
      }

      // scale, leave out rows that are not there
      float vs[kSub][2];
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float ks = sc;
          const int at = u * 16 + g + 8 * r;
          if constexpr (BITS == 8) {
            const float* sp = reinterpret_cast<const float*>(ring + (kt - smem_u32(ring)) + 2 * Sh::kTile);
            ks *= sp[at];
            vs[u][r] = sp[TK + at];
          }
          const bool there = mt.z >> at & 1;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) c[u][n][2 * r + j] = there ? c[u][n][2 * r + j] * ks : -INFINITY;
        }
      bool grew = false;
      float mn[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(c[0][n][j], c[0][n][j + 2]);
          if constexpr (kSub > 1) x = fmaxf(x, fmaxf(c[kSub - 1][n][j], c[kSub - 1][n][j + 2]));
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
      constexpr int kParts = QP > 1 ? QP : 2;
      uint32_t pf[kSub][kParts][NT][2];
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* x = c[u][n];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float base = m[n][j] == -INFINITY ? 0.f : m[n][j];
            x[j] = exp2_fast(x[j] - base);
            x[j + 2] = exp2_fast(x[j + 2] - base);
            l[n][j] += x[j] + x[j + 2];
            if constexpr (BITS == 8) {
              x[j] *= vs[u][0];
              x[j + 2] *= vs[u][1];
            }
          }
          // tokens to the rows of the second product's right operand; bf16 q takes
          // p in two parts, 2^-15 of it off at most, fp32 q takes p whole
          if constexpr (QP == 1) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = x[j];
            pf[u][0][n][0] = movm_t(take2(x[0], x[1]));
            pf[u][0][n][1] = movm_t(take2(x[2], x[3]));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // 8 bits: values are finite but for their scale, whose infinity the first part holds
              if constexpr (BITS == 16)
                x[j] = some_left(x[j], p[j]);
              else if (x[j] != x[j])
                x[j] = 0.f;
            }
            pf[u][1][n][0] = movm_t(pack2(x[0], x[1]));
            pf[u][1][n][1] = movm_t(pack2(x[2], x[3]));
          } else {
#pragma unroll
            for (int p = 0; p < QP; ++p) {
              pf[u][p][n][0] = movm_t(take2(x[0], x[1]));
              pf[u][p][n][1] = movm_t(take2(x[2], x[3]));
            }
          }
        }
      // O^T += V^T P^T.  fp32 q: a tile's sums are formed from zero, its first
      // parts apart from the rest, and added to the output by fp32 additions,
      // which round where the MMA cuts.  bf16 q: four sums take their first part
      // before any takes its second, which would wait for it (16 sequences of up
      // to 4000 tokens, 16 over 1 heads of 256: 26.0 against 30.1 us one by one).
      auto add = [&](int k, int u, int p, const uint32_t (&f)[4], float (&tile)[2][NT][4]) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma(QP == 1 ? o[k][n] : tile[p > 0][n], f[0], f[1], f[2], f[3], pf[u][p][n][0], pf[u][p][n][1]);
      };
      auto settle = [&](int k, const float (&tile)[2][NT][4]) {
        if constexpr (QP > 1) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // an infinite value times a part that is 0 is no number: the first
              // parts, which are 0 only where p is, have the infinity
              const float rest = tile[1][n][j];
              o[k][n][j] += tile[0][n][j] + (rest == rest ? rest : 0.f);
            }
        }
      };
      constexpr int kStep = BITS == 8 ? 2 : QP == 1 ? 4 : 1;
#pragma unroll
      for (int k = 0; k < kKs; k += kStep) {
        float tile[kStep][2][NT][4] = {};
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          uint32_t f[kStep][4];
          if constexpr (BITS == 16) {
            // matrices: tokens 0-7 and 8-15 of values 0-7, then of values 8-15
            const int vrow = (lane & 7) + (lane >> 4 & 1) * 8;
#pragma unroll
            for (int j = 0; j < kStep; ++j)
              ldsm4_t(vt + (u * 16 + vrow) * Sh::kRow + piece_at<kChunks>(vrow, 2 * (k + j) + (lane >> 3 & 1)) * 16, f[j]);
          } else {
            uint32_t c[4];
            ldsm4_t(vt + (u * 16 + row) * Sh::kRow + piece_at<kChunks>(row, k + (lane >> 4)) * 16, c);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              f[j][0] = codes2(c[2 * j]), f[j][1] = codes2(c[2 * j] >> 8);
              f[j][2] = codes2(c[2 * j + 1]), f[j][3] = codes2(c[2 * j + 1] >> 8);
            }
          }
#pragma unroll
          for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int j = 0; j < kStep; ++j) add(k + j, u, p, f[j], tile[j]);
        }
#pragma unroll
        for (int j = 0; j < kStep; ++j) settle(k + j, tile[j]);
      }

      // ---- the unit, or this warp's piece of the line, ends here
      const bool ends = mt.w & kEnds, last = mt.w & kLast;
      if (ends || last) {
        fresh = true;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            for (int d = 4; d < 32; d <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], d);
        if (begun && ends && !last) {
          // the whole unit was this warp's: its result, from the registers
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int h = h0 + n * 8 + 2 * t4 + j;
              if (h >= G) continue;
              const bool none = l[n][j] == 0.f;            // an empty sum stays 0 whatever the values were
              const float r = none ? 0.f : 1.f / l[n][j];
              X* to = static_cast<X*>(a.out) + mt.x * a.ldo + static_cast<int64_t>(kh * G + h) * D +
                      (BITS == 8 ? 2 * g : g);
#pragma unroll
              for (int k = 0; k < kKs; ++k) {
                const float v0 = none ? 0.f : o[k][n][j] * r, v1 = none ? 0.f : o[k][n][j + 2] * r;
                if (k * 16 >= D) continue;
                if constexpr (sizeof(X) == 2) {
                  to[k * 16] = __float2bfloat16_rn(v0);
                  to[k * 16 + (BITS == 8 ? 1 : 8)] = __float2bfloat16_rn(v1);
                } else {
                  to[k * 16] = v0;
                  to[k * 16 + (BITS == 8 ? 1 : 8)] = v1;
                }
              }
              if (a.lse && g == 0) a.lse[static_cast<int64_t>(mt.x) * a.Hq + kh * G + h] = lse_of(m[n][j], l[n][j]);
            }
        } else {
          // a part: in the warp's ring after its last tile (every copy has
          // landed, every lane has read), else in its place in the scratch
          __syncwarp();
          float* to = (last ? reinterpret_cast<float*>(ring + warp * S * Sh::kStage)
                            : ws.warp_o + (static_cast<size_t>(blockIdx.x) * W + warp) * kHeads * DP) +
                      2 * t4 * DP + (BITS == 8 ? 2 * g : g);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
              for (int k = 0; k < kKs; ++k) {
                to[(n * 8 + j) * DP + k * 16] = o[k][n][j];
                to[(n * 8 + j) * DP + k * 16 + (BITS == 8 ? 1 : 8)] = o[k][n][j + 2];
              }
              if (g == 0) slot_stat[2 * warp + last][n * 8 + 2 * t4 + j] = make_float2(m[n][j], l[n][j]);
            }
          if (lane == 0) slot[2 * warp + last] = make_int4(mt.x, mt.y, begun, ends);
        }
      }
      stage = stage == S - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- join the CTA's parts, in the line's order.  Parts of one unit are
    // neighbours: lane k of every warp holds part k, a warp takes some heads.
    const int4 part = lane < 2 * W ? slot[lane] : make_int4(-1, 0, 0, 0);
    const uint32_t valid = __ballot_sync(0xffffffffu, part.x >= 0);
    const uint32_t below = valid & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : lane;
    const int prev_b = __shfl_sync(0xffffffffu, part.x, prev), prev_hu = __shfl_sync(0xffffffffu, part.y, prev);
    const uint32_t firsts =
        __ballot_sync(0xffffffffu, part.x >= 0 && !(below && prev_b == part.x && prev_hu == part.y));
    const uint32_t upto_here = firsts & (0xffffffffu >> (31 - lane)), after_here = firsts & ~(0xffffffffu >> (31 - lane));
    const int first = upto_here ? 31 - __clz(upto_here) : 0;       // this lane's group of parts
    const int end = after_here ? __ffs(after_here) - 2 : 31;
    for (int h = warp; h < kHeads; h += W) {
      const float2 st = part.x >= 0 ? slot_stat[lane][h] : make_float2(-INFINITY, 0.f);
      float M = st.x;
      for (int d = 1; d < 32; d <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, M, d);
        if (lane - d >= first) M = fmaxf(M, v);
      }
      M = __shfl_sync(0xffffffffu, M, end);
      const float w = weight(st.x, M);
      float L = st.y * w;
      for (int d = 1; d < 32; d <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, L, d);
        if (lane - d >= first) L += v;
      }
      L = __shfl_sync(0xffffffffu, L, end);
      if (part.x >= 0) {
        // a part without weight is left out, whatever it holds (marked by -1)
        slot_weight[lane][h] = st.x == -INFINITY && st.y == 0.f ? -1.f : w;
        unit_stat[lane][h] = make_float2(M, L);
      }
    }
    __syncthreads();
    // A thread's places of the output; the values of four parts, or of four
    // places of one, asked for at once (one after the other: 13.4 against 12.1
    // us at 1040 tokens and 8 over 1 heads of 256).
    constexpr int kPlaces = kHeads * DP / 4, kItems = (kPlaces + 32 * W - 1) / (32 * W);
    constexpr int kAhead = kItems < 4 ? 4 / kItems : 1;
    static_assert(kItems == 1 || kPlaces % (32 * W) == 0, "every thread has all its places or none");
    float4 v[kItems];
    int begins = 0;
#pragma unroll 1
    for (uint32_t rest = static_cast<int>(threadIdx.x) < kPlaces ? valid : 0u; rest;) {
      float4 p[kAhead][kItems];
      float w[kAhead][kItems];
      uint32_t ask = rest;
#pragma unroll
      for (int b = 0; b < kAhead; ++b, ask &= ask - 1) {
        if (!ask) break;
        const int k = __ffs(ask) - 1;
        const float* src = (k & 1) ? reinterpret_cast<const float*>(ring + (k >> 1) * S * Sh::kStage)
                                   : ws.warp_o + (static_cast<size_t>(blockIdx.x) * W + (k >> 1)) * kHeads * DP;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int x = threadIdx.x + i * 32 * W;
          p[b][i] = *reinterpret_cast<const float4*>(src + x * 4);
          w[b][i] = slot_weight[k][x / (DP / 4)];
        }
      }
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        if (!rest) break;
        const int k = __ffs(rest) - 1;
        if (firsts >> k & 1) {
          begins = slot[k].z;
#pragma unroll
          for (int i = 0; i < kItems; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if (!(w[b][i] < 0.f)) {
            v[i].x += p[b][i].x * w[b][i];
            v[i].y += p[b][i].y * w[b][i];
            v[i].z += p[b][i].z * w[b][i];
            v[i].w += p[b][i].w * w[b][i];
          }
        const uint32_t later = rest &= rest - 1;
        if (later && !(firsts & later & (0u - later))) continue;       // the group goes on
        const int4 u = slot[k];
        const int kh = u.y / HT, h0 = u.y % HT * kHeads;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int x = threadIdx.x + i * 32 * W, h = x / (DP / 4), d = x % (DP / 4) * 4, hg = h0 + h;
          const float2 st = unit_stat[k][h];
          if (begins && u.w) {
            const float r = st.y == 0.f ? 0.f : 1.f / st.y;
            if (hg < G && d < D)
              store_out4<X>(a, u.x, kh * G + hg, d,
                            st.y == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                        : make_float4(v[i].x * r, v[i].y * r, v[i].z * r, v[i].w * r));
            if (d == 0 && a.lse && hg < G) a.lse[static_cast<int64_t>(u.x) * a.Hq + kh * G + hg] = lse_of(st.x, st.y);
          } else {
            // its beginning (slot 1) or a later part (slot 0) of a unit that goes on in other CTAs
            const size_t at = static_cast<size_t>(blockIdx.x) * 2 + (begins ? 1 : 0);
            *reinterpret_cast<float4*>(ws.o + (at * kHeads + h) * DP + d) = v[i];
            if (d == 0) ws.stat[at * kSlotHeads + h] = st;
          }
        }
      }
    }
    if (threadIdx.x == 0 && valid) {
      const int4 u = slot[31 - __clz(valid)];
      if (slot[31 - __clz(firsts)].z && !u.w) {
        // begins here, ends in a later CTA: the one that holds the unit's last
        // tile.  The last warp with work knows the line before its sequence.
        int w = W - 1;
        while (cut.start(blockIdx.x * W + w) == cut.start(blockIdx.x * W + w + 1)) --w;
        int64_t at = start_before[w];
        for (int b = start_b[w]; b < u.x; ++b) at += length(b);
        lead = make_int4(u.x, u.y, cut.owner(at * HU + (static_cast<int64_t>(u.y) + 1) * length(u.x) - 1), 1);
      }
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
  // the statistics of all CTAs that may follow are asked for with the leader's
  // word, which says how many do
  const int h = blockIdx.y, D = a.cache.dim, G = a.Hq / a.cache.heads;
  auto at = [&](int i) -> size_t {
    return i == 0 ? static_cast<size_t>(blockIdx.x) * 2 + 1 : static_cast<size_t>(blockIdx.x + i) * 2;
  };
  const int after = gridDim.x - blockIdx.x;
  const int4 lead = ws.leader[blockIdx.x];
  float2 st[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + 128 * j;
    st[j] = i < after ? ws.stat[at(i) * kSlotHeads + h] : make_float2(-INFINITY, 0.f);
  }
  if (!lead.w) return;
  const int HT = (G + kHeads - 1) / kHeads;
  const int kh = lead.y / HT, hg = lead.y % HT * kHeads + h;
  if (hg >= G) return;
  const int parts = lead.z - blockIdx.x + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (threadIdx.x + 128 * j < parts) M = fmaxf(M, st[j].x);
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + 128 * j;
    if (i >= parts) continue;
    const float x = weight(st[j].x, M);
    // a part without weight is left out (marked by a negative factor)
    w[i] = st[j].x == -INFINITY && st[j].y == 0.f ? -1.f : x;
    L += st[j].y * x;
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

template <typename X, int DP, int NT, int BITS, int W, int S, int TK>
cudaError_t run(const PagedAttnArgs& a, cudaStream_t stream) {
  constexpr int QP = sizeof(X) == 2 ? 1 : 3;
  using Sh = Shape<DP, NT, QP, BITS, W, S, TK>;
  auto kernel = paged_attn_kernel<X, DP, NT, QP, BITS, W, S, TK>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [&] {
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    // the same split of an SM's memory for both kernels: changing it between
    // them would wait for the SM to drain
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(paged_attn_join_kernel<X, DP, NT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    return r;
  });
  if (e != cudaSuccess) return e;
  unsigned int* err = device_error_word();
  const int ctas = split_ctas();
  if (!err || ctas == 0) return cudaErrorUnknown;
  e = launch_pdl(kernel, dim3(ctas), 32 * W, Sh::kSmem, stream, a, err);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_attn_join_kernel<X, DP, NT>, dim3(ctas, 8 * NT), 128, 0, stream, a);
}

// Warps, stages and tokens of a tile: the rings of all warps take most of the
// SM's shared memory, so that two tiles of every warp are on the way (at least
// 128 KB); short rows come 32 to a tile.
template <typename X, int NT>
cudaError_t run_dim(const PagedAttnArgs& a, cudaStream_t stream) {
  const int D = a.cache.dim;
  // fp32 q in three parts at the largest head dim: 16 heads do not fit registers
  constexpr int kNT = sizeof(X) == 4 ? 1 : NT;
  if (a.cache.bits == 16) {
    if (D <= 64) return run<X, 64, NT, 16, 8, 3, 32>(a, stream);
    if (D <= 128) return run<X, 128, NT, 16, 8, 3, 16>(a, stream);
    return run<X, 256, kNT, 16, 4, 3, 16>(a, stream);
  }
  if (D <= 64) return run<X, 64, NT, 8, 16, 3, 32>(a, stream);
  if (D <= 128) return run<X, 128, NT, 8, 8, 3, 32>(a, stream);
  return run<X, 256, kNT, 8, 8, 3, 16>(a, stream);
}

}  // namespace

size_t paged_attn_ws_bytes(int Hq, int heads, int dim) {
  const size_t dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  const size_t h = Hq / heads > 8 ? 16 : 8, warps = dim <= 64 ? 16 : 8;
  return scratch_head_bytes() + static_cast<size_t>(kMaxCtas) * (2 + warps) * h * dp * sizeof(float);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  const bool f32 = a.qdt == QVLA_DTYPE_F32;
  // a unit is a key head with 8, or (for larger groups) 16 of its query heads
  if (a.Hq / a.cache.heads > 8)
    return f32 ? run_dim<float, 2>(a, stream) : run_dim<__nv_bfloat16, 2>(a, stream);
  return f32 ? run_dim<float, 1>(a, stream) : run_dim<__nv_bfloat16, 1>(a, stream);
}

}  // namespace qvla
