// C ABI of the operators around the linears of a decode step: W4A16 products,
// norm + rotation + cache write, attention over the paged cache.  Argument
// validation only; every check runs on the host before anything is launched.
#include <climits>
#include <cmath>
#include <cstring>

#include "qvla_internal.h"

using namespace qvla;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

qvla_status cuda_status(cudaError_t e) { return e == cudaSuccess ? QVLA_OK : QVLA_ERR_CUDA; }

bool valid_dtype(int d) { return d == QVLA_DTYPE_F32 || d == QVLA_DTYPE_BF16; }
size_t dtype_size(int d) { return d == QVLA_DTYPE_F32 ? 4 : 2; }
bool aligned_pitch(int64_t elements, int d) { return elements * dtype_size(d) % 16 == 0; }

constexpr int kMaxN = 1 << 22, kMaxRows = 1 << 20;
constexpr int kMaxGemvRows = 65535 * 16;       // a grid's second extent, 16 rows a pass

qvla_status check_group_shape(int N, int K, int group) {
  if (group != 32 && group != 64 && group != 128 && group != 256) return QVLA_ERR_SHAPE;
  if (N <= 0 || N > kMaxN || K <= 0 || K > QVLA_MAX_K || K % group) return QVLA_ERR_SHAPE;
  return QVLA_OK;
}

qvla_status check_dim(int D) {
  return D < 16 || D > 256 || D % 16 ? QVLA_ERR_SHAPE : QVLA_OK;
}

qvla_status check_cache(const qvla_kv_cache* c) {
  if (!c) return QVLA_ERR_ARG;
  if (c->bits != 16 && c->bits != 8) return QVLA_ERR_ARG;
  if (c->pages <= 0 || c->page_size <= 0 || c->heads <= 0) return QVLA_ERR_SHAPE;
  if (check_dim(c->dim) != QVLA_OK) return QVLA_ERR_SHAPE;
  if (static_cast<int64_t>(c->pages) * c->page_size > INT_MAX) return QVLA_ERR_SHAPE;
  if (!c->k || !c->v) return QVLA_ERR_ARG;
  if (c->bits == 8 && (!c->k_scale || !c->v_scale)) return QVLA_ERR_ARG;
  const int64_t stride[3] = {c->page_stride, c->token_stride, c->head_stride};
  const int extent[3] = {c->pages, c->page_size, c->heads};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] == 1) continue;
    if (stride[i] < c->dim) return QVLA_ERR_SHAPE;
    if (stride[i] * (c->bits / 8) % 16) return QVLA_ERR_ALIGN;
  }
  if (!aligned16(c->k) || !aligned16(c->v)) return QVLA_ERR_ALIGN;
  if (c->bits == 8) {
    const int64_t s[3] = {c->s_page_stride, c->s_token_stride, c->s_head_stride};
    for (int i = 0; i < 3; ++i)
      if (extent[i] > 1 && s[i] < 1) return QVLA_ERR_SHAPE;
    if (!aligned4(c->k_scale) || !aligned4(c->v_scale)) return QVLA_ERR_ALIGN;
  }
  return QVLA_OK;
}

// A copy whose strides of extents of 1 are 0 (whatever the caller left there).
qvla_kv_cache plain_cache(const qvla_kv_cache& c) {
  qvla_kv_cache r = c;
  if (c.pages == 1) r.page_stride = r.s_page_stride = 0;
  if (c.page_size == 1) r.token_stride = r.s_token_stride = 0;
  if (c.heads == 1) r.head_stride = r.s_head_stride = 0;
  return r;
}

qvla_status check_sm100() {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return QVLA_ERR_CUDA;
  return major == 10 ? QVLA_OK : QVLA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

qvla_status qvla_pack_weights_w4g(const float* W, int N, int K, int group, qvla_dtype sdt,
                                  uint8_t* wq_out, void* w_scale_out, uint8_t* w_zero_out,
                                  cudaStream_t stream) {
  qvla_status st = check_group_shape(N, K, group);
  if (st != QVLA_OK) return st;
  if (!valid_dtype(sdt)) return QVLA_ERR_ARG;
  if (!W || !wq_out || !w_scale_out) return QVLA_ERR_ARG;
  if (!aligned16(W) || !aligned16(wq_out) || !aligned16(w_scale_out) ||
      (w_zero_out && !aligned16(w_zero_out)))
    return QVLA_ERR_ALIGN;
  return cuda_status(launch_pack_w4g(W, N, K, group, sdt, wq_out, w_scale_out, w_zero_out, stream));
}

qvla_status qvla_w4a16_gemv(const void* x, qvla_dtype xdt, int M, int ldx,
                            const qvla_group_linear* L, void* y, qvla_dtype ydt, int ldy,
                            cudaStream_t stream) {
  if (!L) return QVLA_ERR_ARG;
  qvla_status st = check_group_shape(L->N, L->K, L->group);
  if (st != QVLA_OK) return st;
  if (!valid_dtype(xdt) || !valid_dtype(ydt) || !valid_dtype(L->sdt)) return QVLA_ERR_ARG;
  if (!L->wq || !L->w_scale) return QVLA_ERR_ARG;
  if (!aligned16(L->wq) || !aligned16(L->w_scale) || !aligned16(L->w_zero) || !aligned16(L->bias))
    return QVLA_ERR_ALIGN;
  if (M < 0 || M > kMaxGemvRows) return QVLA_ERR_SHAPE;
  if (M == 0) return QVLA_OK;
  if (!x || !y) return QVLA_ERR_ARG;
  if (ldx < L->K || ldy < L->N) return QVLA_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(y) || !aligned_pitch(ldx, xdt) || !aligned_pitch(ldy, ydt))
    return QVLA_ERR_ALIGN;
  if ((st = check_sm100()) != QVLA_OK) return st;
  GemvArgs a = {};
  a.x = x;
  a.xdt = xdt;
  a.M = M;
  a.ldx = ldx;
  a.N = L->N;
  a.K = L->K;
  a.group = L->group;
  a.sdt = static_cast<qvla_dtype>(L->sdt);
  a.wq = L->wq;
  a.scale = L->w_scale;
  a.zero = L->w_zero;
  a.bias = L->bias;
  a.y = y;
  a.ydt = ydt;
  a.ldy = ldy;
  return cuda_status(launch_w4a16_gemv(a, stream));
}

qvla_status qvla_rope_table(const double* inv_freq, int half, int P, float* table,
                            cudaStream_t stream) {
  if (half < 1 || half > 128 || P < 0) return QVLA_ERR_SHAPE;
  if (P == 0) return QVLA_OK;
  if (!inv_freq || !table) return QVLA_ERR_ARG;
  if (!aligned16(table)) return QVLA_ERR_ALIGN;
  RopeFreqs f = {};
  std::memcpy(f.f, inv_freq, sizeof(double) * half);
  return cuda_status(launch_rope_table(f, half, P, table, stream));
}

qvla_status qvla_qk_norm_rope(const void* q, const void* k, const void* v, qvla_dtype xdt, int T,
                              int Hq, int Hkv, int D, int ldq, int ldk, int ldv,
                              const float* q_norm, const float* k_norm, float eps,
                              const float* rope_table, int P, int rot, int interleaved,
                              const int32_t* positions, const qvla_kv_cache* cache,
                              const int32_t* slots, void* q_out, int ldqo, void* k_out, int ldko,
                              cudaStream_t stream) {
  if (!valid_dtype(xdt)) return QVLA_ERR_ARG;
  qvla_status st = check_dim(D);
  if (st != QVLA_OK) return st;
  if (T < 0 || T > kMaxRows || Hq < 0 || Hkv < 0 || Hq > 4096 || Hkv > 4096 || Hq + Hkv == 0)
    return QVLA_ERR_SHAPE;
  if ((interleaved != 0 && interleaved != 1) || !std::isfinite(eps) || eps < 0.f) return QVLA_ERR_ARG;
  if (rope_table) {
    if (rot < 16 || rot > D || rot % 16 || P <= 0) return QVLA_ERR_SHAPE;
    if (!aligned16(rope_table)) return QVLA_ERR_ALIGN;
  }
  if (cache) {
    if ((st = check_cache(cache)) != QVLA_OK) return st;
    if (cache->heads != Hkv || cache->dim != D) return QVLA_ERR_SHAPE;
  }
  if (T == 0) return QVLA_OK;
  if (rope_table && !positions) return QVLA_ERR_ARG;
  if (cache && (!slots || !k || !v)) return QVLA_ERR_ARG;
  if (Hq && (!q || !q_out)) return QVLA_ERR_ARG;
  if (Hkv && (!k || (!cache && !k_out))) return QVLA_ERR_ARG;
  const int64_t nq = static_cast<int64_t>(Hq) * D, nk = static_cast<int64_t>(Hkv) * D;
  if (Hq && (ldq < nq || ldqo < nq)) return QVLA_ERR_SHAPE;
  if (Hkv && (ldk < nk || (cache && ldv < nk) || (k_out && ldko < nk))) return QVLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(q_norm) || !aligned16(k_norm) || !aligned4(positions) || !aligned4(slots))
    return QVLA_ERR_ALIGN;
  if ((Hq && (!aligned_pitch(ldq, xdt) || !aligned_pitch(ldqo, xdt))) ||
      (Hkv && (!aligned_pitch(ldk, xdt) || (cache && !aligned_pitch(ldv, xdt)) ||
               (k_out && !aligned_pitch(ldko, xdt)))))
    return QVLA_ERR_ALIGN;
  // in place, a row may only be written where it was read
  if (T > 1 && ((Hq && q == q_out && ldq != ldqo) || (Hkv && k == k_out && ldk != ldko)))
    return QVLA_ERR_ARG;
  if ((st = check_sm100()) != QVLA_OK) return st;
  NormRopeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.xdt = xdt;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.eps = eps;
  a.table = rope_table;
  a.P = P;
  a.rot = rope_table ? rot : 0;
  a.interleaved = interleaved;
  a.positions = positions;
  a.slots = slots;
  a.has_cache = cache != nullptr;
  if (cache) a.cache = plain_cache(*cache);
  a.q_out = q_out;
  a.k_out = Hkv ? k_out : nullptr;
  a.ldqo = ldqo;
  a.ldko = ldko;
  return cuda_status(launch_qk_norm_rope(a, stream));
}

qvla_status qvla_paged_attn_workspace_bytes(int Hq, int heads, int dim, size_t* bytes) {
  if (!bytes) return QVLA_ERR_ARG;
  if (heads <= 0 || heads > 4096 || Hq <= 0 || Hq > 4096 || Hq % heads || check_dim(dim) != QVLA_OK)
    return QVLA_ERR_SHAPE;
  *bytes = paged_attn_ws_bytes(Hq, heads, dim);
  return QVLA_OK;
}

qvla_status qvla_paged_attn_decode(const void* q, qvla_dtype qdt, int B, int Hq, int ldq,
                                   const qvla_kv_cache* cache, const int32_t* page_table,
                                   int max_pages, const int32_t* seq_lens, float scale,
                                   int window, int sinks, void* out, int ldo, float* lse,
                                   void* workspace, size_t ws_bytes, cudaStream_t stream) {
  qvla_status st = check_cache(cache);
  if (st != QVLA_OK) return st;
  if (!valid_dtype(qdt) || !std::isfinite(scale)) return QVLA_ERR_ARG;
  if (window < 0 || sinks < 0) return QVLA_ERR_ARG;
  size_t need = 0;
  if ((st = qvla_paged_attn_workspace_bytes(Hq, cache->heads, cache->dim, &need)) != QVLA_OK)
    return st;
  if (B < 0 || B > 65536 || max_pages <= 0) return QVLA_ERR_SHAPE;
  // a sequence's token numbers, rounded up to whole tiles, are 32 bits wide
  if (static_cast<int64_t>(max_pages) * cache->page_size > (1 << 30)) return QVLA_ERR_SHAPE;
  if (B == 0) return QVLA_OK;
  if (!q || !page_table || !seq_lens || !out) return QVLA_ERR_ARG;
  const int64_t row = static_cast<int64_t>(Hq) * cache->dim;
  if (ldq < row || ldo < row) return QVLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out) || !aligned_pitch(ldq, qdt) || !aligned_pitch(ldo, qdt) ||
      !aligned4(page_table) || !aligned4(seq_lens) || !aligned4(lse))
    return QVLA_ERR_ALIGN;
  if (B > 1 && q == out && ldq != ldo) return QVLA_ERR_ARG;      // in place, row on row only
  if (!workspace || ws_bytes < need) return QVLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QVLA_ERR_ALIGN;
  if ((st = check_sm100()) != QVLA_OK) return st;
  PagedAttnArgs a = {};
  a.q = q;
  a.qdt = qdt;
  a.B = B;
  a.Hq = Hq;
  a.ldq = ldq;
  a.cache = plain_cache(*cache);
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.out = out;
  a.ldo = ldo;
  a.lse = lse;
  a.ws = workspace;
  return cuda_status(launch_paged_attn(a, stream));
}

}  // extern "C"
