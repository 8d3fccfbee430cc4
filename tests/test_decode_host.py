"""Host-side refusals of the decode-step operators: every bad call is turned away before any
CUDA call (no GPU here), by the C ABI and by the binding."""
import ctypes

import numpy as np
import pytest
import torch

P = ctypes.c_void_p(1 << 20)       # an aligned address that nothing reads
ODD = ctypes.c_void_p((1 << 20) + 8)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def q():
    from w4a4_post_quantization_zigzag_b200 import build
    build.build()
    from w4a4_post_quantization_zigzag_b200 import qvla
    return qvla


def call(fn, defaults, **kw):
    """fn with the default arguments, some of them replaced by name."""
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


def group_linear(q, **kw):
    d = dict(N=128, K=256, group=64, sdt=0, wq=1 << 20, w_scale=1 << 20, w_zero=1 << 20, bias=1 << 20)
    return q.qvla_group_linear(*{**d, **kw}.values())


def cache(q, **kw):
    d = dict(pages=10, page_size=16, heads=2, dim=64, bits=16, k=1 << 20, v=1 << 20,
             page_stride=2048, token_stride=128, head_stride=64, k_scale=None, v_scale=None,
             s_page_stride=0, s_token_stride=0, s_head_stride=0)
    assert set(kw) <= set(d)
    return q.qvla_kv_cache(*{**d, **kw}.values())


def test_pack_w4g(q):
    f = q._lib.qvla_pack_weights_w4g
    d = dict(W=P, N=64, K=256, group=64, sdt=0, wq=P, scale=P, zero=P, stream=None)
    for kw, code in [(dict(W=None), q.QVLA_ERR_ARG), (dict(wq=None), q.QVLA_ERR_ARG),
                     (dict(scale=None), q.QVLA_ERR_ARG), (dict(sdt=2), q.QVLA_ERR_ARG),
                     (dict(sdt=-1), q.QVLA_ERR_ARG), (dict(group=48), q.QVLA_ERR_SHAPE),
                     (dict(group=0), q.QVLA_ERR_SHAPE), (dict(group=512), q.QVLA_ERR_SHAPE),
                     (dict(K=250), q.QVLA_ERR_SHAPE), (dict(K=0), q.QVLA_ERR_SHAPE),
                     (dict(K=65536), q.QVLA_ERR_SHAPE), (dict(N=0), q.QVLA_ERR_SHAPE),
                     (dict(N=-5), q.QVLA_ERR_SHAPE), (dict(N=(1 << 22) + 1), q.QVLA_ERR_SHAPE),
                     (dict(W=ODD), q.QVLA_ERR_ALIGN), (dict(wq=ODD), q.QVLA_ERR_ALIGN),
                     (dict(scale=ODD), q.QVLA_ERR_ALIGN), (dict(zero=ODD), q.QVLA_ERR_ALIGN)]:
        assert call(f, d, **kw) == code, kw


def test_gemv(q):
    f = q._lib.qvla_w4a16_gemv
    d = dict(x=P, xdt=1, M=4, ldx=256, L=group_linear(q), y=P, ydt=1, ldy=128, stream=None)
    for kw, code in [(dict(L=None), q.QVLA_ERR_ARG), (dict(x=None), q.QVLA_ERR_ARG),
                     (dict(y=None), q.QVLA_ERR_ARG), (dict(xdt=2), q.QVLA_ERR_ARG),
                     (dict(ydt=7), q.QVLA_ERR_ARG), (dict(M=-1), q.QVLA_ERR_SHAPE),
                     (dict(M=(1 << 20) + 1), q.QVLA_ERR_SHAPE), (dict(ldx=248), q.QVLA_ERR_SHAPE),
                     (dict(ldy=120), q.QVLA_ERR_SHAPE), (dict(ldx=260), q.QVLA_ERR_ALIGN),
                     (dict(ldy=130), q.QVLA_ERR_ALIGN), (dict(x=ODD), q.QVLA_ERR_ALIGN),
                     (dict(y=ODD), q.QVLA_ERR_ALIGN),
                     (dict(L=group_linear(q, group=96)), q.QVLA_ERR_SHAPE),
                     (dict(L=group_linear(q, K=288)), q.QVLA_ERR_SHAPE),
                     (dict(L=group_linear(q, N=0)), q.QVLA_ERR_SHAPE),
                     (dict(L=group_linear(q, sdt=3)), q.QVLA_ERR_ARG),
                     (dict(L=group_linear(q, wq=None)), q.QVLA_ERR_ARG),
                     (dict(L=group_linear(q, w_scale=None)), q.QVLA_ERR_ARG),
                     (dict(L=group_linear(q, wq=24)), q.QVLA_ERR_ALIGN),
                     (dict(L=group_linear(q, w_scale=24)), q.QVLA_ERR_ALIGN),
                     (dict(L=group_linear(q, w_zero=24)), q.QVLA_ERR_ALIGN),
                     (dict(L=group_linear(q, bias=24)), q.QVLA_ERR_ALIGN)]:
        assert call(f, d, **kw) == code, kw
    assert call(f, d, M=0, x=None, y=None) == q.QVLA_OK


def test_gemv_rows_past_the_grid(q):
    d = dict(x=P, xdt=1, M=65535 * 16 + 1, ldx=256, L=group_linear(q), y=P, ydt=1, ldy=128, stream=None)
    assert call(q._lib.qvla_w4a16_gemv, d) == q.QVLA_ERR_SHAPE
    assert call(q._lib.qvla_w4a16_gemv, d, M=1 << 20) == q.QVLA_ERR_SHAPE


def test_rope_table(q):
    f = q._lib.qvla_rope_table
    d = dict(inv=P, half=32, P=100, table=P, stream=None)
    for kw, code in [(dict(half=0), q.QVLA_ERR_SHAPE), (dict(half=129), q.QVLA_ERR_SHAPE),
                     (dict(P=-1), q.QVLA_ERR_SHAPE), (dict(inv=None), q.QVLA_ERR_ARG),
                     (dict(table=None), q.QVLA_ERR_ARG), (dict(table=ODD), q.QVLA_ERR_ALIGN)]:
        assert call(f, d, **kw) == code, kw
    assert call(f, d, P=0, inv=None, table=None) == q.QVLA_OK


BAD_CACHES = [
    (dict(bits=4), "ARG"), (dict(bits=0), "ARG"), (dict(pages=0), "SHAPE"), (dict(pages=-1), "SHAPE"),
    (dict(page_size=0), "SHAPE"), (dict(pages=1 << 20, page_size=1 << 12), "SHAPE"),
    (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(k=24), "ALIGN"), (dict(v=24), "ALIGN"),
    (dict(page_stride=0), "SHAPE"), (dict(token_stride=-128), "SHAPE"), (dict(head_stride=32), "SHAPE"),
    (dict(page_stride=2049), "ALIGN"), (dict(token_stride=132), "ALIGN"), (dict(head_stride=66), "ALIGN"),
    (dict(bits=8), "ARG"), (dict(bits=8, k_scale=1 << 20, v_scale=1 << 20), "SHAPE"),
    (dict(bits=8, k_scale=2, v_scale=1 << 20, s_page_stride=32, s_token_stride=2, s_head_stride=1), "ALIGN"),
    (dict(bits=8, k_scale=4, v_scale=6, s_page_stride=32, s_token_stride=2, s_head_stride=1), "ALIGN"),
    (dict(bits=8, k_scale=4, v_scale=4, s_page_stride=32, s_token_stride=2, s_head_stride=-1), "SHAPE"),
    (dict(bits=8, k_scale=4, v_scale=4, s_page_stride=32, s_token_stride=2, s_head_stride=1,
          token_stride=136), "ALIGN"),
]


def test_qk_norm_rope(q):
    f = q._lib.qvla_qk_norm_rope
    d = dict(q=P, k=P, v=P, xdt=1, T=4, Hq=8, Hkv=2, D=64, ldq=768, ldk=768, ldv=768, qn=P, kn=P, eps=1e-6,
             table=P, P=100, rot=64, inter=0, pos=P, cache=cache(q), slots=P, q_out=P, ldqo=512, k_out=P,
             ldko=128, stream=None)
    arg, shape, align = q.QVLA_ERR_ARG, q.QVLA_ERR_SHAPE, q.QVLA_ERR_ALIGN
    for kw, code in [(dict(xdt=5), arg), (dict(D=72), shape), (dict(D=0), shape), (dict(D=272), shape),
                     (dict(T=-1), shape), (dict(T=(1 << 20) + 1), shape), (dict(Hq=-1), shape),
                     (dict(Hkv=-1), shape), (dict(Hq=5000), shape), (dict(Hq=0, Hkv=0, cache=None), shape),
                     (dict(inter=2), arg), (dict(eps=NAN), arg), (dict(eps=INF), arg), (dict(eps=-1.0), arg),
                     (dict(rot=0), shape), (dict(rot=24), shape), (dict(rot=80), shape), (dict(P=0), shape),
                     (dict(table=ODD), align), (dict(pos=None), arg), (dict(slots=None), arg),
                     (dict(q=None), arg), (dict(k=None), arg), (dict(v=None), arg), (dict(q_out=None), arg),
                     (dict(cache=None, k_out=None), arg), (dict(ldq=504), shape), (dict(ldk=120), shape),
                     (dict(ldv=120), shape), (dict(ldqo=504), shape), (dict(ldko=120), shape),
                     (dict(ldq=772), align), (dict(ldk=132), align), (dict(ldv=132), align),
                     (dict(ldqo=516), align), (dict(ldko=132), align), (dict(q=ODD), align),
                     (dict(k=ODD), align), (dict(v=ODD), align), (dict(q_out=ODD), align),
                     (dict(k_out=ODD), align), (dict(qn=ODD), align), (dict(kn=ODD), align),
                     (dict(pos=ctypes.c_void_p(6)), align), (dict(slots=ctypes.c_void_p(6)), align),
                     (dict(cache=cache(q, heads=3)), shape), (dict(cache=cache(q, dim=32)), shape)]:
        assert call(f, d, **kw) == code, kw
    for kw, code in BAD_CACHES:
        assert call(f, d, cache=cache(q, **kw)) == getattr(q, "QVLA_ERR_" + code), kw
    assert call(f, d, T=0, q=None, k=None, v=None, pos=None, slots=None, q_out=None) == q.QVLA_OK


def test_qk_norm_rope_in_place_with_another_pitch(q):
    """Rows written at another pitch over their own inputs would overwrite rows not yet read."""
    Q, O = ctypes.c_void_p(1 << 21), ctypes.c_void_p(1 << 22)
    d = dict(q=Q, k=P, v=P, xdt=1, T=4, Hq=8, Hkv=2, D=64, ldq=768, ldk=768, ldv=768, qn=P, kn=P, eps=1e-6,
             table=P, P=100, rot=64, inter=0, pos=P, cache=cache(q), slots=P, q_out=O, ldqo=512, k_out=O,
             ldko=128, stream=None)
    f = q._lib.qvla_qk_norm_rope
    assert call(f, d, q_out=Q) == q.QVLA_ERR_ARG
    assert call(f, d, k_out=P) == q.QVLA_ERR_ARG


def test_paged_attn(q):
    b = ctypes.c_size_t()
    g = q._lib.qvla_paged_attn_workspace_bytes
    assert g(8, 2, 64, ctypes.byref(b)) == q.QVLA_OK and b.value > 0
    assert q.qvla_paged_attn_workspace_bytes(8, 2, 64) == b.value
    assert g(8, 2, 64, None) == q.QVLA_ERR_ARG
    for a in ((8, 3, 64), (0, 2, 64), (8, 0, 64), (8, 2, 72), (8, 2, 0), (8, 2, 512), (-8, 2, 64), (8192, 2, 64)):
        assert g(*a, ctypes.byref(b)) == q.QVLA_ERR_SHAPE, a
    need = q.qvla_paged_attn_workspace_bytes(8, 2, 64)
    f = q._lib.qvla_paged_attn_decode
    d = dict(q=P, qdt=1, B=3, Hq=8, ldq=512, cache=cache(q), table=P, max_pages=10, lens=P, scale=0.125, window=0,
             sinks=0, out=P, ldo=512, lse=P, ws=P, ws_bytes=need, stream=None)
    arg, shape, align = q.QVLA_ERR_ARG, q.QVLA_ERR_SHAPE, q.QVLA_ERR_ALIGN
    for kw, code in [(dict(cache=None), arg), (dict(qdt=2), arg), (dict(scale=NAN), arg), (dict(scale=INF), arg),
                     (dict(window=-1), arg), (dict(sinks=-1), arg), (dict(Hq=7), shape), (dict(Hq=0), shape),
                     (dict(B=-1), shape), (dict(B=65537), shape), (dict(max_pages=0), shape),
                     (dict(max_pages=1 << 28), shape), (dict(q=None), arg), (dict(table=None), arg),
                     (dict(lens=None), arg), (dict(out=None), arg), (dict(ldq=504), shape), (dict(ldo=504), shape),
                     (dict(ldq=516), align), (dict(ldo=516), align), (dict(q=ODD), align), (dict(out=ODD), align),
                     (dict(table=ctypes.c_void_p(6)), align), (dict(lens=ctypes.c_void_p(6)), align),
                     (dict(lse=ctypes.c_void_p(6)), align), (dict(ws=None), q.QVLA_ERR_WORKSPACE),
                     (dict(ws_bytes=need - 1), q.QVLA_ERR_WORKSPACE), (dict(ws=ODD), align)]:
        assert call(f, d, **kw) == code, kw
    for kw, code in BAD_CACHES:
        assert call(f, d, cache=cache(q, **kw)) == getattr(q, "QVLA_ERR_" + code), kw
    assert call(f, d, B=0, q=None, table=None, lens=None, out=None, ws=None) == q.QVLA_OK


def test_paged_attn_sequence_past_its_token_numbers(q):
    """Pages may be shared, so a sequence's length is bounded by its table, not by the cache."""
    need = q.qvla_paged_attn_workspace_bytes(8, 2, 64)
    d = dict(q=P, qdt=1, B=3, Hq=8, ldq=512, cache=cache(q), table=P, max_pages=(1 << 26) + 1, lens=P, scale=0.125,
             window=0, sinks=0, out=P, ldo=512, lse=P, ws=P, ws_bytes=need, stream=None)
    assert call(q._lib.qvla_paged_attn_decode, d) == q.QVLA_ERR_SHAPE
    assert call(q._lib.qvla_paged_attn_decode, d, max_pages=(1 << 27) - 1) == q.QVLA_ERR_SHAPE


def test_paged_attn_in_place_with_another_pitch(q):
    need = q.qvla_paged_attn_workspace_bytes(8, 2, 64)
    d = dict(q=P, qdt=1, B=3, Hq=8, ldq=768, cache=cache(q), table=P, max_pages=10, lens=P, scale=0.125, window=0,
             sinks=0, out=P, ldo=512, lse=P, ws=P, ws_bytes=need, stream=None)
    assert call(q._lib.qvla_paged_attn_decode, d) == q.QVLA_ERR_ARG


def test_binding_refuses_what_32_bits_do_not_hold(q):
    """Pitches, windows and sizes past 32 bits must not reach the C call cut to their low bits."""
    def meta(shape, strides=None, dt=torch.bfloat16):
        if strides is None:
            return torch.empty(shape, dtype=dt, device="meta")
        return torch.empty_strided(shape, strides, dtype=dt, device="meta")
    far = (1 << 32) + 128
    wq, s = meta((128, 64), dt=torch.uint8), meta((128, 4))
    x, i32 = meta((2, 128)), dict(dt=torch.int32)
    h, kc = meta((2, 4, 16)), meta((5, 8, 4, 16))
    tab, lens = meta((2, 3), **i32), meta((2,), **i32)
    calls = [lambda: q.qvla_w4a16_gemv(meta((2, 128), (far, 1)), wq, s),
             lambda: q.qvla_w4a16_gemv(x, wq, s, y=meta((2, 128), (far, 1))),
             lambda: q.qvla_qk_norm_rope(meta((2, 4, 16), (far, 16, 1)), None),
             lambda: q.qvla_qk_norm_rope(h, None, q_out=meta((2, 4, 16), (far, 16, 1))),
             lambda: q.qvla_qk_norm_rope(h, None, rope_table=meta((1 << 31, 16), dt=torch.float32),
                                         positions=meta((2,), **i32)),
             lambda: q.qvla_paged_attn_decode(h, kc, kc, tab, lens, window=(1 << 32) + 5),
             lambda: q.qvla_paged_attn_decode(h, kc, kc, tab, lens, window=5, sinks=1 << 32),
             lambda: q.qvla_paged_attn_decode(h, kc, kc, tab, lens, window=-1),
             lambda: q.qvla_paged_attn_decode(h, meta((far, 8, 4, 16)), meta((far, 8, 4, 16)), tab, lens)]
    for f in calls:
        with pytest.raises(q.QvlaError):
            f()


def test_binding_refuses_host_and_mismatched_tensors(q):
    """Wrong types, shapes and places raise in the binding; nothing of them reaches a kernel."""
    x, wq, s = torch.zeros(2, 128), torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4)
    for args in [(x, wq, s), (x[:, :64], wq, s), (x, wq.float(), s), (x, wq, s[:, :3]), (x, wq, s.T),
                 (x, wq, s, s), (x, wq, s, None, s), (x.T, wq, s)]:
        with pytest.raises((ValueError, TypeError)):
            q.qvla_w4a16_gemv(*args)
    with pytest.raises(ValueError):
        q.qvla_w4a16_gemv(x, wq, s, y=torch.zeros(2, 9))
    with pytest.raises(ValueError):
        q.qvla_pack_weights_w4g(torch.zeros(4, 128))
    with pytest.raises(q.QvlaError):
        q.qvla_pack_weights_w4g(torch.zeros(4, 128), 48)
    with pytest.raises(ValueError):
        q.qvla_rope_table(np.ones((2, 2)), 4, device="cpu")
    h, kc = torch.zeros(3, 4, 16), torch.zeros(5, 8, 4, 16, dtype=torch.bfloat16)
    i3 = torch.zeros(3, dtype=torch.int32)
    for kw in [dict(q=None, k=None), dict(q=h, k=None), dict(q=h, k=h[:2]), dict(q=h, k=h.double()),
               dict(q=h.transpose(0, 1), k=None), dict(q=h, k=h, rope_table=torch.zeros(9, 16)),
               dict(q=h, k=h, q_norm=torch.zeros(15)), dict(q=h, k=h, k_cache=kc),
               dict(q=h, k=h, v=h, k_cache=kc, v_cache=kc, slots=i3.long()),
               dict(q=h, k=h, v=h, k_cache=kc, v_cache=kc[:4], slots=i3),
               dict(q=h, k=h, v=h, k_cache=kc, v_cache=kc, slots=i3, k_scale=kc),
               dict(q=h, k=h, v=h, k_cache=kc.char(), v_cache=kc.char(), slots=i3),
               dict(q=h, k=h, v=h, k_cache=kc.float(), v_cache=kc.float(), slots=i3),
               dict(q=h, k=None, q_out=h[:2]), dict(q=h.to(torch.float16), k=None)]:
        with pytest.raises((ValueError, TypeError)):
            q.qvla_qk_norm_rope(**kw)
    tab, lens = torch.zeros(3, 2, dtype=torch.int32), i3
    for a in [(h, kc, kc, tab, lens), (h, kc, kc, tab.long(), lens), (h, kc, kc, tab, lens[:2]),
              (h[:, :, :8], kc, kc, tab, lens), (h, kc, kc[:3], tab, lens), (h, kc[0], kc[0], tab, lens),
              (h, kc, kc, tab[0], lens), (h.half(), kc, kc, tab, lens)]:
        with pytest.raises((ValueError, TypeError)):
            q.qvla_paged_attn_decode(*a)


def test_binding_refuses_every_size_that_32_bits_do_not_hold(q):
    """Counts of outputs, inputs, positions, heads and head values too."""
    def meta(*shape, dt=torch.bfloat16):
        return torch.empty(shape, dtype=dt, device="meta")
    far, u8, f32 = (1 << 32) + 128, torch.uint8, torch.float32
    kc, tab = meta(5, 8, 4, 16), meta(1, 3, dt=torch.int32)
    lens = meta(1, dt=torch.int32)
    calls = [lambda: q.qvla_w4a16_gemv(meta(1, 32), meta(far, 16, dt=u8), meta(far, 1, dt=f32)),
             lambda: q.qvla_w4a16_gemv(meta(1, far), meta(4, far // 2, dt=u8), meta(4, far // 128, dt=f32)),
             lambda: q.qvla_pack_weights_w4g(meta(far, 32, dt=f32), 32),
             lambda: q.qvla_pack_weights_w4g(meta(1, far, dt=f32), 128),
             lambda: q.qvla_rope_table(np.ones(1), far, device="meta"),
             lambda: q.qvla_rope_table(np.ones(1), 1 << 31, device="meta"),
             lambda: q.qvla_qk_norm_rope(meta(1, far, 16), None),
             lambda: q.qvla_qk_norm_rope(meta(1, 4, far), None),
             lambda: q.qvla_qk_norm_rope(None, meta(2, far, 16)),
             lambda: q.qvla_paged_attn_decode(meta(1, far, 16), kc, kc, tab, lens),
             lambda: q.qvla_paged_attn_decode(meta(1, 4, 16), meta(5, 8, far, 16), meta(5, 8, far, 16), tab, lens),
             lambda: q.qvla_paged_attn_decode(meta(1, 4, 16), meta(5, 8, 4, (1 << 32) + 16),
                                              meta(5, 8, 4, (1 << 32) + 16), tab, lens)]
    for i, f in enumerate(calls):
        with pytest.raises(q.QvlaError):
            f()
            pytest.fail(f"call {i}")
