"""The decode-step operators one after the other, as a served layer runs them: a W4A4 (or W4A16)
qkv linear, norm + rotation + cache write, attention over the cache, a W4A16 output projection,
captured once and replayed for every new token.  Each stage is held to fp64 of its own inputs, and
the attention to a dense history kept beside the cache."""
import os
import subprocess
import sys

import pytest
import torch

import _decode_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def q():
    from w4a4_post_quantization_zigzag_b200 import build
    build.build()
    from w4a4_post_quantization_zigzag_b200 import qvla
    assert torch.cuda.is_available()
    qvla.qvla_read_error_word(clear=True)
    return qvla


@pytest.mark.parametrize("bits,window,linear", [(16, 0, "w4a4"), (8, 24, "w4a16"), (16, 24, "w4a16")])
def test_decode_loop(q, bits, window, linear):
    B, hid, Hq, Hkv, D, ps, steps, sinks = 5, 256, 8, 2, 64, 8, 40, 3
    g = torch.Generator(device="cuda").manual_seed(bits + window)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    nqkv = (Hq + 2 * Hkv) * D
    Wqkv, Wo = randn(nqkv, hid) * 0.1, randn(hid, Hq * D) * 0.1
    bias = randn(nqkv) * 0.1
    L4 = q.qvla_pack_weights(Wqkv, 64, bias=bias) if linear == "w4a4" else None
    qkv_w = q.qvla_pack_weights_w4g(Wqkv, 64, True, BF)
    o_w = q.qvla_pack_weights_w4g(Wo, 128)
    qn, kn = (1 + 0.1 * randn(2, D)).unbind(0)
    qn, kn = qn.contiguous(), kn.contiguous()
    table = q.qvla_rope_table(10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D), 64)
    width = steps // ps
    pages = B * width + 1
    kc, vc = (torch.zeros(pages, ps, Hkv, D, dtype=BF if bits == 16 else torch.int8, device="cuda")
              for _ in range(2))
    ks, vs = ((torch.zeros(pages, ps, Hkv, device="cuda") for _ in range(2)) if bits == 8 else (None, None))
    ptab = torch.randperm(pages, device="cuda", generator=g)[:B * width].int().view(B, width).contiguous()
    x = torch.zeros(B, hid, dtype=BF, device="cuda")
    pos, slots, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    rows = torch.empty(B, nqkv, dtype=BF, device="cuda")
    qr, at, y = (torch.empty(B, Hq, D, dtype=BF, device="cuda"), torch.empty(B, Hq, D, dtype=BF, device="cuda"),
                 torch.empty(B, hid, dtype=BF, device="cuda"))
    ws = torch.empty(q.qvla_paged_attn_workspace_bytes(Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    codes = (torch.empty(B, hid // 2, dtype=torch.uint8, device="cuda"), torch.empty(B, device="cuda"))
    a, b = Hq * D, (Hq + Hkv) * D

    def step():
        if linear == "w4a4":
            q.qvla_rotate_quant_act(x, L4, xq=codes[0], s_x=codes[1])
            q.qvla_w4a4_gemm(*codes, L4, y=rows)
        else:
            q.qvla_w4a16_gemv(x, *qkv_w, bias, y=rows)
        q.qvla_qk_norm_rope(rows[:, :a].unflatten(1, (Hq, D)), rows[:, a:b].unflatten(1, (Hkv, D)),
                            rows[:, b:].unflatten(1, (Hkv, D)), qn, kn, table, pos, slots, kc, vc, ks, vs,
                            eps=EPS, q_out=qr)
        q.qvla_paged_attn_decode(qr, kc, vc, ptab, lens, window=window, sinks=sinks, k_scale=ks, v_scale=vs,
                                 out=at, workspace=ws)
        q.qvla_w4a16_gemv(at.view(B, a), *o_w, y=y)

    slots.fill_(-1)                     # a dry step writes nothing
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert not kc.any() and not vc.any()
    hist_k, hist_v = [], []
    for t in range(steps):
        x.copy_(randn(B, hid))
        pos.fill_(t)
        slots.copy_(ptab[:, t // ps] * ps + t % ps)
        lens.fill_(t + 1)
        graph.replay()
        torch.cuda.synchronize()
        if linear == "w4a16":
            R.within(rows, *R.gemv(x, *qkv_w, bias), "qkv")
        cs = table[pos.long()]
        cs = cs[:, :D // 2], cs[:, D // 2:]
        R.within(qr, *R.norm_rope(rows[:, :a].view(B, Hq, D), qn, *cs, D, False, EPS), "q")
        rk, sk = R.norm_rope(rows[:, a:b].view(B, Hkv, D), kn, *cs, D, False, EPS)
        hist_k.append(rk)
        hist_v.append(rows[:, b:].view(B, Hkv, D).double())
        ro, _, so, _ = R.paged_attn(qr, kc, vc, ptab, lens, D ** -0.5, window, sinks, ks, vs)
        R.within(at, ro, so, "attention")
        R.within(y, *R.gemv(at.view(B, a), *o_w), "o")
        # against the unrounded history: each key and value is off by one rounding of the cache
        k, v = torch.stack(hist_k, 1), torch.stack(hist_v, 1)          # [B, t, Hkv, D]
        see = torch.arange(t + 1, device="cuda")
        see = (see < sinks) | (see >= t + 1 - window) if window else see >= 0
        k, v = (m[:, see].repeat_interleave(Hq // Hkv, 2) for m in (k, v))
        s = torch.einsum("bhd,bthd->bht", qr.double(), k) * D ** -0.5
        p = torch.softmax(s, 2)
        dense = torch.einsum("bht,bthd->bhd", p, v)
        if bits == 16:
            step_k, step_v = k.abs() * R.half_step(BF), v.abs() * 0
        else:
            step_k, step_v = (m.abs().amax(-1, keepdim=True).expand_as(m) / 127 * 0.51 for m in (k, v))
        ds = torch.einsum("bhd,bthd->bht", qr.double().abs(), step_k).amax(2) * D ** -0.5 * 1.01
        slack = so + torch.einsum("bht,bthd->bhd", p, v.abs()) * (torch.exp(2 * ds) - 1)[..., None] \
            + torch.einsum("bht,bthd->bhd", p, step_v) * torch.exp(2 * ds)[..., None]
        R.within(at, dense, slack, "history")
    assert q.qvla_read_error_word(clear=True) == 0


def test_first_calls_inside_a_capture():
    """Every operator's first call of a process may be the captured one."""
    code = '''
import torch
from w4a4_post_quantization_zigzag_b200 import qvla as q
dev, BF = "cuda", torch.bfloat16
x = torch.randn(3, 256, device=dev).to(BF)
W = torch.randn(64, 256, device=dev)
h = torch.randn(2, 6, 64, device=dev).to(BF)
kc, vc = (torch.zeros(4, 16, 2, 64, device=dev, dtype=BF) for _ in range(2))
i32 = dict(dtype=torch.int32, device=dev)
pos, slots = torch.tensor([3, 0], **i32), torch.tensor([3, 16], **i32)
tab, lens = torch.tensor([[0], [1]], **i32), torch.tensor([4, 1], **i32)
freqs = [10000.0 ** (-i / 32) for i in range(32)]
def step():
    wq, s, z = q.qvla_pack_weights_w4g(W, 64, True)
    table = q.qvla_rope_table(freqs, 8)
    out = q.qvla_qk_norm_rope(h[:, :4], h[:, 4:], h[:, 4:], None, None, table, pos, slots, kc, vc)
    return (q.qvla_w4a16_gemv(x, wq, s, z), q.qvla_w4a16_gemv(x[:1], wq, s, z), out,
            q.qvla_paged_attn_decode(out, kc, vc, tab, lens))
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert q.qvla_read_error_word() == 0
'''
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_bench_decode_workload():
    """The bench's decode workload: one line, the whole step in the library's kernels (rotation,
    its permuted copy, GEMM, norm, attention and its join, output projection)."""
    import json
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--workload",
                        "backbone_decode", "--steps", "4", "--warmup", "3", "--quick"], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    (line,) = [json.loads(l) for l in r.stdout.splitlines() if l.startswith("{")]
    assert line["value"] > 0 and line["config"]["workload"].startswith("backbone_decode")
    assert line["kernels_per_step"] >= 6 and line["gpu_launches"] == 4 * line["kernels_per_step"]
    assert line["e2e"]["value"] > 0 and line["e2e"]["h2d_bytes_per_step"] == 2048 * 2


def test_calls_after_a_failed_one():
    """The error of a call that cannot run (the error word read inside a capture) belongs to that
    call alone: each operator's next call runs and says so."""
    code = '''
import torch
from w4a4_post_quantization_zigzag_b200 import qvla as q
dev, BF = "cuda", torch.bfloat16
x = torch.randn(3, 256, device=dev).to(BF)
W = torch.randn(64, 256, device=dev)
h = torch.randn(2, 4, 64, device=dev).to(BF)
kc, vc = (torch.randn(4, 16, 2, 64, device=dev).to(BF) for _ in range(2))
i32 = dict(dtype=torch.int32, device=dev)
tab, lens = torch.tensor([[0], [1]], **i32), torch.tensor([4, 1], **i32)
wq, s, z = q.qvla_pack_weights_w4g(W, 64, True)
calls = [lambda: q.qvla_pack_weights_w4g(W, 64, True)[0], lambda: q.qvla_rope_table([1.0, 0.5], 8),
         lambda: q.qvla_qk_norm_rope(h, None)[0], lambda: q.qvla_w4a16_gemv(x, wq, s, z),
         lambda: q.qvla_paged_attn_decode(h, kc, vc, tab, lens)]
want = [f() for f in calls]
torch.cuda.synchronize()
for f, w in zip(calls, want):
    failed = 0
    try:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            try:
                q.qvla_read_error_word()
            except q.QvlaError:
                failed += 1
    except RuntimeError:
        failed += 1
    assert failed == 2
    got = f()
    torch.cuda.synchronize()
    assert torch.equal(got, w)
assert q.qvla_read_error_word() == 0
'''
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
