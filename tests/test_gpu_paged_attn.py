"""Attention of one new token over the paged cache on the GPU against fp64."""
import pytest
import torch

import _decode_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    from w4a4_post_quantization_zigzag_b200 import build
    build.build()
    from w4a4_post_quantization_zigzag_b200 import qvla
    assert torch.cuda.is_available()
    qvla.qvla_read_error_word(clear=True)
    return qvla


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def setup(lens, Hq, Hkv, D, dt=BF, ps=16, bits=16, hnd=False, seed=0, junk=True, spare=3):
    """Random pages in random order.  With `junk`, every slot that no token owns holds NaN (its
    scale for an 8-bit cache) and unused table entries point nowhere."""
    g = gen(seed)
    B = len(lens)
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, device="cuda", generator=g).int()
    width = max(max(need), 1)
    tab = torch.full((B, width), -(2 ** 31) if junk else 0, dtype=torch.int32, device="cuda")
    owned = torch.zeros(pages, ps, dtype=torch.bool, device="cuda")
    at = 0
    for b in range(B):
        mine = order[at:at + need[b]]
        tab[b, :need[b]] = mine
        at += need[b]
        t = torch.arange(lens[b], device="cuda")
        owned[mine.long()[t // ps], t % ps] = True
    d = dict(q=torch.randn(B, Hq, D, device="cuda", generator=g).to(dt), tab=tab,
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), ks=None, vs=None)
    for c in "kv":
        x = torch.randn(pages, ps, Hkv, D, device="cuda", generator=g)
        if bits == 16:
            x = x.to(BF)
            if junk:
                x[~owned] = float("nan")
        else:
            x = torch.randint(-128, 128, x.shape, dtype=torch.int8, device="cuda", generator=g)
            s = 0.004 + 0.02 * torch.rand(pages, ps, Hkv, device="cuda", generator=g)
            if junk:
                s[~owned] = float("nan")
            d[c + "s"] = s.transpose(1, 2).contiguous().transpose(1, 2) if hnd else s
        d[c + "c"] = x.transpose(1, 2).contiguous().transpose(1, 2) if hnd else x
    return d


def run(q, d, **kw):
    return q.qvla_paged_attn_decode(d["q"], d["kc"], d["vc"], d["tab"], d["lens"], k_scale=d["ks"],
                                    v_scale=d["vs"], **kw)


def check(q, d, scale=None, window=0, sinks=0, error=0):
    B, Hq, D = d["q"].shape
    lse = torch.full((B, Hq), 9.0, device="cuda")
    o = run(q, d, scale=scale, window=window, sinks=sinks, lse=lse)
    ro, rl, so, sl = R.paged_attn(d["q"], d["kc"], d["vc"], d["tab"], d["lens"],
                                  D ** -0.5 if scale is None else scale, window, sinks, d["ks"], d["vs"])
    R.within(o, ro, so, "o")
    empty = rl == -torch.inf
    assert torch.equal(lse == -torch.inf, empty)
    assert (o[empty] == 0).all()
    R.within(lse[~empty], rl[~empty], sl[~empty], "lse")
    assert q.qvla_read_error_word(clear=True) == error
    return o


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 240, 256])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bits", [16, 8])
def test_dims_and_types(q, D, dt, bits):
    check(q, setup([37, 1, 130], 6, 2, D, dt, bits=bits, seed=D))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (12, 12), (32, 8), (7, 1), (9, 1), (16, 1), (17, 1),
                                    (34, 2), (71, 1), (128, 2)])
@pytest.mark.parametrize("dt,bits,D", [(BF, 16, 128), (F32, 16, 64), (BF, 8, 256), (F32, 8, 128)])
def test_head_groups(q, Hq, Hkv, dt, bits, D):
    check(q, setup([70, 5], Hq, Hkv, D, dt, bits=bits, seed=Hq))


@pytest.mark.parametrize("ps", [1, 2, 3, 8, 16, 24, 100, 256])
@pytest.mark.parametrize("hnd", [False, True])
@pytest.mark.parametrize("bits", [16, 8])
def test_pages_that_end_inside_a_tile(q, ps, hnd, bits):
    check(q, setup([1, 15, 16, 17, 31, 33, 200, ps, ps + 1, max(ps - 1, 1)], 8, 2, 64, ps=ps, hnd=hnd,
                   bits=bits, seed=ps))


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [1] * 40, [0, 700, 0, 1, 0], list(range(40)),
                                  [5000], [3] * 700, [1000, 1, 1, 1, 1, 1, 1, 2000]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_lengths(q, lens, dt):
    check(q, setup(lens, 4, 2, 64, dt, seed=len(lens)))


@pytest.mark.parametrize("L", [1, 4, 5, 63, 64, 65, 66, 70, 1000])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (64, 0), (64, 1), (64, 4), (60, 100),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (3, 2 ** 31 - 1)])
def test_window_and_sinks(q, L, window, sinks):
    check(q, setup([L, 17, 0, 300], 8, 2, 64, ps=7, seed=L), window=window, sinks=sinks)


def test_hidden_tokens_are_not_read(q):
    """NaN between sinks and window changes nothing."""
    for bits in (16, 8):
        d = setup([500, 90], 8, 2, 64, ps=9, bits=bits)
        want = check(q, d, window=50, sinks=4)
        for b, n in enumerate([500, 90]):
            t = torch.arange(4, n - 50, device="cuda")
            p, o = d["tab"][b].long()[t // 9], t % 9
            if bits == 16:
                d["kc"][p, o] = float("nan")
                d["vc"][p, o] = float("nan")
            else:
                d["ks"][p, o] = float("nan")
                d["vs"][p, o] = float("nan")
        assert torch.equal(run(q, d, window=50, sinks=4), want)


@pytest.mark.parametrize("dt,bits", [(BF, 16), (F32, 16), (BF, 8)])
def test_long(q, dt, bits):
    check(q, setup([20000, 3, 9000], 8, 1, 128, dt, ps=32, bits=bits))


def test_large_scores_and_one_hot(q):
    """One token takes all the weight; scores of hundreds neither overflow nor lose the rest."""
    d = setup([300], 4, 1, 64, F32)
    d["kc"][d["tab"][0, 3].long(), 2] = (d["q"][0].mean(0) * 64).to(BF)
    check(q, d, scale=2.0)
    check(q, d, scale=-3.0)
    check(q, d, scale=0.0)


def test_infinite_scores(q):
    """A visible score of minus infinity has no weight, all of them give an empty row; a visible
    NaN makes its rows NaN and no others."""
    d = setup([40, 40], 4, 2, 64, F32, junk=False)
    d["q"].abs_()
    page = d["tab"][0].long()
    d["kc"][page, :, 0, 0] = -float("inf")             # every key of head 0, sequence 0
    d["kc"][d["tab"][1, 0].long(), 5, 1, 0] = -float("inf")
    o = run(q, d)
    assert (o[0, :2] == 0).all() and o.isfinite().all()
    d["kc"][d["tab"][1, 1].long(), 3, 0, 7] = float("nan")
    p = run(q, d)
    assert p[1, :2].isnan().all() and torch.equal(p[0], o[0]) and torch.equal(p[1, 2:], o[1, 2:])


def test_bad_lengths_and_pages(q):
    d = setup([50, 60, 70, 80], 8, 2, 64)
    want = check(q, d)
    d["lens"][1], d["lens"][3] = -1, d["tab"].shape[1] * 16 + 1
    o = run(q, d)
    assert q.qvla_read_error_word(clear=True) == q.QVLA_DEVERR_CACHE_RANGE
    assert (o[[1, 3]] == 0).all()
    # the order of the sums may differ with the lengths, the bound does not
    R.within(o[[0, 2]], want[[0, 2]].double(), 2.0 ** -7 * want[[0, 2]].double().abs() + 2.0 ** -7)
    d = setup([50, 60, 70, 80], 8, 2, 64)
    d["tab"][0, 1], d["tab"][2, 0] = d["kc"].shape[0], -5
    d["tab"][3] = 2 ** 31 - 1
    check(q, d, error=q.QVLA_DEVERR_CACHE_RANGE)


def test_pitches_given_output_and_workspace(q):
    d = setup([90, 33, 5], 8, 2, 64)
    want = check(q, d)
    wide = torch.zeros(3, 1024, dtype=BF, device="cuda")
    wide[:, :512] = d["q"].flatten(1)
    d["q"] = wide[:, :512].unflatten(1, (8, 64))
    buf = torch.full((3, 1024), 7.0, dtype=BF, device="cuda")
    ws = torch.full((q.qvla_paged_attn_workspace_bytes(8, 2, 64),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        run(q, d, out=buf[:, 256:768].unflatten(1, (8, 64)), workspace=ws)
        assert torch.equal(buf[:, 256:768].reshape(3, 8, 64), want)
        assert (buf[:, :256] == 7).all() and (buf[:, 768:] == 7).all()


@pytest.mark.parametrize("lens", [[700], [3, 900, 0, 40, 16], [20] * 64])
@pytest.mark.parametrize("dt", [BF, F32])
def test_in_place(q, lens, dt):
    """out may be q: a row's last reader is done before it is written, however it is split."""
    d = setup(lens, 24, 2, 64, dt)
    want = check(q, d)
    assert run(q, d, out=d["q"]) is d["q"]
    assert torch.equal(d["q"], want)


def test_shared_pages_and_equal_calls(q):
    """Sequences may share pages; equal calls give equal bits."""
    d = setup([200, 200], 8, 2, 64)
    d["tab"][1] = d["tab"][0]
    d["q"][1] = d["q"][0]
    a = check(q, d)
    R.within(a[1], a[0].double(), 2.0 ** -7 * a[0].double().abs() + 2.0 ** -9)
    for _ in range(5):
        assert torch.equal(run(q, d), a)


def test_cache_past_32_bits(q):
    """Pages past 2^32 bytes and 2^31 values."""
    D, H, ps = 256, 8, 64
    pages = 2 ** 31 // (D * H * ps) + 10
    kc = torch.zeros(pages, ps, H, D, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    kc[-4:].normal_(generator=gen(1))
    vc[-4:].normal_(generator=gen(2))
    d = dict(q=torch.randn(1, 16, D, device="cuda", generator=gen(3)).to(BF), kc=kc, vc=vc, ks=None, vs=None,
             tab=torch.tensor([[pages - 1, pages - 3, 0, pages - 2]], dtype=torch.int32, device="cuda"),
             lens=torch.tensor([250], dtype=torch.int32, device="cuda"))
    check(q, d)


def test_wide_batch(q):
    """More sequences than any block has threads."""
    lens = [(i * 37) % 23 for i in range(3000)]
    d = setup(lens, 2, 1, 16)
    o = run(q, d)
    pick = torch.arange(0, 3000, 97, device="cuda")
    ro, rl, so, sl = R.paged_attn(d["q"][pick], d["kc"], d["vc"], d["tab"][pick], d["lens"][pick], 0.25)
    R.within(o[pick], ro, so)


def test_graph_replay_with_growing_lengths(q):
    """Lengths and pages are read on the device: one graph serves every step.  Two graphs with a
    workspace each may run at the same time."""
    d = setup([500, 20, 0], 8, 2, 128, junk=False, spare=8)
    outs = [torch.empty_like(d["q"]) for _ in range(2)]
    wss = [torch.empty(q.qvla_paged_attn_workspace_bytes(8, 2, 128), dtype=torch.uint8, device="cuda")
           for _ in range(2)]
    run(q, d)
    torch.cuda.synchronize()
    graphs = []
    for o, ws in zip(outs, wss):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(q, d, out=o, workspace=ws)
        graphs.append(g)
    side = torch.cuda.Stream()
    for step in range(4):
        d["lens"] += torch.tensor([-70, 5, 9], dtype=torch.int32, device="cuda")
        want = check(q, d)
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_side_stream(q):
    d = setup([300, 70], 8, 2, 128)
    want = run(q, d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = [run(q, d, stream=st) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_lse_joins_two_caches(q):
    """Attention over a whole cache equals its two halves joined by their lse."""
    d = setup([64, 96], 8, 2, 64, F32)
    whole = run(q, d)
    parts, lses = [], []
    for lo, n in ((0, [32, 32]), (2, [32, 64])):
        e = dict(d, tab=d["tab"][:, lo:].contiguous(), lens=torch.tensor(n, dtype=torch.int32, device="cuda"))
        l = torch.empty(2, 8, device="cuda")
        parts.append(run(q, e, lse=l).double())
        lses.append(l.double())
    w = torch.softmax(torch.stack(lses), 0)[..., None]
    _, _, so, _ = R.paged_attn(d["q"], d["kc"], d["vc"], d["tab"], d["lens"], 64 ** -0.5)
    R.within(whole, w[0] * parts[0] + w[1] * parts[1], 3 * so)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq", [8, 20])
@pytest.mark.parametrize("bits", [16, 8])
def test_probabilities_lose_nothing_that_shows(q, D, Hq, bits):
    """bf16 queries: the output takes one rounding of its own, and the probabilities none that is
    near it, however much the values cancel."""
    d = setup([2, 3, 5, 17, 200, 1500], Hq, 2, D, bits=bits, seed=D + Hq)
    if bits == 8:
        d["vc"].clamp_(min=-127)                       # so that the codes have magnitudes
    o = run(q, d)
    args = d["tab"], d["lens"], D ** -0.5, 0, 0, d["ks"], d["vs"]
    ro, _, so, _ = R.paged_attn(d["q"].float(), d["kc"], d["vc"], *args)
    mag = R.paged_attn(d["q"].float(), d["kc"], d["vc"].abs(), *args)[0]
    # so is the bound of fp32 probabilities; cut to 8 bits one leaves less than 2^-7 of itself,
    # and the bf16 rounding of that is off by 2^-8 of it
    R.within(o, ro, so + 2.0 ** -15 * mag, "o")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 20), (256, 4)])
def test_infinite_values(q, dt, D, Hq):
    """A visible infinite value makes its component infinite (of both signs: NaN), also where its
    token has all the weight, and changes no other."""
    d = setup([40, 1], Hq, 2, D, dt, junk=False)
    want, G, inf = run(q, d), Hq // 2, float("inf")
    p, one = d["tab"][0].long(), d["tab"][1, 0].long()
    d["vc"][p[1], 3, 0, 7] = d["vc"][p[0], 5, 0, 11] = d["vc"][one, 0, 1, 3] = inf
    d["vc"][p[0], 2, 0, 9] = d["vc"][p[2], 5, 0, 11] = -inf
    o = run(q, d)
    assert (o[0, :G, 7] == inf).all() and (o[0, :G, 9] == -inf).all() and o[0, :G, 11].isnan().all()
    assert (o[1, G:, 3] == inf).all()
    o[0, :G, [7, 9, 11]], o[1, G:, 3] = want[0, :G, [7, 9, 11]], want[1, G:, 3]
    assert torch.equal(o, want)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 20), (256, 4)])
def test_infinite_scale_of_a_value(q, dt, D, Hq):
    """The same in an 8-bit cache: scale times code, NaN where the code is 0."""
    d = setup([40, 1], Hq, 2, D, dt, bits=8, junk=False)
    want, G = run(q, d), Hq // 2
    p, one = d["tab"][0].long(), d["tab"][1, 0].long()
    d["vc"][p[1], 3, 0, 6] = 0
    d["vs"][p[1], 3, 0] = d["vs"][one, 0, 1] = float("inf")
    o = run(q, d)
    for b, heads, code in ((0, slice(0, G), d["vc"][p[1], 3, 0]), (1, slice(G, Hq), d["vc"][one, 0, 1])):
        value = (code.float() * float("inf")).to(dt).expand(G, D)
        assert torch.equal(o[b, heads].isnan(), value.isnan())
        assert torch.equal(o[b, heads].nan_to_num(7.0), value.nan_to_num(7.0))
    assert torch.equal(o[0, G:], want[0, G:]) and torch.equal(o[1, :G], want[1, :G])


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_query_of_any_payload(q, D, bits):
    """A NaN in an fp32 query makes its head NaN, whichever of its bits say so, and no other head."""
    d = setup([40, 3], 4, 2, D, F32, bits=bits, junk=False)
    d["kc"][..., 7] = -1
    want = run(q, d)
    for payload in (0x7fc00000, 0x7f800001, 0x7f80ffff, -0x7fffff):          # the last: 0xff800001
        d["q"][0, 1].view(torch.int32)[7] = payload
        o = run(q, d)
        assert o[0, 1].isnan().all()
        o[0, 1] = want[0, 1]
        assert torch.equal(o, want)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bits", [16, 8])
def test_probabilities_that_vanish(q, dt, bits):
    """Beside a token that takes all the weight and whose values are 0, the others' share: a
    probability counts as long as it is 2^-126 of the largest one, or more."""
    D = 128
    d = setup([30, 3, 2], 8, 2, D, dt, bits=bits, junk=False)
    for b in range(3):
        d["vc"][d["tab"][b, 0].long(), 1] = 0
        d["kc"][d["tab"][b, 0].long(), 1] = 3
    d["q"].abs_()
    for scale in (0.05, 0.2, 0.5, 1.5):
        o = run(q, d, scale=scale)
        ro, _, so, _ = R.paged_attn(d["q"], d["kc"], d["vc"], d["tab"], d["lens"], scale, 0, 0, d["ks"], d["vs"])
        # each of the 30 tokens may lose 2^-126 of its value, twice: cut off, or left in parts
        most = d["vc"].abs().max().item() if bits == 16 else 128 * d["vs"].max().item()
        R.within(o, ro, so + 30 * 2.0 ** -125 * most, f"scale {scale}")
