"""Norm, rotation and cache write of query and key heads on the GPU against fp64."""
import pytest
import torch

import _decode_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


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


def inv_freq(rot, theta=10000.0):
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def setup(T, Hq, Hkv, D, dt, ps=16, pages=None, bits=16, hnd=False, seed=0):
    """Fused qkv rows, norms, a cache full of marks, and distinct slots in random order."""
    g = gen(seed)
    qkv = (torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda", generator=g) * 2).to(dt)
    a, b = Hq * D, (Hq + Hkv) * D
    d = dict(q=qkv[:, :a].unflatten(1, (Hq, D)), k=qkv[:, a:b].unflatten(1, (Hkv, D)),
             v=qkv[:, b:].unflatten(1, (Hkv, D)))
    d["qn"], d["kn"] = (1 + 0.3 * torch.randn(2, D, device="cuda", generator=g)).unbind(0)
    d["qn"], d["kn"] = d["qn"].contiguous(), d["kn"].contiguous()
    pages = pages or -(-T // ps) + 2
    shape = (pages, Hkv, ps, D) if hnd else (pages, ps, Hkv, D)
    perm = (lambda t: t.transpose(1, 2)) if hnd else (lambda t: t)
    ct = BF if bits == 16 else torch.int8
    d["kc"], d["vc"] = (perm(torch.full(shape, m, dtype=ct, device="cuda")) for m in (77, 55))
    d["ks"] = d["vs"] = None
    if bits == 8:
        d["ks"], d["vs"] = (perm(torch.full(shape[:3], m, device="cuda")) for m in (3.0, 5.0))
    d["slots"] = torch.randperm(pages * ps, device="cuda", generator=g)[:T].int()
    return d


def run(q, d, table, pos, inter=False, **kw):
    return q.qvla_qk_norm_rope(d["q"], d["k"], d["v"], d["qn"], d["kn"], table, pos, d["slots"],
                               d["kc"], d["vc"], d["ks"], d["vs"], eps=EPS, interleaved=inter, **kw)


def check_cache(d, ref, slack, slots, which):
    """Written slots hold the reference rows, every other slot its mark."""
    c, s, mark, smark = ((d["kc"], d["ks"], 77, 3.0) if which == "k" else (d["vc"], d["vs"], 55, 5.0))
    ps = c.shape[1]
    ok = (slots >= 0) & (slots < c.shape[0] * ps)
    sl = slots[ok].long()
    got = c[sl // ps, sl % ps]
    if s is None:
        R.within(got, ref[ok], slack[ok], which)
    else:
        sc = s[sl // ps, sl % ps].double()
        mx, sx = ref[ok].abs().amax(-1), slack[ok].amax(-1)
        # the largest value's error, and the rounding of the division by 127
        assert ((sc - mx / 127).abs() <= (sx + 2 * R.U * mx) / 127).all()
        err = (got.double() * sc[..., None] - ref[ok]).abs()
        # a code is off by half a step, plus its value's error and three roundings of a quotient
        # of at most 128 steps
        assert (err <= sc[..., None] * (0.5 + 128 * 3 * R.U) + 2 * slack[ok]).all(), which
        assert int(got.max()) <= 127 and int(got.abs().amax(-1).min()) == 127
    left = torch.ones(c.shape[0], ps, dtype=torch.bool, device="cuda")
    left[sl // ps, sl % ps] = False
    assert (c[left] == mark).all(), f"{which}: a slot that no token owns was written"
    if s is not None:
        assert (s[left] == smark).all()


def check(q, d, table, pos, rot, inter=False, **kw):
    k0 = d["k"].clone()
    v0 = d["v"].clone()
    rows = table[pos.long()]
    cos, sin = rows[:, :rot // 2], rows[:, rot // 2:]
    rq, sq = R.norm_rope(d["q"], d["qn"], cos, sin, rot, inter, EPS)
    rk, sk = R.norm_rope(k0, d["kn"], cos, sin, rot, inter, EPS)
    out = run(q, d, table, pos, inter, **kw)
    R.within(out, rq, sq, "q")
    check_cache(d, rk, sk, d["slots"], "k")
    check_cache(d, v0.double(), torch.zeros_like(v0, dtype=torch.float64), d["slots"], "v")
    assert q.qvla_read_error_word(clear=True) == 0
    return out


@pytest.mark.parametrize("D,rot", [(16, 16), (32, 16), (64, 64), (80, 80), (96, 48), (112, 112),
                                   (128, 128), (128, 64), (144, 96), (240, 240), (256, 256),
                                   (256, 16)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bits", [16, 8])
def test_dims_types_and_styles(q, D, rot, dt, inter, bits):
    d = setup(5, 6, 2, D, dt, ps=3, bits=bits, seed=D + rot)
    table = q.qvla_rope_table(inv_freq(rot), 40)
    check(q, d, table, torch.tensor([0, 39, 7, 1, 20], dtype=torch.int32, device="cuda"), rot, inter)


@pytest.mark.parametrize("T", [1, 2, 17, 300])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (32, 8, 128), (12, 12, 64), (1, 1, 16), (71, 1, 64),
                                      (128, 128, 128)])
@pytest.mark.parametrize("ps,hnd,bits", [(16, False, 16), (1, False, 8), (24, True, 16), (7, True, 8)])
def test_heads_tokens_and_pages(q, T, Hq, Hkv, D, ps, hnd, bits):
    d = setup(T, Hq, Hkv, D, BF, ps=ps, bits=bits, hnd=hnd, seed=T)
    table = q.qvla_rope_table(inv_freq(D), T + 100)
    pos = torch.arange(100, 100 + T, dtype=torch.int32, device="cuda")
    check(q, d, table, pos, D)


def test_far_positions(q):
    """The table's angles are formed in 64 bits: 2^-24 of the value at any position."""
    f = inv_freq(128, 5e5)
    P = 1 << 20
    table = q.qvla_rope_table(f, P)
    a = torch.arange(P, dtype=torch.float64, device="cuda")[-70000:, None] * f.cuda()
    want = torch.cat([a.cos(), a.sin()], 1)
    # half a step of the result, and of the fp64 product at 2^20 (2^-33 in the angle)
    assert ((table[-70000:].double() - want).abs() <= R.U * want.abs() + 2.0 ** -32).all()
    assert (table[0, :64] == 1).all() and (table[0, 64:] == 0).all()
    d = setup(3, 4, 2, 128, F32)
    check(q, d, table, torch.tensor([P - 1, 0, P // 2], dtype=torch.int32, device="cuda"), 128)


def test_padding_and_rows_outside(q):
    """Negative slots write nothing; a slot or a position outside sets the error bit, and the
    other tokens are served."""
    d = setup(6, 4, 2, 64, BF)
    table = q.qvla_rope_table(inv_freq(64), 10)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    d["slots"][1], d["slots"][4] = -1, -7
    check(q, d, table, pos, 64)

    d = setup(6, 4, 2, 64, BF)
    total = d["kc"].shape[0] * d["kc"].shape[1]
    d["slots"][2] = total
    d["slots"][3] = 2 ** 31 - 1
    d["slots"][5] = total - 1
    rows = table[pos.long()]
    rq, sq = R.norm_rope(d["q"], d["qn"], rows[:, :32], rows[:, 32:], 64, False, EPS)
    rk, sk = R.norm_rope(d["k"], d["kn"], rows[:, :32], rows[:, 32:], 64, False, EPS)
    out = run(q, d, table, pos)
    assert q.qvla_read_error_word(clear=True) == q.QVLA_DEVERR_CACHE_RANGE
    R.within(out, rq, sq)
    check_cache(d, rk, sk, d["slots"], "k")

    d = setup(6, 4, 2, 64, BF)
    bad = pos.clone()
    bad[0], bad[4] = -1, 10
    out = run(q, d, table, bad)
    assert q.qvla_read_error_word(clear=True) == q.QVLA_DEVERR_CACHE_RANGE
    assert (out[[0, 4]] == 0).all()
    keep = torch.tensor([1, 2, 3, 5], device="cuda")
    R.within(out[keep], rq.new_tensor(R.norm_rope(d["q"], d["qn"], rows[:, :32], rows[:, 32:], 64, False, EPS)[0].tolist())[keep],
             R.norm_rope(d["q"], d["qn"], rows[:, :32], rows[:, 32:], 64, False, EPS)[1][keep])
    slots = d["slots"].clone()
    slots[[0, 4]] = -1
    rk, sk = R.norm_rope(d["k"], d["kn"], rows[:, :32], rows[:, 32:], 64, False, EPS)
    check_cache(d, rk, sk, slots, "k")


@pytest.mark.parametrize("dt", [BF, F32])
def test_in_place(q, dt):
    d = setup(9, 8, 2, 128, dt)
    e = dict(d, q=d["q"].clone(), k=d["k"].clone(), kc=d["kc"].clone(), vc=d["vc"].clone())
    table = q.qvla_rope_table(inv_freq(128), 10)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    k_rot = torch.empty_like(d["k"].contiguous())
    want = run(q, d, table, pos, k_out=k_rot)
    got = run(q, e, table, pos, q_out=e["q"], k_out=e["k"])
    assert got is e["q"] and torch.equal(got, want) and torch.equal(e["k"], k_rot)
    assert torch.equal(e["kc"], d["kc"]) and torch.equal(e["vc"], d["vc"])
    if dt == BF:      # the cache holds the rounded key
        ps = d["kc"].shape[1]
        s = d["slots"].long()
        assert torch.equal(d["kc"][s // ps, s % ps], k_rot)


def test_parts_left_out(q):
    """No norm, no rotation, no cache, queries or keys alone."""
    d = setup(4, 4, 2, 64, F32)
    table = q.qvla_rope_table(inv_freq(32), 10)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    rows = table[pos.long()]
    cs = rows[:, :16], rows[:, 16:]
    a, b = q.qvla_qk_norm_rope(d["q"], d["k"], q_norm=d["qn"], rope_table=table, positions=pos)
    R.within(a, *R.norm_rope(d["q"], d["qn"], *cs, 32, False, EPS))
    R.within(b, *R.norm_rope(d["k"], None, *cs, 32, False, EPS))
    a, b = q.qvla_qk_norm_rope(d["q"], None, q_norm=d["qn"], eps=0.5)
    assert b is None
    R.within(a, *R.norm_rope(d["q"], d["qn"], None, None, 0, False, 0.5))
    a, b = q.qvla_qk_norm_rope(None, d["k"])
    assert a is None and torch.equal(b, d["k"])
    assert q.qvla_qk_norm_rope(None, d["k"], d["v"], slots=d["slots"], k_cache=d["kc"].float().to(BF),
                               v_cache=d["vc"].clone()) is None
    e = setup(0, 4, 2, 64, F32)
    assert q.qvla_qk_norm_rope(e["q"], e["k"])[0].shape == (0, 4, 64)
    assert q.qvla_read_error_word(clear=True) == 0


def test_zero_rows_and_non_finite_neighbours(q):
    """A row of zeros stays zero (codes and scale too); NaN and infinity stay in their row."""
    for bits in (16, 8):
        d = setup(4, 4, 2, 64, F32, bits=bits)
        e = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in d.items()}
        e["k"][1, 0] = 0
        e["q"][1, 2] = 0
        e["q"][2, 1, 3], e["k"][3, 1, 5], e["v"][3, 0, 5] = float("nan"), float("inf"), float("nan")
        table = q.qvla_rope_table(inv_freq(64), 10)
        pos = torch.arange(4, dtype=torch.int32, device="cuda")
        a, b = run(q, d, table, pos), run(q, e, table, pos)
        assert (b[1, 2] == 0).all() and b[2, 1].isnan().all()
        same = torch.ones(4, 4, dtype=torch.bool, device="cuda")
        same[1, 2] = same[2, 1] = False
        assert torch.equal(a[same], b[same])
        ps = d["kc"].shape[1]
        s = d["slots"].long()
        ka, kb = d["kc"][s // ps, s % ps], e["kc"][s // ps, s % ps]
        assert (kb[1, 0] == 0).all()
        if bits == 8:
            assert (e["ks"][s // ps, s % ps][1, 0] == 0).all()
        for t, h in ((0, 0), (0, 1), (1, 1), (2, 0), (2, 1), (3, 0)):
            assert torch.equal(ka[t, h], kb[t, h])


def test_cache_past_32_bits(q):
    """A cache of more than 2^32 bytes and 2^31 values: its last slots."""
    D, H, ps = 256, 8, 64
    pages = 2 ** 31 // (D * H * ps) + 300
    kc = torch.zeros(pages, ps, H, D, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    d = setup(2, 8, H, D, BF)
    d["kc"], d["vc"] = kc, vc
    d["slots"] = torch.tensor([pages * ps - 1, pages * ps - 65], dtype=torch.int32, device="cuda")
    run(q, d, q.qvla_rope_table(inv_freq(D), 4), torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(vc[-1, -1], d["v"][0]) and torch.equal(vc[-2, -1], d["v"][1])
    assert int((kc[-300:] != 0).any(-1).sum()) == 2 * H and not vc[:-2].any()


def test_graph_replay(q):
    """Positions and slots are read on the device: one graph serves every step."""
    d = setup(2, 8, 2, 128, BF)
    table = q.qvla_rope_table(inv_freq(128), 64)
    pos = torch.tensor([3, 9], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 8, 128, dtype=BF, device="cuda")
    run(q, d, table, pos, q_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(q, d, table, pos, q_out=out)
    for step in range(3):
        pos += 1
        d["slots"].copy_((d["slots"] + 1) % 32)
        e = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in d.items()}
        want = run(q, e, table, pos)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(d["kc"], e["kc"]) and torch.equal(d["vc"], e["vc"])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("normed", [True, False])
def test_non_finite_rows_of_an_8_bit_cache(q, dt, D, normed):
    """A key or value row with a NaN or an infinity has no 8-bit form: codes 0 and a NaN scale, so
    that attention over it is NaN as over a bf16 cache; the other rows are what they were."""
    d = setup(5, 4, 2, D, dt, bits=8, pages=1, seed=D)
    d["slots"] = torch.arange(5, dtype=torch.int32, device="cuda")
    if not normed:
        d["kn"] = None
    table = q.qvla_rope_table(inv_freq(D), 10)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    e = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in d.items()}
    nan, inf = float("nan"), float("inf")
    e["k"][0, 1, 3], e["k"][1, 0, 5], e["k"][2, 0, D - 1] = nan, inf, -inf
    e["v"][2, 1, 0], e["v"][3, 0, D - 1], e["v"][4, 1, 2] = nan, inf, -inf
    run(q, d, table, pos)
    run(q, e, table, pos)
    for c, s, bad in (("kc", "ks", ((0, 1), (1, 0), (2, 0))), ("vc", "vs", ((2, 1), (3, 0), (4, 1)))):
        hit = torch.zeros(16, 2, dtype=torch.bool, device="cuda")
        for t, h in bad:
            hit[t, h] = True
        assert torch.equal(e[s][0].isnan(), hit) and (e[c][0][hit] == 0).all()
        assert torch.equal(e[s][0][~hit], d[s][0][~hit]) and torch.equal(e[c][0][~hit], d[c][0][~hit])
    x = torch.randn(2, 4, D, device="cuda", generator=gen(1)).to(dt)
    tab = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 5], dtype=torch.int32, device="cuda")
    o = q.qvla_paged_attn_decode(x, e["kc"], e["vc"], tab, lens, k_scale=e["ks"], v_scale=e["vs"])
    assert o[0, :2].isfinite().all() and o[0, 2:].isnan().all() and o[1].isnan().all()
    assert q.qvla_read_error_word(clear=True) == 0


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("eps", [EPS, 0.0])
def test_squares_outside_the_range_of_fp32(q, dt, D, eps):
    """Rows whose squares overflow, and (eps 0) rows whose squares vanish, beside ordinary ones; an
    infinite row stays NaN."""
    d = setup(9, 4, 2, D, dt, seed=D)
    top = torch.finfo(dt).max / 32
    scale = torch.tensor([1.0, 1e19, 1e22, 1e30, top, 1.0, 1e-19, 1e-25, 1e-30], device="cuda")[:, None, None]
    for c in "qk":
        d[c].copy_(d[c].float() * (scale if eps == 0 else scale.clamp(min=1.0)))
    table = q.qvla_rope_table(inv_freq(D), 10)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    rows = table[pos.long()]
    a, b = q.qvla_qk_norm_rope(d["q"], d["k"], None, d["qn"], d["kn"], table, pos, eps=eps)
    for y, x, w in ((a, d["q"], d["qn"]), (b, d["k"], d["kn"])):
        R.within(y, *R.norm_rope(x, w, rows[:, :D // 2], rows[:, D // 2:], D, False, eps))
    d["q"][3, 1, 5] = float("inf")
    c, _ = q.qvla_qk_norm_rope(d["q"], d["k"], None, d["qn"], d["kn"], table, pos, eps=eps)
    assert c[3, 1].isnan().any()
    c[3, 1] = a[3, 1]
    assert torch.equal(c, a)
