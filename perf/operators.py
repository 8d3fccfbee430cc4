"""The operators of a decode step around the packed linears, as they are measured.

Three operators, each in two forms that take the same state and return the
same outputs:

  gemv   y = x W^T + b with 4-bit weight codes and one scale (optionally one
         zero point) per group of inputs, activations kept in 16 or 32 bits
  rope   RMS norm of every query and key head and the position rotation in one
         pass, keys and values written into a paged cache
  attn   attention of one new token per sequence over that paged cache, with
         an optional sliding window and always-visible first tokens

`run` computes them in elementary torch operations (fp32, rounded once at the
end) or, with `own` set, through the package's entry points.
"""
import functools
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0


def listed():
    return [
        # gate / up projection of the action head for one token: the smallest call,
        # launch latency counts
        dict(name="gemv 1x1024->4096", op="gemv", M=1, K=1024, N=4096, group=64, zero=False,
             bias=True, x="bf16", y="bf16", s="f32"),
        # the backbone's down projection in a decode step of one sequence
        dict(name="gemv 1x16384->2048", op="gemv", M=1, K=16384, N=2048, group=128, zero=True,
             bias=False, x="bf16", y="bf16", s="bf16"),
        # a small head kept in fp32 (state and action projections), odd batch, finest groups
        dict(name="gemv 7x1536->6144 f32", op="gemv", M=7, K=1536, N=6144, group=32, zero=False,
             bias=True, x="f32", y="f32", s="f32"),
        # a vocabulary head for sixteen sequences, logits in fp32
        dict(name="gemv 16x2048->131072", op="gemv", M=16, K=2048, N=131072, group=128, zero=True,
             bias=False, x="bf16", y="f32", s="bf16"),
        # one decode step of the backbone (width 2048 = 8 heads of 256, one shared key head)
        dict(name="rope 1x(8+1)x256", op="rope", T=1, Hq=8, Hkv=1, D=256, rot=256, inter=False,
             x="bf16", page=16, first=900, pad=0, hnd=False),
        # its prefill
        dict(name="rope 1024x(8+1)x256", op="rope", T=1024, Hq=8, Hkv=1, D=256, rot=256,
             inter=False, x="bf16", page=64, first=0, pad=0, hnd=False),
        # the action head's rows (512 x 1536) in fp32, pairs side by side, half of each head turned
        dict(name="rope 512x(12+12)x128 f32", op="rope", T=512, Hq=12, Hkv=12, D=128, rot=64,
             inter=True, x="f32", page=16, first=100000, pad=0, hnd=True),
        # a long prefill with grouped heads, odd length, some padding rows that own no slot
        dict(name="rope 16381x(32+8)x128", op="rope", T=16381, Hq=32, Hkv=8, D=128, rot=128,
             inter=False, x="bf16", page=16, first=0, pad=37, hnd=False),
        # one robot's context: prefix of about a thousand tokens, one shared key head
        dict(name="attn 1x8/1x256 L1040", op="attn", B=1, Hq=8, Hkv=1, D=256, L=1040, page=16,
             window=0, sinks=0, x="bf16", bits=16, hnd=False),
        # a batch of ragged contexts, one of them still empty
        dict(name="attn 32x32/8x128 L8192", op="attn", B=32, Hq=32, Hkv=8, D=128, L=8192, page=16,
             window=0, sinks=0, x="bf16", bits=16, hnd=False),
        # one long context: the split over its length has to fill the card
        dict(name="attn 1x32/8x128 L131072", op="attn", B=1, Hq=32, Hkv=8, D=128, L=131072,
             page=64, window=0, sinks=0, x="bf16", bits=16, hnd=True),
        # sliding window with sinks over an 8-bit cache, pages that end inside a tile
        dict(name="attn 64x16/2x64 W2000 8bit", op="attn", B=64, Hq=16, Hkv=2, D=64, L=16000,
             page=24, window=2000, sinks=4, x="f32", bits=8, hnd=False),
    ]


@functools.lru_cache(maxsize=None)
def _package():
    from w4a4_post_quantization_zigzag_b200 import qvla
    return qvla


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "rope", "attn"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemv":
        group = rng.choice([32, 64, 128, 256])
        K = group * max(1, _log(rng, 256, 16384) // group)
        N = _log(rng, 64, min(131072, 2 ** 28 // K))
        return dict(op=op, M=rng.randint(1, 16), K=K, N=N, group=group,
                    zero=rng.random() < 0.5, bias=rng.random() < 0.5, x=x,
                    y=rng.choice(["bf16", "f32"]), s=rng.choice(["bf16", "f32"]))
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([1, 8, 16, 24, 64, 256])
    if op == "rope":
        T = _log(rng, 1, 2 ** 25 // ((Hq + 2 * Hkv) * D))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 32 * 16]),
                    inter=rng.random() < 0.3, x=x, page=page, first=_log(rng, 1, 200000) - 1,
                    pad=rng.choice([0, T // 8]), hnd=rng.random() < 0.3)
    B = _log(rng, 1, 64)
    most = 2 ** 27 // (B * Hkv * D)
    L = _log(rng, 1, min(131072, most))
    window = rng.choice([0, 0, _log(rng, 1, max(2, L))])
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, L=L, page=page, window=window,
                sinks=rng.choice([0, 4, 33]) if window else 0, x=x, bits=rng.choice([16, 16, 8]),
                hnd=rng.random() < 0.3)


def lengths(case):
    """Tokens in each sequence's cache: the longest, then a spread of shorter ones;
    from eight sequences on, one has nothing yet."""
    B, L = case["B"], case["L"]
    n = [L] + [1 + int((L - 1) * ((b * 0.6180339887) % 1.0)) for b in range(1, B)]
    if B >= 8:
        n[3] = 0
    return n


def visible(case):
    """Tokens each sequence's new token sees."""
    w, s = case["window"], case["sinks"]
    return [n if not w or n <= w + s else w + s for n in lengths(case)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    rand = lambda *s: torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    st = dict(case)
    dt = TYPES[case["x"]]
    if case["op"] == "gemv":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        st["wq"] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        st["w_scale"] = (0.002 + 0.006 * rand(N, K // G)).to(TYPES[case["s"]])
        st["w_zero"] = (torch.randint(4, 12, (N, K // G), dtype=torch.uint8, device="cuda",
                                      generator=g) if case["zero"] else None)
        st["b"] = randn(N) * 0.01 if case["bias"] else None
        st["xin"] = randn(M, K).to(dt)
        return st
    Hq, Hkv, D, ps = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "rope":
        T, rot, first = case["T"], case["rot"], case["first"]
        n = T - case["pad"]
        qkv = randn(T, (Hq + 2 * Hkv) * D).to(dt)
        st["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        st["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        st["q_norm"], st["k_norm"] = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D)
        pos = torch.arange(first, first + T, device="cuda", dtype=torch.int32)
        st["positions"] = pos
        inv = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        a = torch.arange(first + T, device="cuda", dtype=torch.float64)[:, None] * inv
        st["rope_table"] = torch.cat([a.cos(), a.sin()], 1).float()
        pages = -(-n // ps) + 2
        # one page more than the cache has, where the plain form puts what owns no slot
        shape = (pages + 1, Hkv, ps, D) if case["hnd"] else (pages + 1, ps, Hkv, D)
        for c in ("k_store", "v_store"):
            t = randn(*shape).to(torch.bfloat16)
            st[c] = t.permute(0, 2, 1, 3) if case["hnd"] else t
        st["k_cache"], st["v_cache"] = st["k_store"][:pages], st["v_store"][:pages]
        order = torch.randperm(pages, device="cuda", generator=g)
        i = torch.arange(n, device="cuda")
        st["slots"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        st["slots"][:n] = (order[i // ps] * ps + i % ps).int()
        return st
    B = case["B"]
    n = lengths(case)
    need = [-(-v // ps) for v in n]
    pages = sum(need) + 1
    order = torch.randperm(pages, device="cuda", generator=g).int()
    tab = torch.full((B, max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        tab[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    st["page_table"] = tab
    st["seq_lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    st["q"] = randn(B, Hq, D).to(dt)
    shape = (pages, Hkv, ps, D) if case["hnd"] else (pages, ps, Hkv, D)
    for c in ("k", "v"):
        if case["bits"] == 8:
            t = torch.empty(shape, dtype=torch.int8, device="cuda")
            t.random_(-127, 128, generator=g)
            st[c + "_scale"] = 0.005 + 0.02 * rand(*shape[:3])
        else:
            t = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            st[c + "_scale"] = None
        if case["hnd"]:
            t = t.permute(0, 2, 1, 3)
            if case["bits"] == 8:
                st[c + "_scale"] = st[c + "_scale"].permute(0, 2, 1)
        st[c + "_cache"] = t
    return st


# ------------------------------------------------------------- plain forms
def _plain_gemv(st):
    N, K, G = st["N"], st["K"], st["group"]
    wq = st["wq"]
    u = torch.stack([wq & 15, wq >> 4], 2).view(N, K // G, G)
    if st["w_zero"] is not None:
        w = u.float() - st["w_zero"].float()[:, :, None]
    else:
        w = (u ^ 8).float() - 8.0
    w = (w * st["w_scale"].float()[:, :, None]).view(N, K)
    y = st["xin"].float() @ w.T
    if st["b"] is not None:
        y = y + st["b"]
    return y.to(TYPES[st["y"]])


def _plain_norm_rope(x, w, cos, sin, rot, inter):
    """x [T, H, D]: RMS norm over D, then the rotation of its first `rot` values."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    cos, sin = cos[:, None, :], sin[:, None, :]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_rope(st):
    rot, inter, ps = st["rot"], st["inter"], st["page"]
    rows = st["rope_table"][st["positions"].long()]
    cos, sin = rows[:, :rot // 2], rows[:, rot // 2:]
    q = _plain_norm_rope(st["q"], st["q_norm"], cos, sin, rot, inter).to(st["q"].dtype)
    k = _plain_norm_rope(st["k"], st["k_norm"], cos, sin, rot, inter)
    slot = st["slots"].long()
    page = torch.where(slot < 0, st["k_cache"].shape[0], slot // ps)
    off = torch.where(slot < 0, 0, slot % ps)
    st["k_store"][page, off] = k.to(torch.bfloat16)
    st["v_store"][page, off] = st["v"].to(torch.bfloat16)
    return q, st["k_cache"], st["v_cache"]


def _plain_attn(st):
    B, Hq, Hkv, D = st["B"], st["Hq"], st["Hkv"], st["D"]
    tab = st["page_table"].long().clamp(min=0)
    def rows(c):  # [B, Hkv, tokens, D] in fp32
        x = st[c + "_cache"][tab].float()
        if st["bits"] == 8:
            x = x * st[c + "_scale"][tab][..., None]
        return x.flatten(1, 2).transpose(1, 2)
    q = st["q"].float().view(B, Hkv, Hq // Hkv, D)
    s = (q @ rows("k").transpose(2, 3)) / math.sqrt(D)
    n = st["seq_lens"].long()[:, None]
    t = torch.arange(s.shape[-1], device=s.device)[None, :]
    see = t < n
    if st["window"]:
        see = see & ((t >= n - st["window"]) | (t < st["sinks"]))
    see = see[:, None, None, :]
    s = torch.where(see, s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ rows("v")) / torch.where(total == 0, 1.0, total)
    return o.view(B, Hq, D).to(st["q"].dtype)


def run(st):
    op = st["op"]
    if own:
        Q = _package()
        if op == "gemv":
            return Q.qvla_w4a16_gemv(st["xin"], st["wq"], st["w_scale"], st["w_zero"], st["b"],
                                     out_dtype=TYPES[st["y"]])
        if op == "rope":
            q = Q.qvla_qk_norm_rope(st["q"], st["k"], st["v"], st["q_norm"], st["k_norm"],
                                    st["rope_table"], st["positions"], st["slots"],
                                    st["k_cache"], st["v_cache"], eps=EPS,
                                    interleaved=st["inter"])
            return q, st["k_cache"], st["v_cache"]
        return Q.qvla_paged_attn_decode(st["q"], st["k_cache"], st["v_cache"], st["page_table"],
                                        st["seq_lens"], window=st["window"], sinks=st["sinks"],
                                        k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"gemv": _plain_gemv, "rope": _plain_rope, "attn": _plain_attn}[op](st)


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "gemv":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        per_group = size[case["s"]] + (1 if case["zero"] else 0)
        return {"bytes": N * K // 2 + N * (K // G) * per_group + M * K * size[case["x"]]
                + M * N * size[case["y"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    e = size[case["x"]]
    if case["op"] == "rope":
        T, n = case["T"], case["T"] - case["pad"]
        return {"bytes": T * Hq * D * e * 2 + n * 2 * Hkv * D * (e + 2) + T * (4 * case["rot"] + 8)
                + 8 * D,
                "flops": T * (Hq + Hkv) * D * 7}
    seen = sum(visible(case))
    row = D * (2 if case["bits"] == 16 else 1) + (4 if case["bits"] == 8 else 0)
    return {"bytes": seen * Hkv * 2 * row + case["B"] * Hq * D * e * 2 + 4 * case["B"]
            + 4 * (seen // case["page"] + 1),
            "flops": 4 * seen * Hq * D}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    return {"gemv": _exact_gemv, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](st)


def _exact_gemv(st):
    """y[m, n] = sum over the groups of s (sum u x - z sum x), a block of rows at a time."""
    N, K, G = st["N"], st["K"], st["group"]
    x = st["xin"].double().view(-1, K // G, G)
    sx = x.sum(2)                                            # [M, groups]
    parts = []
    step = max(1, 2 ** 25 // K)
    for n0 in range(0, N, step):
        wq = st["wq"][n0:n0 + step].int()
        u = torch.empty(wq.shape[0], K, dtype=torch.float64, device=wq.device)
        u[:, 0::2], u[:, 1::2] = wq % 16, wq // 16
        if st["w_zero"] is None:
            u[u >= 8] -= 16
        dots = torch.einsum("mgk,ngk->mng", x, u.view(-1, K // G, G))
        if st["w_zero"] is not None:
            dots = dots - sx[:, None, :] * st["w_zero"][n0:n0 + step].double()
        parts.append((dots * st["w_scale"][n0:n0 + step].double()).sum(2))
    y = torch.cat(parts, 1)
    return y if st["b"] is None else y + st["b"].double()


def _exact_rope(st):
    """Pairs as complex numbers times e^{i angle}, the angle's cosine and sine as the table
    holds them."""
    rot, half = st["rot"], st["rot"] // 2
    rows = st["rope_table"].double()[st["positions"].long()]
    turn = torch.complex(rows[:, :half], rows[:, half:])[:, None, :]

    def turned(x, w):
        x = x.double()
        x = w.double() * x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        y = x.clone()
        if st["inter"]:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (half, 2)).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :half], x[..., half:rot]) * turn
            y[..., :half], y[..., half:rot] = z.real, z.imag
        return y

    q, k = turned(st["q"], st["q_norm"]), turned(st["k"], st["k_norm"])
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    own_slot = st["slots"] >= 0
    slot = st["slots"][own_slot].long()
    page, off = slot.div(st["page"], rounding_mode="floor"), slot.remainder(st["page"])
    kc[page, off] = k[own_slot]
    vc[page, off] = st["v"][own_slot].double()
    return q, kc, vc


def _exact_attn(st):
    """One sequence and key head at a time, over the tokens it sees."""
    B, Hq, Hkv, D, ps = st["B"], st["Hq"], st["Hkv"], st["D"], st["page"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths(st)):
        if n == 0:
            continue
        tok = torch.arange(n, device="cuda")
        if st["window"]:
            tok = tok[(tok < st["sinks"]) | (tok + st["window"] >= n)]
        page, off = st["page_table"][b].long()[tok // ps], tok % ps
        for h in range(Hkv):
            k, v = st["k_cache"][page, off, h].double(), st["v_cache"][page, off, h].double()
            if st["bits"] == 8:
                k = k * st["k_scale"][page, off, h].double()[:, None]
                v = v * st["v_scale"][page, off, h].double()[:, None]
            G = Hq // Hkv
            s = st["q"][b, h * G:(h + 1) * G].double() @ k.T * D ** -0.5
            out[b, h * G:(h + 1) * G] = torch.softmax(s, 1) @ v
    return out
