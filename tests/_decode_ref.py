"""fp64 restatements of the decode-step operators, and the error bounds their
tests use.  Every bound is a count of roundings: U = 2**-24 per fp32 operation
relative to the magnitudes it adds up, half a step of the output's type for the
one rounding at the end."""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(out, ref, slack, what=""):
    """|out - ref| <= slack + the rounding of the output (its own error included)."""
    lim = slack + half_step(out.dtype) * (ref.abs() + slack)
    if out.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -134            # half of the smallest subnormal step
    err = (out.double() - ref).abs()
    bad = ~(err <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values outside, worst "
                           f"{(err / lim)[bad].max():.4g} x the bound, at {bad.nonzero()[0].tolist()}: "
                           f"{out[bad][0].item()!r} for {ref[bad][0].item()!r}")


def unpack(wq, signed):
    """codes [N, K] of packed bytes: the low nibble comes first."""
    u = torch.stack([wq & 15, wq >> 4], 2).flatten(1).double()
    return torch.where(u >= 8, u - 16, u) if signed else u


def gemv(x, wq, scale, zero=None, bias=None):
    """(y, slack): y = x W^T + b in fp64; slack: K + 4 fp32 operations on the sum of magnitudes
    (each product is exact, each group's sum is scaled once and added)."""
    N, K = wq.shape[0], 2 * wq.shape[1]
    G = K // scale.shape[1]
    w = unpack(wq, zero is None).view(N, K // G, G)
    if zero is not None:
        w = w - (zero & 15).double()[:, :, None]
    w = (w * scale.double()[:, :, None]).view(N, K)
    y, mag = x.double() @ w.T, x.double().abs() @ w.abs().T
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    return y, (K + 4) * U * mag


def norm_rope(x, w, cos, sin, rot, interleaved, eps):
    """x [T, H, D] -> (y, slack).  The sum of D squares and the mean cost at most D + 2
    roundings of a positive sum, halved by the root; root, reciprocal, two products and three
    operations of the rotation come to fewer than 10 more."""
    x = x.double()
    if w is not None:
        x = x * w.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    mag = x.abs()
    if rot:
        y, ym = x.clone(), mag.clone()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
               (slice(0, rot // 2), slice(rot // 2, rot))
        c, s = cos.double()[:, None, :], sin.double()[:, None, :]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        ym[..., a] = mag[..., a] * c.abs() + mag[..., b] * s.abs()
        ym[..., b] = mag[..., b] * c.abs() + mag[..., a] * s.abs()
        x, mag = y, ym
    D = x.shape[-1]
    return x, ((D + 2) / 2 + 10) * U * mag


def paged_attn(q, k_cache, v_cache, table, lens, scale, window=0, sinks=0, k_scale=None,
               v_scale=None):
    """(o, lse, slack of o, slack of lse), token by token from the definition.  A score is off
    by (D + 3) U of its magnitudes, which moves every probability by that factor twice (its own
    and the sum's); exponential, sums over n tokens and products add (n + 16) U; for bf16 the
    probabilities take one more half step."""
    B, Hq, D = q.shape
    pages, ps, Hkv, _ = k_cache.shape
    o = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -torch.inf, dtype=torch.float64, device=q.device)
    so, sl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n = int(lens[b])
        t = torch.arange(max(n, 0), device=q.device)
        if n <= 0 or n > table.shape[1] * ps:
            continue
        if window:
            t = t[(t >= n - window) | (t < sinks)]
        page, off = table[b, (t // ps)].long(), t % ps
        ok = (page >= 0) & (page < pages)
        page, off = page[ok], off[ok]
        if not len(page):
            continue
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            k, v = k_cache[page, off, hk].double(), v_cache[page, off, hk].double()
            if k_scale is not None:
                k = k * k_scale[page, off, hk].double()[:, None]
                v = v * v_scale[page, off, hk].double()[:, None]
            s = k @ q[b, h].double() * scale
            ds = (D + 3) * U * (k.abs() @ q[b, h].double().abs()).max() * abs(scale)
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[b, h])
            o[b, h] = p @ v
            rel = 2 * ds + (len(page) + 16) * U + (half_step(torch.bfloat16) if
                                                  q.dtype == torch.bfloat16 else 0)
            so[b, h] = rel * (p @ v.abs())
            sl[b, h] = ds + (len(page) + 16) * U + 4 * U * lse[b, h].abs()
    return o, lse, so, sl
