"""W4A16 products with group scales on the GPU against fp64."""
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
    return qvla


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weights(N, K, G, sdt=F32, zero=False, seed=0):
    g = gen(seed)
    wq = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = (0.01 + 0.05 * torch.rand(N, K // G, device="cuda", generator=g)).to(sdt)
    z = torch.randint(0, 16, (N, K // G), dtype=torch.uint8, device="cuda", generator=g) if zero else None
    return wq, s, z


def rows(M, K, dt, seed=1):
    return torch.randn(M, K, device="cuda", generator=gen(seed)).to(dt)


def check(q, x, wq, s, z=None, bias=None, ydt=None, **kw):
    y = q.qvla_w4a16_gemv(x, wq, s, z, bias, out_dtype=ydt, **kw)
    ref, slack = R.gemv(x, wq, s, z, bias)
    R.within(y, ref, slack, f"x {tuple(x.shape)} w {tuple(wq.shape)} groups {tuple(s.shape)}")
    return y


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("xdt,ydt,sdt,zero", [(BF, BF, F32, False), (BF, F32, BF, True),
                                              (F32, F32, F32, True), (F32, BF, BF, False)])
def test_types_groups_and_batches(q, group, M, xdt, ydt, sdt, zero):
    N, K = 200, group * 5
    wq, s, z = weights(N, K, group, sdt, zero, seed=group + M)
    bias = torch.randn(N, device="cuda", generator=gen(3))
    check(q, rows(M, K, xdt), wq, s, z, bias, ydt)


@pytest.mark.parametrize("N", [1, 3, 8, 15, 16, 17, 31, 33, 127, 1000, 4096])
@pytest.mark.parametrize("K", [32, 96, 128, 160, 1024, 2080])
def test_odd_sizes(q, N, K):
    wq, s, z = weights(N, K, 32, seed=N + K)
    check(q, rows(1, K, BF), wq, s)
    check(q, rows(5, K, F32), wq, s)


@pytest.mark.parametrize("M", [17, 31, 32, 33, 64, 100])
def test_many_rows(q, M):
    wq, s, z = weights(130, 512, 128, zero=True)
    check(q, rows(M, 512, BF), wq, s, z)
    check(q, rows(M, 512, F32), wq, s, z)


@pytest.mark.parametrize("dt", [BF, F32])
def test_most_rows(q, dt):
    """As many rows as one grid takes; one more is refused."""
    M = 65535 * 16
    wq, s, _ = weights(8, 32, 32)
    x = rows(M + 1, 32, dt)
    check(q, x[:M], wq, s)
    with pytest.raises(q.QvlaError):
        q.qvla_w4a16_gemv(x, wq, s)


@pytest.mark.parametrize("N,K,group,M", [(64, 16384, 128, 1), (100, 32768, 32, 2), (8200, 32768, 32, 1),
                                         (8200, 32768, 32, 3), (20000, 8192, 64, 2), (9000, 4096, 128, 9), (2048, 16384, 128, 3),
                                         (16384, 2048, 64, 1), (40, 32768, 256, 16),
                                         (70000, 256, 32, 2)])
def test_long_and_wide(q, N, K, group, M):
    wq, s, z = weights(N, K, group, BF, True)
    check(q, rows(M, K, BF), wq, s, z)
    check(q, rows(M, K, F32), wq, s, z)


def test_offsets_past_32_bits(q):
    """Codes of 4.3 GB: the last rows lie past 2^32 bytes."""
    N, K = 262144 + 40, 32768
    wq = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    wq.random_(0, 256, generator=gen(5))
    s = 0.01 + 0.05 * torch.rand(N, K // 256, device="cuda", generator=gen(6))
    x = rows(1, K, BF)
    y = q.qvla_w4a16_gemv(x, wq, s, out_dtype=F32)
    for part in (slice(0, 64), slice(N - 64, N)):
        ref, slack = R.gemv(x, wq[part], s[part])
        R.within(y[:, part], ref, slack, "rows at the ends")


def test_one_input_at_a_time_is_exact(q):
    """A row with a single nonzero input is one exact product, one scaling: fp32 activations
    enter whole (all 24 bits), at every place of K."""
    N, K, G = 32, 512, 64
    wq, s, z = weights(N, K, G, zero=True)
    k = torch.arange(K, device="cuda")
    for m0 in range(0, K, 16):
        x = torch.zeros(16, K, device="cuda")
        x[torch.arange(16), k[m0:m0 + 16]] = 1.0 + torch.rand(16, device="cuda", generator=gen(m0)) \
            + 2.0 ** -23
        y = q.qvla_w4a16_gemv(x, wq, s, z)
        ref, _ = R.gemv(x, wq, s, z)
        # the product of 24 and 4 bits may round once, the scaling once, both sums are with zeros
        R.within(y, ref, 2 * R.U * ref.abs(), f"k {m0}..")


def test_one_input_at_a_time_few_rows(q):
    """The same for one and two rows, where activations enter as 32-bit (bf16: 24-bit) integers
    of their group: the largest one is exact."""
    N, K, G = 32, 512, 64
    for zero in (False, True):
        wq, s, z = weights(N, K, G, zero=zero)
        for k in list(range(0, K, 37)) + [K - 1]:
            for dt in (F32, BF):
                x = torch.zeros(2, K, device="cuda", dtype=dt)
                x[0, k] = -(1.0 + torch.rand(1, device="cuda", generator=gen(k)).item())
                x[1, K - 1 - k] = 1.9921875 if dt == BF else 2.0 - 2.0 ** -23
                y = q.qvla_w4a16_gemv(x, wq, s, z, out_dtype=F32)
                ref, _ = R.gemv(x, wq, s, z)
                # scaling rounds once, the planes' sum once, the smaller planes below 2^-6 of both
                R.within(y, ref, (2 + 2.0 ** -5) * R.U * ref.abs(), f"k {k} {dt}")


@pytest.mark.parametrize("M", [1, 2, 3])
@pytest.mark.parametrize("big", [30.0, 1e4, 1e8])
def test_outliers_next_to_small_values(q, M, big):
    """A group's largest value sets the grid of its others for one and two rows: their error is
    counted in 2^-23 (bf16) and 2^-30 (fp32) of it."""
    N, K, G = 64, 512, 128
    wq, s, z = weights(N, K, G, zero=True)
    for dt in (BF, F32):
        x = rows(M, K, dt)
        x[:, ::G] *= big
        y = q.qvla_w4a16_gemv(x, wq, s, z, out_dtype=F32)
        ref, slack = R.gemv(x, wq, s, z)
        w = ((R.unpack(wq, False).view(N, K // G, G) - z.double()[..., None]) * s.double()[..., None]).abs().sum(2)
        top = x.double().abs().view(M, K // G, G).amax(2)
        grid = 2.0 ** -23 if dt == BF else 2.0 ** -30
        R.within(y, ref, slack + grid * (top @ w.T), f"{dt}")


def test_extreme_activations(q):
    """The largest finite fp32 values and values below bf16's normal range; an infinite or NaN
    row leaves the others alone."""
    N, K, G = 48, 256, 64
    wq, s, _ = weights(N, K, G)
    wq = wq & 0x11                             # codes 0 and 1: sums of few large values
    for big in (3.0e38, 1e-37, 1e-38):
        x = torch.zeros(3, K, device="cuda")
        x[:, 5] = big * torch.tensor([1.0, 0.77, 0.123456789], device="cuda")
        y = q.qvla_w4a16_gemv(x, wq, s)
        ref, _ = R.gemv(x, wq, s)
        R.within(y, ref, 2 * R.U * ref.abs() + 2.0 ** -126 * 2 ** -8, f"value {big}")
    x = rows(5, K, F32)
    clean = q.qvla_w4a16_gemv(x, wq, s)
    x[1, 7], x[3, 9] = float("inf"), float("nan")
    y = q.qvla_w4a16_gemv(x, wq, s)
    assert torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])
    assert y[3].isnan().all() and not y[1].isfinite().any()


def test_rows_do_not_depend_on_the_batch(q):
    wq, s, z = weights(300, 1024, 128, zero=True)
    for dt in (BF, F32):
        x = rows(40, 1024, dt)
        whole = q.qvla_w4a16_gemv(x, wq, s, z, out_dtype=F32)
        for M in (3, 8, 9, 17):
            assert torch.equal(q.qvla_w4a16_gemv(x[:M], wq, s, z, out_dtype=F32), whole[:M])
        two = q.qvla_w4a16_gemv(x[:2], wq, s, z, out_dtype=F32)
        assert torch.equal(q.qvla_w4a16_gemv(x[:1], wq, s, z, out_dtype=F32), two[:1])
        assert torch.equal(q.qvla_w4a16_gemv(x[1:2], wq, s, z, out_dtype=F32), two[1:])


def test_pitches_and_given_output(q):
    """Rows inside wider buffers; what lies outside the output rows stays."""
    N, K = 72, 256
    wq, s, _ = weights(N, K, 64)
    xb = rows(6, 512, BF)
    for ydt in (BF, F32):
        buf = torch.full((6, 128), 7.0, dtype=ydt, device="cuda")
        y = q.qvla_w4a16_gemv(xb[:, 128:384], wq, s, y=buf[:, 16:16 + N])
        ref, slack = R.gemv(xb[:, 128:384], wq, s)
        R.within(y, ref, slack)
        assert (buf[:, :16] == 7).all() and (buf[:, 16 + N:] == 7).all()


def test_zero_points_use_their_low_bits(q):
    wq, s, z = weights(40, 128, 32, zero=True)
    x = rows(2, 128, BF)
    assert torch.equal(q.qvla_w4a16_gemv(x, wq, s, z), q.qvla_w4a16_gemv(x, wq, s, z + 32))


def test_nothing_to_do(q):
    wq, s, _ = weights(40, 128, 32)
    assert q.qvla_w4a16_gemv(rows(0, 128, BF), wq, s).shape == (0, 40)


def test_graph_and_side_stream(q):
    wq, s, z = weights(500, 1024, 128, zero=True)
    x = rows(3, 1024, BF)
    y = torch.empty(3, 500 + 4, dtype=BF, device="cuda")[:, :500]
    want = q.qvla_w4a16_gemv(x, wq, s, z)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        q.qvla_w4a16_gemv(x, wq, s, z, y=y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            q.qvla_w4a16_gemv(x, wq, s, z, y=y)
    torch.cuda.synchronize()
    x2 = rows(3, 1024, BF, seed=9)
    x.copy_(x2)
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, q.qvla_w4a16_gemv(x2, wq, s, z))
    assert not torch.equal(y, want)
    other = q.qvla_w4a16_gemv(x2, wq, s, z, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(other, y)


@pytest.mark.parametrize("N,K,M", [(40, 16384, 1), (40, 16384, 5), (200, 2048, 2), (9000, 512, 16)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_graphs_at_the_same_time(q, N, K, M, dt):
    """The split over a cluster included: calls share nothing, so graphs may run side by side."""
    wq, s, z = weights(N, K, 128, zero=True)
    x = rows(M, K, dt)
    want = check(q, x, wq, s, z)
    torch.cuda.synchronize()
    ys, graphs = [], []
    for _ in range(2):
        y = torch.empty(M, (N + 7) // 8 * 8, dtype=dt, device="cuda")[:, :N]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                q.qvla_w4a16_gemv(x, wq, s, z, y=y)
        ys.append(y)
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(5):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        eager = q.qvla_w4a16_gemv(x, wq, s, z)
        torch.cuda.synchronize()
        for y in (*ys, eager):
            assert torch.equal(y, want)


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("sdt", [F32, BF])
@pytest.mark.parametrize("zero", [False, True])
def test_pack(q, group, sdt, zero):
    """Codes, scales and zero points by the stated rule (the same IEEE fp32 operations in torch),
    and the packed product near the original one."""
    N, K = 50, 2 * 256
    W = torch.randn(N, K, device="cuda", generator=gen(group)) * 0.02
    W[0] = 0
    W[1, :group] = W[1, :group].abs()
    W[2, :group] = -W[2, :group].abs()
    wq, s, z = q.qvla_pack_weights_w4g(W, group, zero, sdt)
    w = W.view(N, K // group, group)
    seven, fifteen = (torch.full((), v, device="cuda") for v in (7.0, 15.0))   # tensors: a true division
    if zero:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        want_s = ((hi - lo) / fifteen).to(sdt)
        sf = want_s.float()
        want_z = torch.where(sf > 0, torch.round(-lo / sf).clamp(0, 15), 0.0)
        c = torch.where(sf[..., None] > 0, (torch.round(w / sf[..., None]) + want_z[..., None]).clamp(0, 15), 0.0)
        assert torch.equal(z, want_z.to(torch.uint8))
        err = (c - want_z[..., None]) * sf[..., None] - w
    else:
        want_s = (w.abs().amax(2) / seven).to(sdt)
        sf = want_s.float()
        c = torch.where(sf[..., None] > 0, torch.round(w / sf[..., None]).clamp(-7, 7), 0.0)
        assert z is None
        err = c * sf[..., None] - w
    assert torch.equal(s, want_s)
    assert torch.equal(R.unpack(wq, not zero), c.view(N, K).double())
    # rounding to a step, the ends may miss by the rounding of the scale
    assert (err.abs() <= sf[..., None] * (0.5 + 15 * R.half_step(sdt) + (1.0 if zero else 0) * 0.5 + 1e-5)).all()
    check(q, rows(2, K, BF), wq, s, z)


@pytest.mark.parametrize("sdt", [F32, BF])
def test_pack_spans_past_the_largest_float(q, sdt):
    """Finite weights whose span is not: the scale is, and the codes are the stated ones."""
    W = torch.zeros(3, 64, device="cuda")
    W[0, :3] = torch.tensor([-3e38, 3e38, 1e38], device="cuda")
    W[1, :2] = torch.tensor([-3.4e38, 3.4e38], device="cuda")
    W[2, :2] = torch.tensor([-1.0, 2.0], device="cuda")
    wq, s, z = q.qvla_pack_weights_w4g(W, 64, True, sdt)
    w = W.double()
    want = ((w.amax(1) - w.amin(1)) / 15).to(sdt)
    assert torch.equal(s[:, 0], want)
    sf = want.double()
    zero = torch.round(-w.amin(1) / sf).clamp(0, 15)
    assert torch.equal(z[:, 0].double(), zero)
    assert torch.equal(R.unpack(wq, False), (torch.round(w / sf[:, None]) + zero[:, None]).clamp(0, 15))


@pytest.mark.parametrize("M", [1, 2, 3])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("zero", [False, True])
def test_ends_of_the_range_of_activations(q, M, dt, zero):
    """The largest finite activations, the places where a group's grid changes, and values down to
    the smallest subnormal, by both kernels."""
    N, K, G = 48, 256, 64
    wq, s, z = weights(N, K, G, zero=zero)
    wq, z = wq & 0x11, z & 1 if zero else None          # codes times values stay in range
    big, tiny = torch.finfo(dt).max, 2.0 ** (-133 if dt == BF else -149)
    part = torch.tensor([1.0, 0.77, 0.123456789], device="cuda")[:M]
    w = R.unpack(wq, False) - (z.double().repeat_interleave(G, 1) if zero else 0)
    w = (w.view(N, K // G, G) * s.double()[..., None]).abs()
    for value in (big, 1.9921875 * 2.0 ** 120, 2.0 ** 120, 1.9921875, 1.984375, 2.0, 1.0, 1e-30, 2.0 ** -116, 2.0 ** -117,
                  2.0 ** -123, 1e-37, 1e-38, 2.0 ** -130, tiny):
        x = torch.zeros(M, K, dtype=torch.float64, device="cuda")
        x[:, 5], x[:, 6], x[:, 70] = value * part, value * part / 300, -0.6 * value * part
        x = x.to(dt)
        y = q.qvla_w4a16_gemv(x, wq, s, z, out_dtype=F32)
        ref, slack = R.gemv(x, wq, s, z)
        # One and two rows: half of the group's grid, 2^-21 (bf16) or 2^-29 of a power of two up
        # to its largest value, or 2^-145 if that is more.  More rows: an fp32 value is three
        # values of bf16, whose subnormals are multiples of 2^-133, and loses what is below.
        # Results below the normal range are off by 2^-150 for each of fewer than 64 operations.
        top = x.double().abs().view(M, K // G, G).amax(2)
        grid = (top * 2.0 ** (-21 if dt == BF else -29)).clamp(min=2.0 ** -145)
        lost = grid / 2 @ w.sum(2).T if M < 3 else (x != 0).double() * 2.0 ** -133 @ w.flatten(1).T * (dt == F32)
        R.within(y, ref, slack + lost + 2.0 ** -144, f"{value}")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,G", [(48, 256, 64), (72, 512, 256), (33, 96, 32)])
def test_non_finite_row_of_two(q, dt, zero, N, K, G):
    """One and two rows: an infinity or a NaN makes its row NaN, and the other row is what it is
    without it."""
    wq, s, z = weights(N, K, G, zero=zero)
    x = rows(2, K, dt)
    clean = q.qvla_w4a16_gemv(x, wq, s, z, out_dtype=F32)
    for bad in (float("inf"), -float("inf"), float("nan")):
        for m in (0, 1):
            for k in (0, 7, K - 1):
                e = x.clone()
                e[m, k] = bad
                y = q.qvla_w4a16_gemv(e, wq, s, z, out_dtype=F32)
                assert y[m].isnan().all() and torch.equal(y[1 - m], clean[1 - m])
                assert q.qvla_w4a16_gemv(e[m:m + 1], wq, s, z, out_dtype=F32).isnan().all()
