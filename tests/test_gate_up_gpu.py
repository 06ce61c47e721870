"""The gated projection and its gradients against plain 64-bit formulas.

Tolerances: products of bf16 values are exact; a tensor-core sum of K of them is taken to be
off by at most K 2^-23 of the sum of their magnitudes (one fp32 step a term, also where the
hardware truncates).  Activations and their slopes are off by less than 2^-19 (1 + |z|); the
slopes lie within [-0.13, 1.13].  Each bf16 rounding is 2^-8 relative: the result's own, and in
the gradients that of dg and du, whose terms' magnitudes bound its effect on each element; as
rounding errors of one sum are independent of each other, the whole result (2-norm) has to be
within 2^-8 too: two roundings of at most 2^-8 / sqrt(3) rms each."""
import pytest
import torch

pytestmark = pytest.mark.gpu
B, U = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module")
def nv():
    import bit_quantized_moe_nvfp4_b200 as m
    return m


def draw(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def act_fn(act, z):
    if act == 0:
        return z * torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))


def close(got, ref, slack):
    g = got.detach().cpu().double()
    ref, slack = ref.cpu(), slack.cpu()
    assert g.shape == ref.shape
    bad = (g - ref).abs() > B * ref.abs() + slack
    assert not bad.any(), (int(bad.sum()), float((g - ref).abs().max()), bad.nonzero()[:4])


def near(got, ref):
    d = torch.linalg.vector_norm(got.detach().double().cpu() - ref.cpu())
    n = torch.linalg.vector_norm(ref.cpu())
    assert d <= B * n, float(d / n)


def inputs(T, H, I):
    return draw(T + H, T, H), draw(I + H, 2 * I, H, std=H ** -0.5)


# T up to 16, 32 and above: each column tile of the split kernel.  Many rows and columns: pairs of
# CTAs, with tiles cut in half (34, 36 tiles), whole ones only (72), a whole round and a cut one
# (90), and four rounds (289), where accumulators and stages are used again.  Sizes that end
# inside every tile.
SHAPES = [(1, 64, 8), (2, 200, 72), (16, 264, 64), (17, 136, 200), (33, 64, 136), (64, 512, 64),
          (65, 72, 328), (129, 264, 520), (300, 128, 8), (257, 192, 2056), (1000, 520, 1032),
          (2049, 64, 1024), (2500, 72, 1032), (4100, 136, 2056)]


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
def test_gate_up(nv, T, H, I, act):
    x, w = inputs(T, H, I)
    gu = torch.full((T, 2 * I), float("nan"), dtype=torch.bfloat16, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = nv.moe_nvfp4_gate_up(x.cuda(), w.cuda(), act=act, gu=gu, error_flag=flag)
    alone = nv.moe_nvfp4_gate_up(x.cuda(), w.cuda(), act=act)
    assert int(flag) == 0
    assert torch.equal(h, alone)
    xd, wd = x.cuda().double(), w.cuda().double()
    ref = xd @ wd.t()
    mag = (xd.abs() @ wd.abs().t()) * (H * U)
    close(gu, ref, mag)
    g, u, eg, eu = ref[:, :I], ref[:, I:], mag[:, :I], mag[:, I:]
    a = act_fn(act, g)
    ea = 1.13 * eg + 2.0 ** -19 * (1 + g.abs())
    close(h, a * u, ea * u.abs() + a.abs() * eu + ea * eu)


def dgu_ref(gu, dh, act):
    gu = gu.double().requires_grad_()
    I = gu.shape[1] // 2
    d, = torch.autograd.grad(act_fn(act, gu[:, :I]) * gu[:, I:], gu, dh.double())
    return d


@pytest.mark.parametrize("T,H,I", SHAPES + [(4096, 256, 64), (40, 2048, 1032), (1100, 1544, 72),
                                           (4100, 4104, 72)])
@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
def test_gate_up_backward(nv, T, H, I, act):
    x, w = (t.cuda() for t in inputs(T, H, I))
    gu, dh = draw(3, T, 2 * I, std=1.5).cuda(), draw(4, T, I, std=0.1).cuda()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = nv.moe_nvfp4_gate_up_backward(dh, x, w, gu, act=act, error_flag=flag)
    one = nv.moe_nvfp4_gate_up_backward(dh, x, w, gu, act=act, need_dw=False)
    two = nv.moe_nvfp4_gate_up_backward(dh, x, w, gu, act=act, need_dx=False)
    assert int(flag) == 0
    assert one[1] is None and two[0] is None
    assert torch.equal(one[0], dx) and torch.equal(two[1], dw)   # one order of summation
    d = dgu_ref(gu, dh, act)
    # terms of d whose error is not relative to d itself: 2^-19 (1 + |z|) |dh| (1 + |u|)
    ed = 2.0 ** -19 * (1 + gu.double().abs()) * dh.double().abs().repeat(1, 2) * \
        (1 + gu.double().abs().roll(I, 1))
    xd, wd = x.double(), w.double()
    for got, ref, m in ((dx, d @ wd, lambda t: t @ wd.abs()),
                        (dw, d.t() @ xd, lambda t: t.t() @ xd.abs())):
        K = 2 * I if got is dx else T
        close(got, ref, m(d.abs()) * (B + K * U) + m(ed))
        near(got, ref)


def test_gradients_against_differences(nv):
    T, H, I, h = 5, 72, 40, 1e-5
    x, w = inputs(T, H, I)
    dh = draw(9, T, I)
    gu = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    nv.moe_nvfp4_gate_up(x.cuda(), w.cuda(), gu=gu)
    got = nv.moe_nvfp4_gate_up_backward(dh.cuda(), x.cuda(), w.cuda(), gu)

    def f(x, w):
        z = x @ w.t()
        return float((act_fn(0, z[:, :I]) * z[:, I:] * dh.double()).sum())

    xd, wd = x.double(), w.double()
    d = dgu_ref((xd @ wd.t()), dh, 0).abs()
    # dg and du: rounded once, from g and u that were rounded once (slopes up to 1.13, second
    # derivatives up to 0.8): 4 roundings of their terms bound both
    mags = ((d + dh.double().abs().repeat(1, 2)) @ wd.abs(),
            (d + dh.double().abs().repeat(1, 2)).t() @ xd.abs())
    for k in range(2):
        e = torch.randn((xd, wd)[k].shape, generator=torch.Generator().manual_seed(k),
                        dtype=torch.float64)
        a = (xd + h * e, wd) if k == 0 else (xd, wd + h * e)
        b = (xd - h * e, wd) if k == 0 else (xd, wd - h * e)
        diff = (f(*a) - f(*b)) / (2 * h)
        tol = float((mags[k] * e.abs()).sum()) * 4 * B + 1e-3
        assert abs(diff - float((got[k].cpu().double() * e).sum())) <= tol


def test_large_and_special_pre_activations(nv):
    """|z| far beyond exp's range, zeros, and infinities: what the formulas give."""
    I, H = 8, 8
    z = torch.tensor([-200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e4]).bfloat16()
    x = torch.zeros(1, H, dtype=torch.bfloat16)
    x[0, 0] = 1
    w = torch.zeros(2 * I, H, dtype=torch.bfloat16)
    w[:I, 0], w[I:, 0] = z, 1
    for act in (0, 1):
        h = nv.moe_nvfp4_gate_up(x.cuda(), w.cuda(), act=act).cpu().double()[0]
        ref = act_fn(act, z.double())
        assert ((h - ref).abs() <= B * ref.abs() + 2.0 ** -19 * (1 + z.double().abs())).all()
        gu = torch.cat([z, torch.ones(I).bfloat16()]).unsqueeze(0).cuda()
        dh = torch.ones(1, I, dtype=torch.bfloat16).cuda()
        _, dw = nv.moe_nvfp4_gate_up_backward(dh, x.cuda(), w.cuda(), gu, act=act)
        assert dw.isfinite().all()
        assert (dw[:I, 0].cpu().double() - dgu_ref(gu.cpu(), dh.cpu(), act)[0, :I]).abs().max() \
            <= 2 * B


def test_rows_of_nan_stay_their_own(nv):
    for T in (5, 40, 700):
        x, w = inputs(T, 136, 520)
        bad = x.clone()
        bad[2] = float("nan")
        a = nv.moe_nvfp4_gate_up(x.cuda(), w.cuda())
        b = nv.moe_nvfp4_gate_up(bad.cuda(), w.cuda())
        keep = torch.arange(T) != 2
        assert torch.equal(a.cpu()[keep], b.cpu()[keep])
        assert b[2].isnan().all()


def test_outputs_end_where_they_end(nv):
    """Rows behind the last token and the bytes around a result stay as they were."""
    for T, H, I in ((5, 136, 72), (300, 136, 1032)):
        x, w = inputs(T, H, I)
        buf = torch.full((T + 8, I), 7.0, dtype=torch.bfloat16, device="cuda")
        gbuf = torch.full((T + 8, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
        nv.moe_nvfp4_gate_up(x.cuda(), w.cuda(), h=buf[:T], gu=gbuf[:T])
        assert (buf[T:] == 7).all() and (gbuf[T:] == 7).all()
        dxb = torch.full((T + 8, H), 7.0, dtype=torch.bfloat16, device="cuda")
        dwb = torch.full((2 * I + 8, H), 7.0, dtype=torch.bfloat16, device="cuda")
        nv.moe_nvfp4_gate_up_backward(buf[:T], x.cuda(), w.cuda(), gbuf[:T], dx=dxb[:T],
                                      dw_gu=dwb[:2 * I])
        assert (dxb[T:] == 7).all() and (dwb[2 * I:] == 7).all()


def test_results_beyond_32_bit_offsets(nv):
    """h and gu of more than 2^31 elements: the first, middle and last rows are right."""
    T, H, I = 140000, 8, 8192
    x, w = draw(1, T, H), draw(2, 2 * I, H, std=0.5)
    gu = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    h = nv.moe_nvfp4_gate_up(x.cuda(), w.cuda(), gu=gu)
    for t in (0, 131071, 131072, T - 1):
        ref = x[t].double() @ w.double().t()
        mag = x[t].double().abs() @ w.double().abs().t() * (H * U)
        close(gu[t], ref, mag)
        g, u, e = ref[:I], ref[I:], 1.13 * mag[:I] + 2.0 ** -19 * (1 + ref[:I].abs())
        close(h[t], act_fn(0, g) * u, e * u.abs() + act_fn(0, g).abs() * mag[I:] + e * mag[I:])


def test_zero_tokens(nv):
    x, w = torch.empty(0, 64, dtype=torch.bfloat16).cuda(), draw(1, 32, 64).cuda()
    h = nv.moe_nvfp4_gate_up(x, w)
    assert h.shape == (0, 16)
    gu = torch.empty(0, 32, dtype=torch.bfloat16).cuda()
    dx, dw = nv.moe_nvfp4_gate_up_backward(h, x, w, gu, dw_gu=torch.ones_like(w))
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_another_stream_and_a_graph(nv):
    for T in (8, 600):
        x, w = (t.cuda() for t in inputs(T, 256, 1024))
        dh = draw(5, T, 1024).cuda()

        def step(x):
            gu = torch.empty(T, 2048, dtype=torch.bfloat16, device="cuda")
            h = nv.moe_nvfp4_gate_up(x, w, gu=gu)
            return (h,) + nv.moe_nvfp4_gate_up_backward(dh, x, w, gu)

        want = step(x)
        torch.cuda.synchronize()
        s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(s):
            a = step(x)
        with torch.cuda.stream(s2):   # two calls at once
            b = step(x)
        torch.cuda.synchronize()
        xin = torch.zeros_like(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c = step(xin)
        xin.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        for got in (a, b, c):
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def gate_of(z, T, I, H=8):
    """x, w_gu, gu, dh with which every row's pre-activations are z (I of them) and 1."""
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 1
    w = torch.zeros(2 * I, H, dtype=torch.bfloat16)
    w[:I, 0], w[I:, 0] = z, 1
    gu = torch.cat([z, torch.ones(I).bfloat16()]).repeat(T, 1)
    return x.cuda(), w.cuda(), gu.cuda(), torch.ones(T, I, dtype=torch.bfloat16).cuda()


def gelu_64(z):
    """GELU's tanh form without its cancellation: (1 + tanh v) / 2 = 1 / (1 + exp(-2 v))."""
    return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))


@pytest.mark.parametrize("T,I", [(1, 520), (40, 520), (700, 1032)])
def test_gelu_of_negative_gates(nv, T, I):
    """Where (1 + tanh v) / 2 is small, act and slope are as exact as elsewhere.  v is off by
    5 u (u = 2^-24; constant, square, fma and product, the constant's own rounding), so exp(-2 v)
    by 10 |v| u + 4 u, at |v| <= 43 (z >= -10) 434 u < 2^-15; sum, division and product add 4 u.
    The slope's second factor 1 + 2 z (1 - s) v' is at least 1 in magnitude for z <= -2 and its
    terms at most 2 (1 + |it|): below 20 u.  All within 2^-14, and the rounding to bf16."""
    z = -torch.linspace(2, 10, I).bfloat16()
    x, w, gu, dh = gate_of(z, T, I)
    zd = z.double().requires_grad_()
    ref = gelu_64(zd)
    slope, = torch.autograd.grad(ref.sum(), zd)
    h = nv.moe_nvfp4_gate_up(x, w, act=nv.ACT_GELU).cpu().double()
    assert ((h - ref.detach()).abs() <= (B + 2.0 ** -14) * ref.detach().abs()).all()
    # one row reaches dw (its column 0 is the sum of dg over the rows): dg itself
    one = torch.zeros_like(x)
    one[T - 1] = x[T - 1]
    _, dw = nv.moe_nvfp4_gate_up_backward(dh, one, w, gu, act=nv.ACT_GELU)
    got = dw[:I, 0].cpu().double()
    assert ((got - slope).abs() <= (B + 2.0 ** -14) * slope.abs()).all()


@pytest.mark.parametrize("T,I", [(1, 8), (700, 1032)])
def test_huge_gates(nv, T, I):
    """Gates whose square or cube leaves fp32: the activation is z or 0, its slope 1 or 0."""
    z = torch.tensor([1e10, -1e10, 2e19, -2e19, 1e30, -1e30, 3e38, -3e38]).bfloat16()
    z = z.repeat((I + 7) // 8)[:I]
    x, w, gu, dh = gate_of(z, T, I)
    one = torch.zeros_like(x)
    one[T - 1] = x[T - 1]
    for act in (0, 1):
        h = nv.moe_nvfp4_gate_up(x, w, act=act).cpu()
        assert torch.equal(h, torch.where(z > 0, z, torch.zeros_like(z)).expand(T, I))
        _, dw = nv.moe_nvfp4_gate_up_backward(dh, one, w, gu, act=act)
        assert torch.equal(dw[:I, 0].cpu(), (z > 0).bfloat16())


@pytest.mark.parametrize("T,I", [(1, 8), (700, 1032)])
def test_infinite_gates(nv, T, I):
    """+infinity passes through; -infinity, for which z / (1 + exp(-z)) is not a number, never
    gives a finite value but 0, and neither touches another column or row."""
    z = torch.linspace(-3, 3, I).bfloat16()
    x, w, _, _ = gate_of(z, T, I)
    bad = w.clone()
    bad[1, 0], bad[2, 0] = float("inf"), -float("inf")
    keep = torch.ones(I, dtype=torch.bool)
    keep[1:3] = False
    for act in (0, 1):
        a = nv.moe_nvfp4_gate_up(x, w, act=act).cpu()
        b = nv.moe_nvfp4_gate_up(x, bad, act=act).cpu()
        assert torch.equal(a[:, keep], b[:, keep])
        assert (b[:, 1] == float("inf")).all()
        assert (b[:, 2].isnan() | (b[:, 2] == 0)).all()


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
def test_no_nan_comes_of_finite_inputs(nv, T, H, I, act):
    """Every element is written (memory that held NaN before) and is a number."""
    x, w = (t.cuda() for t in inputs(T, H, I))
    h, gu, dx, dw = (torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
                     for s in ((T, I), (T, 2 * I), (T, H), (2 * I, H)))
    nv.moe_nvfp4_gate_up(x, w, act=act, h=h, gu=gu)
    nv.moe_nvfp4_gate_up_backward(h, x, w, gu, act=act, dx=dx, dw_gu=dw)
    for t in (h, gu, dx, dw):
        assert t.isfinite().all()


def test_huge_up_values_beside_a_closed_gate(nv):
    """dh u leaves fp32, dh u act'(g) is 0."""
    z = torch.full((8,), -200.0).bfloat16()
    x, w, gu, dh = gate_of(z, 1, 8)
    gu[:, 8:] = 3e38
    for act in (0, 1):
        _, dw = nv.moe_nvfp4_gate_up_backward(4 * dh, x, w, gu, act=act)
        assert (dw == 0).all()


@pytest.mark.parametrize("T,H,I", [(3, 65536, 8), (300, 65536, 8), (3, 8, 65536), (300, 16, 65536)])
def test_largest_widths(nv, T, H, I):
    """H and I at their limits, in both kernels, forward and backward."""
    test_gate_up(nv, T, H, I, 0)
    test_gate_up_backward(nv, T, H, I, 0)
    test_no_nan_comes_of_finite_inputs(nv, T, H, I, 0)
