"""The norms before and after a block, their gradients and the 8-bit rows, against plain
64-bit formulas.

Tolerances, with u = 2^-24 (fp32) and the result's own rounding to bf16 (2^-8 relative):
a row's sum of squares is added in chains of at most 32 values a thread, then trees and at
most 32 warps, so it is off by < 80 u; r = rsqrt is off by half of that and 4 u more; n, the
weight, the gate and the sum add < 8 u.  Every fp32 value before the last rounding is then
within E = 2^-17 = 128 u of the sum of the magnitudes of its terms.  A sum over T rows adds
T u of its terms' magnitudes."""
import functools

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
EPS = 1e-5
B, E, U = 2.0 ** -8, 2.0 ** -17, 2.0 ** -24


@pytest.fixture(scope="module")
def nv():
    import bit_quantized_moe_nvfp4_b200 as m
    return m


def draw(seed, *shape, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(torch.bfloat16)


def close(got, ref, slack):
    """|got - ref| <= 2^-8 |ref| + slack, element by element."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape
    bad = (g - ref).abs() > B * ref.abs() + slack
    assert not bad.any(), (int(bad.sum()), float((g - ref).abs().max()))


def rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


# rows of a warp (H <= 1536), of a CTA of 256 threads, of 1024 threads; partly filled vectors
SHAPES = [(1, 8), (3, 64), (5, 264), (9, 1024), (1, 1032), (7, 1536), (150, 2056), (2, 6144),
          (333, 6144), (160, 8200), (3, 32768)]


@pytest.mark.parametrize("T,H", SHAPES)
def test_pre_norm(nv, T, H):
    x, w = draw(T + H, T, H), draw(H, H, std=0.1, mean=1.0)
    out = nv.moe_nvfp4_pre_norm(x.cuda(), w.cuda(), EPS)
    xd, wd = x.double(), w.double()
    ref = wd * xd * rms(xd)
    close(out, ref, E * ref.abs())


@pytest.mark.parametrize("T,H", [(1, 16), (3, 1024), (2, 1040), (40, 6144), (3, 32768)])
def test_pre_norm_int8(nv, T, H):
    """Codes are within half a step (and the fp32 error) of the real quotient."""
    x, w = draw(T + H, T, H), draw(H, H, std=0.1, mean=1.0)
    codes, scales = nv.moe_nvfp4_pre_norm_int8(x.cuda(), w.cuda(), EPS)
    y = w.double() * x.double() * rms(x.double())
    amax = y.abs().amax(-1, keepdim=True)
    s = scales.cpu().double().unsqueeze(1)
    assert ((s - amax / 127).abs() <= 2 * E * amax / 127).all()
    q = codes.cpu().double()
    assert q.abs().max() <= 127
    assert ((q - 127 * y / amax).abs() <= 0.5 + 127 * 4 * E).all()
    assert (q.abs().amax(-1) == 127).all()


@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 48), (9, 1024), (3, 1040), (200, 6144),
                                       (2, 32768)])
def test_int8_quantize_is_exact(nv, rows, cols):
    """Codes against exact integer arithmetic: bf16 values are m 2^e with |m| < 2^8."""
    x = draw(rows + cols, rows, cols) * torch.logspace(-6, 6, rows).unsqueeze(1).bfloat16()
    x[0, :16] = torch.tensor([127, 0.5, 1.5, 2.5, -0.5, -1.5, 63.5, -126.5, 0, -0.0, 1, 2, 3, 4,
                              -127, 0.25]).bfloat16()        # ties: even codes
    x[0, 16:] = 0
    x = x.bfloat16()
    codes, scales = nv.nvfp4_int8_quantize(x.cuda())
    xd = x.double().numpy()
    amax = np.abs(xd).max(1, keepdims=True)
    # x 127 is exact in 64 bits and the quotient cannot meet a tie by rounding
    want = np.rint(xd * 127 / np.where(amax > 0, amax, 1))
    assert np.array_equal(codes.cpu().numpy().astype(np.float64), want)
    s = np.where(amax[:, 0] > 0, amax[:, 0].astype(np.float32) / np.float32(127), np.float32(1))
    assert np.array_equal(scales.cpu().numpy(), s.astype(np.float32))


def test_int8_quantize_extreme_rows(nv):
    """An all-zero row, the largest and the smallest bf16 magnitudes."""
    big, tiny = torch.finfo(torch.bfloat16).max, 2.0 ** -133
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    x[1, 3], x[1, 4], x[1, 5] = big, -big / 2, big / 512
    x[2, 0], x[2, 1] = tiny, -tiny
    x[3] = 1
    codes, scales = nv.nvfp4_int8_quantize(x.cuda())
    q = codes.cpu()
    assert (q[0] == 0).all() and float(scales[0]) == 1.0
    assert q[1, 3] == 127 and q[1, 4] == -64 and q[1, 5] == 0 and q[1, 6] == 0
    assert q[2, 0] == 127 and q[2, 1] == -127
    assert (q[3] == 127).all()


def gates(kind, T, H, seed):
    shape = {"none": None, "1": (1, 1), "t": (T, 1), "h": (1, H), "th": (T, H)}[kind]
    return None if shape is None else draw(seed, *shape, std=0.5, mean=0.5)


@pytest.mark.parametrize("gate", ["none", "1", "t", "h", "th"])
@pytest.mark.parametrize("T,H", [(1, 8), (5, 264), (3, 1032), (150, 2056), (2, 6144), (2, 32768)])
def test_post_norm(nv, T, H, gate):
    y, res = draw(1, T, H), draw(2, T, H)
    w, w2 = draw(3, H, std=0.1, mean=1.0), draw(4, H, std=0.1, mean=1.0)
    g = gates(gate, T, H, 5)
    gc = None if g is None else g.cuda()
    out, nxt = nv.moe_nvfp4_post_norm(y.cuda(), w.cuda(), res.cuda(), EPS, gate=gc,
                                      residual_scale=0.75, next_weight=w2.cuda())
    alone = nv.moe_nvfp4_post_norm(y.cuda(), w.cuda(), res.cuda(), EPS, gate=gc,
                                   residual_scale=0.75)
    assert torch.equal(out, alone)
    yd, rd = y.double(), res.double()
    gd = 1.0 if g is None else g.double()
    m = gd * w.double() * yd * rms(yd)
    ref = 0.75 * rd + m
    mag = (0.75 * rd).abs() + m.abs()
    close(out, ref, E * mag)
    r2 = rms(ref)
    ref2 = w2.double() * ref * r2
    # the error of `out` reaches next through the value and, averaged, through the norm
    row = E * (mag * ref.abs()).mean(-1, keepdim=True) * r2 * r2
    close(nxt, ref2, w2.double().abs() * r2 * (E * mag + row * ref.abs()) + E * ref2.abs())


def grads(y, w, g, d, scale):
    """Formulas in 64 bits and, for each result, the magnitudes of its terms."""
    T, H = y.shape
    yd, wd, dd = y.double(), w.double(), d.double()
    gd = torch.ones(1, 1, dtype=torch.float64) if g is None else g.double()
    r = rms(yd)
    n = yd * r
    dn = dd * gd * wd
    m = (dn * n).mean(-1, keepdim=True)
    mm = (dn * n).abs().mean(-1, keepdim=True)
    dx, dxm = r * (dn - n * m), r * (dn.abs() + n.abs() * mm)
    dw, dwm = (dd * gd * n).sum(0), (dd * gd * n).abs().sum(0)
    dims = [k for k in (0, 1) if gd.shape[k] == 1]
    e = dd * wd * n
    dg = e.sum(dims, keepdim=True) if dims else e
    dgm = e.abs().sum(dims, keepdim=True) if dims else e.abs()
    return dx, dxm, dw, dwm, dg, dgm, scale * dd


@pytest.mark.parametrize("gate", ["none", "1", "t", "h", "th"])
@pytest.mark.parametrize("T,H", [(1, 8), (2, 64), (77, 264), (600, 1024), (3, 1032), (150, 2056),
                                 (700, 6144), (3, 6144), (2, 32768)])
def test_post_norm_backward(nv, T, H, gate):
    y, d = draw(1, T, H), draw(2, T, H, std=0.1)
    w, g = draw(3, H, std=0.1, mean=1.0), gates(gate, T, H, 5)
    gc = None if g is None else g.cuda()
    args = (d.cuda(), y.cuda(), w.cuda(), EPS)
    dy, dw, dg, dr = nv.moe_nvfp4_post_norm_backward(*args, gate=gc, residual_scale=0.75)
    again = nv.moe_nvfp4_post_norm_backward(*args, gate=gc, residual_scale=0.75,
                                            need_dresidual=False)
    assert again[3] is None
    assert torch.equal(dy, again[0]) and torch.equal(dw, again[1])   # one order of summation
    dx, dxm, dwr, dwm, dgr, dgm, drr = grads(y, w, g, d, 0.75)
    close(dy, dx, E * dxm)
    close(dw, dwr, (E + T * U) * dwm)
    close(dr, drr, E * drr.abs())
    if g is None:
        assert dg is None
    else:
        assert torch.equal(dg, again[2])
        close(dg, dgr, (E + T * U) * dgm)


@pytest.mark.parametrize("T,H", [(1, 8), (77, 264), (3, 1032), (700, 6144)])
@pytest.mark.parametrize("skip", [False, True])
def test_pre_norm_backward(nv, T, H, skip):
    x, d, s = draw(1, T, H), draw(2, T, H, std=0.1), draw(3, T, H, std=0.1)
    w = draw(4, H, std=0.1, mean=1.0)
    dx, dw = nv.moe_nvfp4_pre_norm_backward(d.cuda(), x.cuda(), w.cuda(), EPS,
                                            dskip=s.cuda() if skip else None)
    r, rm, wr, wm, *_ = grads(x, w, None, d, 1.0)
    add = s.double() if skip else torch.zeros_like(r)
    close(dx, r + add, E * (rm + add.abs()))
    close(dw, wr, (E + T * U) * wm)


def test_gradients_against_differences(nv):
    """Directional derivatives of the 64-bit forward formula against the kernel's gradients:
    (f(v + h e) - f(v - h e)) / 2h for the sum f = <out, d>."""
    T, H, h = 6, 264, 1e-5
    y, res, d = draw(1, T, H), draw(2, T, H), draw(3, T, H)
    w, g = draw(4, H, std=0.1, mean=1.0), draw(5, 1, H, std=0.5, mean=0.5)
    got = nv.moe_nvfp4_post_norm_backward(d.cuda(), y.cuda(), w.cuda(), EPS, gate=g.cuda(),
                                          residual_scale=0.5)
    leaves = [y.double(), w.double(), g.double(), res.double()]

    def f(v):
        return float(((0.5 * v[3] + v[2] * (v[1] * v[0] * rms(v[0]))) * d.double()).sum())

    for k, grad in enumerate(got):
        e = torch.randn(leaves[k].shape, generator=torch.Generator().manual_seed(k),
                        dtype=torch.float64)
        up = [t + h * e if i == k else t for i, t in enumerate(leaves)]
        dn = [t - h * e if i == k else t for i, t in enumerate(leaves)]
        diff = (f(up) - f(dn)) / (2 * h)
        gr = grad.cpu().double()
        # every element of the gradient is within 2^-8 + E-sized terms of the formula's; the
        # difference itself is off by h^2 times third derivatives and 2^-53 |f| / h
        tol = float((gr.abs() * e.abs()).sum()) * 2 * B + 1e-3
        assert abs(diff - float((gr * e).sum())) <= tol


@pytest.mark.parametrize("T,H", [(3, 264), (700, 6144), (900, 1032)])
def test_in_place(nv, T, H):
    """An output that is an input's own tensor."""
    y, res, w = draw(1, T, H).cuda(), draw(2, T, H).cuda(), draw(3, H, std=0.1, mean=1.0).cuda()
    g, d = draw(4, T, H).cuda(), draw(5, T, H).cuda()
    want = nv.moe_nvfp4_post_norm(y, w, res, EPS, gate=g, next_weight=w)
    a, b = res.clone(), y.clone()
    nv.moe_nvfp4_post_norm(b, w, a, EPS, gate=g, next_weight=w, out=a, next_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    a = y.clone()
    assert torch.equal(nv.moe_nvfp4_pre_norm(a, w, EPS, out=a), nv.moe_nvfp4_pre_norm(y, w, EPS))
    want = nv.moe_nvfp4_pre_norm_backward(d, y, w, EPS, dskip=res)
    for k in range(3):
        args = [d.clone(), y.clone(), res.clone()]
        got = nv.moe_nvfp4_pre_norm_backward(args[0], args[1], w, EPS, dskip=args[2], dx=args[k])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = nv.moe_nvfp4_post_norm_backward(d, y, w, EPS, gate=g, residual_scale=0.5)
    a, b, c = d.clone(), y.clone(), g.clone()
    got = nv.moe_nvfp4_post_norm_backward(a, b, w, EPS, gate=c, residual_scale=0.5, dy=b,
                                          dgate=c, dresidual=a)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    g1 = g[:, :1].contiguous()
    want = nv.moe_nvfp4_post_norm_backward(d, y, w, EPS, gate=g1)
    got = nv.moe_nvfp4_post_norm_backward(d, y, w, EPS, gate=g1, dgate=g1)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_rows_do_not_touch_each_other(nv):
    """NaN and infinity in one row leave the others as they are; a row of zeros gives zeros."""
    T, H = 6, 264
    x, w = draw(1, T, H), draw(2, H, std=0.1, mean=1.0)
    clean = nv.moe_nvfp4_pre_norm(x.cuda(), w.cuda(), EPS).cpu()
    cc, cs = nv.nvfp4_int8_quantize(x[:, :256].contiguous().cuda())
    bad = x.clone()
    bad[1, 7], bad[3, 100], bad[4] = float("nan"), float("inf"), 0
    out = nv.moe_nvfp4_pre_norm(bad.cuda(), w.cuda(), EPS).cpu()
    for t in (0, 2, 5):
        assert torch.equal(out[t], clean[t])
    assert (out[4] == 0).all() and out[1].isnan().all()
    bc, bs = nv.nvfp4_int8_quantize(bad[:, :256].contiguous().cuda())
    for t in (0, 2, 5):
        assert torch.equal(bc[t], cc[t]) and bs[t] == cs[t]


def test_rows_beyond_32_bit_offsets(nv):
    T, H = 350000, 6144
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    w = draw(2, H, std=0.1, mean=1.0)
    rows = [0, 174762, 174763, 349525, T - 1]
    x[rows] = draw(1, len(rows), H).cuda()
    out = nv.moe_nvfp4_pre_norm(x, w.cuda(), EPS)
    xd = x[rows].cpu().double()
    ref = w.double() * xd * rms(xd)
    close(out[rows], ref, E * ref.abs())
    dx, _ = nv.moe_nvfp4_pre_norm_backward(out, x, w.cuda(), EPS)
    dr, drm, *_ = grads(x[rows].cpu(), w, None, out[rows].cpu(), 1.0)
    close(dx[rows], dr, E * drm)


def test_zero_rows(nv):
    H = 264
    x, w = torch.empty(0, H, dtype=torch.bfloat16).cuda(), draw(1, H).cuda()
    assert nv.moe_nvfp4_pre_norm(x, w, EPS).shape == (0, H)
    assert nv.moe_nvfp4_post_norm(x, w, x, EPS).shape == (0, H)
    dx, dw = nv.moe_nvfp4_pre_norm_backward(x, x, w, EPS, dweight=torch.ones_like(w))
    assert dx.shape == (0, H) and (dw == 0).all()
    g = draw(2, 1, H).cuda()
    dy, dw, dg, dr = nv.moe_nvfp4_post_norm_backward(x, x, w, EPS, gate=g,
                                                     dgate=torch.ones_like(g))
    assert (dw == 0).all() and (dg == 0).all() and dr.shape == (0, H)
    codes, scales = nv.nvfp4_int8_quantize(torch.empty(0, 32, dtype=torch.bfloat16).cuda())
    assert codes.shape == (0, 32) and scales.shape == (0,)


def test_another_stream_and_a_graph(nv):
    """Calls on a side stream and captured calls replayed on changed inputs."""
    T, H = 64, 2048
    y, res, w = draw(1, T, H).cuda(), draw(2, T, H).cuda(), draw(3, H).cuda()
    want = nv.moe_nvfp4_post_norm(y, w, res, EPS, next_weight=w)
    dwant = nv.moe_nvfp4_post_norm_backward(res, y, w, EPS)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = nv.moe_nvfp4_post_norm(y, w, res, EPS, next_weight=w)
        b = nv.moe_nvfp4_post_norm_backward(res, y, w, EPS)
    s.synchronize()
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    assert torch.equal(b[0], dwant[0]) and torch.equal(b[1], dwant[1])
    yin = torch.zeros_like(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = nv.moe_nvfp4_post_norm(yin, w, res, EPS, next_weight=w)
        b = nv.moe_nvfp4_post_norm_backward(res, yin, w, EPS)
    yin.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    assert torch.equal(b[0], dwant[0]) and torch.equal(b[1], dwant[1])


@pytest.mark.parametrize("T,H", [(600, 6144), (3000, 1024), (40, 16384)])
def test_pre_norm_int8_codes_are_the_nearest(nv, T, H):
    """A code is the integer nearest to the fp32 quotient.  The row's r is a factor of both y
    and amax and cancels; x r, times w, 127 / amax and the quotient are rounded once each (y and
    amax each carry two of them): the quotient is off by at most 6 u of 127, 7 u with amax taken
    from a neighbour of the largest value."""
    x, w = draw(T + H, T, H), draw(H, H, std=0.1, mean=1.0)
    codes, _ = nv.moe_nvfp4_pre_norm_int8(x.cuda(), w.cuda(), EPS)
    y = w.double() * x.double()
    q = 127 * y / y.abs().amax(-1, keepdim=True)
    assert ((codes.cpu().double() - q).abs() <= 0.5 + 127 * 7 * U).all()


@pytest.mark.parametrize("H", [64, 1040, 1552, 6144, 32768])
def test_8_bit_rows_of_nan_and_infinity_show(nv, H):
    """A row with NaN or an infinity, and only such a row, gets the scale NaN: its products are
    NaN, as they are without the rounding to codes."""
    T, N = 7, 72
    x, w = draw(1, T, H), draw(2, H, std=0.1, mean=1.0)
    bad = x.clone()
    bad[1, H // 3], bad[2, H - 1], bad[4, 0], bad[5] = float("nan"), float("inf"), -float("inf"), 0
    bad[6] = float("nan")
    wq = torch.randint(-127, 128, (N, H), generator=torch.Generator().manual_seed(3),
                       dtype=torch.int8).cuda()
    ws = torch.ones(N, device="cuda")
    for rows in (nv.nvfp4_int8_quantize, lambda t: nv.moe_nvfp4_pre_norm_int8(t, w.cuda(), EPS)):
        cc, cs = rows(x.cuda())
        bc, bs = rows(bad.cuda())
        for t in (0, 3):
            assert torch.equal(bc[t], cc[t]) and bs[t] == cs[t]
        assert (bc[5] == 0).all() and bs[5] == 1
        out = nv.nvfp4_int8_matmul(bc, bs, wq, ws)
        for t in (1, 2, 4, 6):
            assert bs[t].isnan() and out[t].isnan().all(), t
        assert out[[0, 3, 5]].isfinite().all()


@pytest.mark.parametrize("H", [264, 2056, 6144, 16384])
def test_in_place_one_row(nv, H):
    """With one row, a channel gate has the shape of the rows: every output may be its tensor."""
    y, d, w, g = (draw(k, 1, H).cuda() for k in range(4))
    w = w[0].contiguous()
    want = nv.moe_nvfp4_post_norm_backward(d, y, w, EPS, gate=g, residual_scale=0.5)
    for name in ("dresidual", "dy", "dgate"):
        a = g.clone()
        got = nv.moe_nvfp4_post_norm_backward(d, y, w, EPS, gate=a, residual_scale=0.5,
                                              **{name: a})
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name
    want = nv.moe_nvfp4_post_norm(y, w, d, EPS, gate=g, next_weight=w)
    for name in ("out", "next_out"):
        a = g.clone()
        got = nv.moe_nvfp4_post_norm(y, w, d, EPS, gate=a, next_weight=w, **{name: a})
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name


@pytest.fixture
def no_nan(monkeypatch):
    """The comparisons of this module refuse NaN."""
    monkeypatch.setitem(globals(), "close", functools.partial(_no_nan, close))


def _no_nan(compare, got, ref, slack):
    assert not got.isnan().any()
    compare(got, ref, slack)


@pytest.mark.parametrize("H", [64, 2056, 6144])
def test_smallest_eps(nv, no_nan, H):
    """eps below fp32's normal range: rows of zeros give zeros and finite gradients, 1 / sqrt(eps)
    times the gradient of the normed row."""
    eps = 2.0 ** -130
    x, d, w = draw(1, 4, H), draw(2, 4, H, std=0.1), draw(3, H, std=0.1, mean=1.0)
    x[1] = 0
    g = draw(4, 4, 1, std=0.5, mean=0.5)
    assert (nv.moe_nvfp4_pre_norm(x.cuda(), w.cuda(), eps)[1] == 0).all()
    dx, _ = nv.moe_nvfp4_pre_norm_backward(d.cuda(), x.cuda(), w.cuda(), eps)
    dy, _, dg, _ = nv.moe_nvfp4_post_norm_backward(d.cuda(), x.cuda(), w.cuda(), eps,
                                                   gate=g.cuda())
    ref = 2.0 ** 65 * d[1].double() * w.double()
    close(dx[1], ref, E * ref.abs())
    ref = ref * g[1].double()
    close(dy[1], ref, E * ref.abs())
    assert dg[1] == 0
    # the other rows: eps is nothing beside mean(x^2)
    rx, rm, *_ = grads(x[[0, 2, 3]], w, None, d[[0, 2, 3]], 1.0)
    close(dx[[0, 2, 3]], rx, 2 * (E + EPS) * rm)


def test_a_gate_written_by_the_kernel_before(nv):
    """One row after another: a product writes the gate that the norm right behind it reads, into
    the memory that the norm before read its gate from."""
    H, n = 1024, 24
    y, res, w = draw(1, 1, H).cuda(), draw(2, 1, H).cuda(), draw(3, H, std=0.1, mean=1.0).cuda()
    src = [draw(10 + k, 1, H).cuda() for k in range(n)]
    gates = [nv.moe_nvfp4_pre_norm(s, w, EPS) for s in src]
    torch.cuda.synchronize()
    want = []
    for g in gates:
        want.append(nv.moe_nvfp4_post_norm(y, w, res, EPS, gate=g))
        torch.cuda.synchronize()
    gate = torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty_like(y) for _ in range(n)]

    def chain():
        for s, o in zip(src, outs):
            nv.moe_nvfp4_pre_norm(s, w, EPS, out=gate)
            nv.moe_nvfp4_post_norm(y, w, res, EPS, gate=gate, out=o)

    chain()
    torch.cuda.synchronize()
    assert all(torch.equal(o, v) for o, v in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(20):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))


# every (threads, vectors a thread) that row_shape gives, with few and with many rows: warp rows of
# 1 to 6 vectors, CTAs of up to 256 threads with 1 to 4, of up to 1024 threads with 1 to 4
LAYOUTS = [(5, 256), (5, 392), (5, 648), (9, 1000), (9, 1272), (9, 1536), (9, 1544), (300, 1544),
           (300, 2048), (200, 4096), (300, 6144), (160, 6152), (300, 8192), (9, 8200), (160, 8200),
           (160, 16384), (5, 16392), (160, 24576), (5, 24584)]


@pytest.mark.parametrize("gate", ["none", "1", "t", "h", "th"])
@pytest.mark.parametrize("T,H", LAYOUTS + SHAPES)
def test_post_norm_of_every_layout(nv, no_nan, T, H, gate):
    """T at least the SM count: rows of at most 8192 values take CTAs of 256 threads; fewer rows,
    or longer ones: of 1024."""
    test_post_norm(nv, T, H, gate)


@pytest.mark.parametrize("gate", ["none", "1", "t", "h", "th"])
@pytest.mark.parametrize("T,H", LAYOUTS + SHAPES)
def test_post_norm_backward_of_every_layout(nv, no_nan, T, H, gate):
    test_post_norm_backward(nv, T, H, gate)


@pytest.mark.parametrize("T,H", LAYOUTS + SHAPES)
def test_pre_norm_and_8_bit_rows_of_every_layout(nv, no_nan, T, H):
    test_pre_norm(nv, T, H)
    test_pre_norm_backward(nv, T, H, True)
    if H % 16 == 0:
        test_pre_norm_int8(nv, T, H)
        test_int8_quantize_is_exact(nv, T, H)


@pytest.mark.parametrize("T,H", [(5, 264), (700, 1032), (300, 2056)])
@pytest.mark.parametrize("gate", ["1", "t", "h", "th"])
def test_gradients_in_the_place_of_weight_and_gate(nv, T, H, gate):
    """dweight in weight's own tensor, dgate in gate's."""
    y, d, w = draw(1, T, H).cuda(), draw(2, T, H, std=0.1).cuda(), draw(3, H).cuda()
    g = gates(gate, T, H, 5).cuda()
    want = nv.moe_nvfp4_post_norm_backward(d, y, w, EPS, gate=g, residual_scale=0.5)
    a, b = w.clone(), g.clone()
    got = nv.moe_nvfp4_post_norm_backward(d, y, a, EPS, gate=b, residual_scale=0.5, dweight=a,
                                          dgate=b)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    want = nv.moe_nvfp4_pre_norm_backward(d, y, w, EPS)
    a = w.clone()
    got = nv.moe_nvfp4_pre_norm_backward(d, y, a, EPS, dweight=a)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("T,H", [(3, 264), (200, 2056)])
def test_gradients_through_next(nv, no_nan, T, H):
    """The gradient of next reaches the block through dskip: pre_norm's at out, added to dout,
    takes the place of dout.  out and that sum are rounded on the way (2^-8 of out moves n and r
    by as much, 2^-8 of the sum itself): 4 2^-8 of the terms' magnitudes bound both."""
    y, res, d, d2 = (draw(k, T, H) for k in range(4))
    w, w2 = draw(5, H, std=0.1, mean=1.0), draw(6, H, std=0.1, mean=1.0)
    c = lambda *ts: [t.cuda() for t in ts]
    out, _ = nv.moe_nvfp4_post_norm(*c(y, w, res), EPS, residual_scale=0.75, next_weight=w2.cuda())
    both, dw2 = nv.moe_nvfp4_pre_norm_backward(d2.cuda(), out, w2.cuda(), EPS, dskip=d.cuda())
    dy, dw, _, dr = nv.moe_nvfp4_post_norm_backward(both, *c(y, w), EPS, residual_scale=0.75)
    yd, wd, rd, vd = (t.double().requires_grad_() for t in (y, w, res, w2))
    o = 0.75 * rd + wd * yd * rms(yd)
    nxt = vd * o * rms(o)
    want = torch.autograd.grad([o, nxt], [yd, wd, rd, vd], [d.double(), d2.double()])
    # magnitudes: of d + r2 (dn + n |mean|) elementwise, through the norm's own gradient
    with torch.no_grad():
        _, m2, _, mw2, *_ = grads(o, w2, None, d2, 1.0)
        total = d.double().abs() + m2
        _, my, _, mw, *_ = grads(y, w, None, total, 1.0)
    for got, ref, mag in zip((dy, dw, dr, dw2), want, (my, mw, 0.75 * total, mw2)):
        close(got, ref, (4 * B + T * U) * mag)


def test_workspaces_that_are_no_tensors(nv):
    x, w = draw(1, 3, 64).cuda(), draw(2, 64).cuda()
    for bad in ([0] * 64, "workspace", np.zeros(1 << 20, np.uint8), torch.zeros(1 << 20).cuda(),
                torch.zeros(1 << 20, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            nv.moe_nvfp4_pre_norm_backward(x, x, w, EPS, workspace=bad)
