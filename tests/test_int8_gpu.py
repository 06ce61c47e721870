"""The product of 8-bit integers against exact integer sums, and the operators around a block
run together.

Sums are exact, so out differs from the real value by two fp32 products, the sum's conversion
to fp32 (2^-24 each) and one rounding to bf16: (2^-8 + 2^-22) |out|."""
import pytest
import torch

pytestmark = pytest.mark.gpu
B = 2.0 ** -8
EPS = 1e-5


@pytest.fixture(scope="module")
def nv():
    import bit_quantized_moe_nvfp4_b200 as m
    return m


def case(T, N, K, seed=0, full=False):
    g = torch.Generator().manual_seed(seed + T + N + K)
    lo, hi = (-127, 128)
    a = torch.randint(lo, hi, (T, K), generator=g, dtype=torch.int8)
    w = torch.randint(lo, hi, (N, K), generator=g, dtype=torch.int8)
    if full:
        a[:], w[:] = 127, 127
        w[::2] = -127
    return a, torch.rand(T, generator=g) + 0.1, w, torch.rand(N, generator=g) * 1e-3 + 1e-5


SHAPES = [(1, 8, 16), (1, 1000, 784), (2, 72, 2064), (16, 136, 128), (17, 264, 400), (33, 64, 128),
          (65, 328, 272), (129, 1000, 528), (300, 8, 16), (257, 2056, 336), (1000, 2064, 1040),
          (2049, 1032, 64), (4, 256, 32768), (2500, 2056, 144), (4100, 4104, 272)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("full", [False, True], ids=["random", "extreme"])
def test_int8_matmul(nv, T, N, K, full):
    a, sa, w, sw = case(T, N, K, full=full)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = nv.nvfp4_int8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), error_flag=flag)
    assert int(flag) == 0
    acc = (a.cuda().double() @ w.cuda().double().t()).cpu()
    ref = acc * sa.double()[:, None] * sw.double()
    assert ((out.cpu().double() - ref).abs() <= (B + 2.0 ** -22) * ref.abs()).all()


def test_int8_matmul_of_minus_128(nv):
    """Codes of -128, which the quantizer never gives, are taken as they are."""
    a = torch.full((3, 64), -128, dtype=torch.int8)
    out = nv.nvfp4_int8_matmul(a.cuda(), torch.ones(3).cuda(), a[:1].repeat(8, 1).cuda(),
                               torch.ones(8).cuda())
    assert (out == 128 * 128 * 64).all()


def test_both_kernels_agree_on_rows(nv):
    """A token's result does not depend on how many tokens come with it."""
    a, sa, w, sw = (t.cuda() for t in case(2300, 2048, 512))
    whole = nv.nvfp4_int8_matmul(a, sa, w, sw)
    for n in (1, 9, 40, 100, 130):
        assert torch.equal(nv.nvfp4_int8_matmul(a[:n], sa[:n], w, sw), whole[:n])


def test_output_ends_where_it_ends(nv):
    for T, N in ((5, 72), (300, 2056)):
        a, sa, w, sw = (t.cuda() for t in case(T, N, 144))
        buf = torch.full((T + 8, N), 7.0, dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_int8_matmul(a, sa, w, sw, out=buf[:T])
        assert (buf[T:] == 7).all()


def test_results_beyond_32_bit_offsets(nv):
    T, N, K = 262200, 8200, 16
    a, sa, w, sw = case(T, N, K)
    out = nv.nvfp4_int8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda())
    for t in (0, 131072, 261889, T - 1):
        ref = (a[t].double() @ w.double().t()) * sa[t].double() * sw.double()
        assert ((out[t].cpu().double() - ref).abs() <= (B + 2.0 ** -22) * ref.abs()).all()


def test_zero_tokens(nv):
    _, _, w, sw = case(1, 64, 64)
    out = nv.nvfp4_int8_matmul(torch.empty(0, 64, dtype=torch.int8).cuda(),
                               torch.empty(0).cuda(), w.cuda(), sw.cuda())
    assert out.shape == (0, 64)


def test_other_streams_and_a_graph(nv):
    for T in (7, 700):
        a, sa, w, sw = (t.cuda() for t in case(T, 2048, 768))
        want = nv.nvfp4_int8_matmul(a, sa, w, sw)
        torch.cuda.synchronize()
        outs = []
        for _ in range(2):
            with torch.cuda.stream(torch.cuda.Stream()):
                outs.append(nv.nvfp4_int8_matmul(a, sa, w, sw))
        ain = torch.zeros_like(a)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(nv.nvfp4_int8_matmul(ain, sa, w, sw))
        ain.copy_(a)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("T", [1, 40, 700])
def test_a_block_between_its_norms(nv, T):
    """pre-norm -> gated projection (bf16) -> 8-bit down projection -> post-norm with a gate
    and the next pre-norm, as a decoder layer runs them, against 64 bits.

    2-norm bound: roundings of the normed rows, of h and of the block's output (2^-8 each, two
    factors h = act(g) u of the first), the 8-bit step of h's rows, and the result's."""
    H, I = 512, 1024
    gen = torch.Generator().manual_seed(T)
    r = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=gen) * std + mean).bfloat16()
    x, w1, w2, w3 = r(T, H), r(H, std=0.1, mean=1.0), r(H, std=0.1, mean=1.0), r(H, std=0.1, mean=1.0)
    w_gu, gate = r(2 * I, H, std=H ** -0.5), r(1, H, std=0.1, mean=0.5)
    w_dn = r(H, I, std=I ** -0.5)
    wq, ws = nv.nvfp4_int8_quantize(w_dn.cuda())
    n1 = nv.moe_nvfp4_pre_norm(x.cuda(), w1.cuda(), EPS)
    h = nv.moe_nvfp4_gate_up(n1, w_gu.cuda())
    y = nv.nvfp4_int8_matmul(*nv.nvfp4_int8_quantize(h), wq, ws)
    out, nxt = nv.moe_nvfp4_post_norm(y, w2.cuda(), x.cuda(), EPS, gate=gate.cuda(),
                                      residual_scale=0.5, next_weight=w3.cuda())
    q, s = nv.moe_nvfp4_pre_norm_int8(x.cuda(), w1.cuda(), EPS)
    d = lambda t: t.double()
    norm = lambda t: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)
    n1d = norm(d(x)) * d(w1)
    z = n1d @ d(w_gu).t()
    hd = z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
    yd = hd @ (wq.cpu().double() * ws.cpu().double()[:, None]).t()
    od = 0.5 * d(x) + d(gate) * (norm(yd) * d(w2))
    nd = norm(od) * d(w3)
    step = hd.abs().amax(-1, keepdim=True) / 127 / 12 ** 0.5     # rms of the rounding to codes
    rel8 = float((step * I ** 0.5).norm() / hd.norm())
    bound = 6 * B + 1.5 * rel8
    for got, ref in ((out, od), (nxt, nd)):
        err = float((got.cpu().double() - ref).norm() / ref.norm())
        assert err <= bound, (err, bound)
    deq = q.cpu().double() * s.cpu().double()[:, None]
    assert ((deq - n1d).abs() <= 0.51 * s.cpu().double()[:, None]).all()


def test_binding_refuses_what_does_not_fit(nv):
    """Shapes, types, strides and mixed devices, each with a ValueError; wrong numbers of rows
    and the library's own limits with its status."""
    a, sa, w, sw = (t.cuda() for t in case(3, 64, 64))
    x, wt = torch.zeros(3, 64).bfloat16().cuda(), torch.ones(64).bfloat16().cuda()
    wg = torch.zeros(32, 64).bfloat16().cuda()
    bad = [lambda: nv.nvfp4_int8_matmul(a, sa, w[:, :32].contiguous(), sw),
           lambda: nv.nvfp4_int8_matmul(a, sa, w.cpu(), sw),
           lambda: nv.nvfp4_int8_matmul(a, sa[:2], w, sw),
           lambda: nv.nvfp4_int8_matmul(a, sa, w, sw.double()),
           lambda: nv.nvfp4_int8_matmul(a.t(), sa, w, sw),
           lambda: nv.nvfp4_int8_matmul(a, sa, w, sw, out=torch.empty(3, 64).cuda()),
           lambda: nv.nvfp4_int8_quantize(x[:, ::2]), lambda: nv.nvfp4_int8_quantize(x[0]),
           lambda: nv.moe_nvfp4_pre_norm(x.float(), wt, EPS),
           lambda: nv.moe_nvfp4_pre_norm(x, wt[:32], EPS),
           lambda: nv.moe_nvfp4_post_norm(x, wt, x, EPS, gate=x[:2]),
           lambda: nv.moe_nvfp4_post_norm(x, wt, x, EPS, next_out=x),
           lambda: nv.moe_nvfp4_post_norm_backward(x, x, wt, EPS, dgate=x),
           lambda: nv.moe_nvfp4_pre_norm_backward(x, x, wt, EPS, workspace=x),
           lambda: nv.moe_nvfp4_gate_up(x, wg[:31]), lambda: nv.moe_nvfp4_gate_up(x, wg.t()),
           lambda: nv.moe_nvfp4_gate_up_backward(x, x, wg, x)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    for call in (lambda: nv.moe_nvfp4_pre_norm_backward(x, x, wt, EPS, workspace=small),
                 lambda: nv.moe_nvfp4_gate_up(x, wg, act=5), lambda: nv.moe_nvfp4_pre_norm(x, wt, 0.0),
                 lambda: nv.moe_nvfp4_gate_up(x[:, :36].contiguous(), wg[:, :36].contiguous())):
        with pytest.raises(nv.NVFP4Error):
            call()


def test_many_calls_on_several_streams(nv):
    """Every operator, few and many tokens, again and again on three streams at once: each
    result is bit for bit what the operator gives alone."""
    H, I, N = 512, 768, 1032
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()
    w, w_gu, gate = r(H), r(2 * I, H) * 0.05, r(1, H)
    wq = torch.randint(-127, 128, (N, H), generator=g, dtype=torch.int8).cuda()
    ws = torch.rand(N, generator=g).cuda()

    def step(x, dh):
        T = x.shape[0]
        y = nv.moe_nvfp4_pre_norm(x, w, EPS)
        gu = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
        h = nv.moe_nvfp4_gate_up(y, w_gu, gu=gu)
        dx, dw = nv.moe_nvfp4_gate_up_backward(dh, y, w_gu, gu)
        q = nv.nvfp4_int8_matmul(*nv.moe_nvfp4_pre_norm_int8(x, w, EPS), wq, ws)
        o = nv.moe_nvfp4_post_norm(y, w, x, EPS, gate=gate, next_weight=w)
        b = nv.moe_nvfp4_post_norm_backward(dx, y, w, EPS, gate=gate)
        return (y, gu, h, dx, dw, q) + o + b

    sizes = (1, 40, 1500)
    data = [(r(T, H), r(T, I)) for T in sizes]
    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    for _ in range(5):
        got = []
        for k in range(4):
            for s, d in zip(streams, data[k % 3:] + data[:k % 3]):
                with torch.cuda.stream(s):
                    got.append((len(d[0]), step(*d)))
        torch.cuda.synchronize()
        for T, o in got:
            assert all(torch.equal(p, q) for p, q in zip(o, want[sizes.index(T)]))


def test_weights_written_by_the_kernel_before(nv):
    """Weights that the launch directly before writes, over and over into the same memory: the
    product takes the new ones (it asks its first weights into L2 before that launch ends)."""
    N, K, n = 4096, 1024, 12
    g = torch.Generator().manual_seed(1)
    ws_in = [torch.randn(N, K, generator=g).bfloat16().cuda() for _ in range(n)]
    a, sa, _, _ = (t.cuda() for t in case(3, 8, K))
    want = []
    for w in ws_in:
        wq, ws = nv.nvfp4_int8_quantize(w)
        torch.cuda.synchronize()
        want.append(nv.nvfp4_int8_matmul(a, sa, wq, ws))
    wq = torch.empty(N, K, dtype=torch.int8, device="cuda")
    ws = torch.empty(N, device="cuda")
    outs = [torch.empty(3, N, dtype=torch.bfloat16, device="cuda") for _ in range(n)]

    def chain():
        for w, o in zip(ws_in, outs):
            nv.nvfp4_int8_quantize(w, codes=wq, scales=ws)
            nv.nvfp4_int8_matmul(a, sa, wq, ws, out=o)

    chain()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(20):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_calls_from_another_current_device(nv, monkeypatch):
    """A call on tensors of a device that is not the current one is made again with it current
    and gives the same (the other device is feigned: the first look answers 1)."""
    a, sa, w, sw = (t.cuda() for t in case(5, 64, 64))
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()
    x, d, wt, gate, wg, dh, gu = r(5, 64), r(5, 64), r(64), r(1, 64), r(32, 64), r(5, 16), r(5, 32)
    calls = [lambda: nv.nvfp4_int8_quantize(x), lambda: nv.nvfp4_int8_matmul(a, sa, w, sw),
             lambda: nv.moe_nvfp4_pre_norm(x, wt, EPS), lambda: nv.moe_nvfp4_pre_norm_int8(x, wt, EPS),
             lambda: nv.moe_nvfp4_pre_norm_backward(d, x, wt, EPS, dskip=d),
             lambda: nv.moe_nvfp4_post_norm(x, wt, d, EPS, gate=gate, residual_scale=0.5,
                                            next_weight=wt),
             lambda: nv.moe_nvfp4_post_norm_backward(d, x, wt, EPS, gate=gate, residual_scale=0.5),
             lambda: nv.moe_nvfp4_gate_up(x, wg, act=nv.ACT_GELU),
             lambda: nv.moe_nvfp4_gate_up_backward(dh, x, wg, gu, act=nv.ACT_GELU)]
    for call in calls:
        want = call()
        looks = iter([1, 0])
        with monkeypatch.context() as m:
            m.setattr(nv, "_current_device", lambda: next(looks))
            got = call()
        assert next(looks, None) is None   # looked twice: refused, then taken
        for p, q in zip(*(t if isinstance(t, tuple) else (t,) for t in (got, want))):
            assert torch.equal(p, q)


def test_scales_written_by_the_kernel_before(nv):
    """Token after token through the same buffers: the product takes the codes and the scale
    that the launch before it has just written, not those of the token before."""
    N, K, n = 4096, 1024, 24
    _, _, w, sw = (t.cuda() for t in case(1, N, K))
    g = torch.Generator().manual_seed(2)
    xs = [(torch.randn(1, K, generator=g) * 2.0 ** (k % 7)).bfloat16().cuda() for k in range(n)]
    want = []
    for x in xs:
        q, s = nv.nvfp4_int8_quantize(x)
        torch.cuda.synchronize()
        want.append(nv.nvfp4_int8_matmul(q, s, w, sw))
        torch.cuda.synchronize()
    q = torch.empty(1, K, dtype=torch.int8, device="cuda")
    s = torch.empty(1, device="cuda")
    outs = [torch.empty(1, N, dtype=torch.bfloat16, device="cuda") for _ in range(n)]

    def chain():
        for x, o in zip(xs, outs):
            nv.nvfp4_int8_quantize(x, codes=q, scales=s)
            nv.nvfp4_int8_matmul(q, s, w, sw, out=o)

    chain()
    torch.cuda.synchronize()
    assert all(torch.equal(o, v) for o, v in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(50):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))


FIRST_CALLS_IN_A_CAPTURE = """
import torch
import bit_quantized_moe_nvfp4_b200 as nv
g = torch.Generator().manual_seed(1)
r = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()
def data(T):
    return r(T, 512), r(512), r(1, 512), r(2 * 640, 512) * 0.05, r(T, 640)
def run(x, w, gate, wg, dh):
    y = nv.moe_nvfp4_pre_norm(x, w, 1e-5)
    gu = torch.empty(len(x), 1280, dtype=torch.bfloat16, device="cuda")
    h = nv.moe_nvfp4_gate_up(y, wg, gu=gu)
    q, s = nv.nvfp4_int8_quantize(h)
    z = nv.nvfp4_int8_matmul(q, s, q[:8].contiguous(), s[:8].contiguous())
    dx, dw = nv.moe_nvfp4_gate_up_backward(dh, y, wg, gu)
    out = nv.moe_nvfp4_post_norm(dx, w, x, 1e-5, gate=gate, next_weight=w)
    return (h, z, dx, dw) + out + nv.moe_nvfp4_post_norm_backward(x, dx, w, 1e-5, gate=gate)
sets = [data(T) for T in (9, 1700)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = [run(*d) for d in sets]
graph.replay()
torch.cuda.synchronize()
for o, d in zip(got, sets):
    assert all(torch.equal(p, q) for p, q in zip(o, run(*d)))
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """What a launch looks up once (maps, limits, residency) may be looked up in a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_IN_A_CAPTURE], cwd=root, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.endswith("same\n"), r.stderr[-2000:]


def test_calls_from_several_host_threads(nv):
    """Four threads, each on its own stream, sizes in another order: every result is the one that
    a call alone gives."""
    import threading
    H, I = 512, 768
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()
    w, wg = r(H), r(2 * I, H) * 0.05
    wq, ws = nv.nvfp4_int8_quantize(r(1032, I))

    def step(x):
        h = nv.moe_nvfp4_gate_up(nv.moe_nvfp4_pre_norm(x, w, EPS), wg)
        return (h, nv.nvfp4_int8_matmul(*nv.nvfp4_int8_quantize(h), wq, ws)) + \
            nv.moe_nvfp4_pre_norm_backward(x, x, w, EPS)

    xs = [r(T, H) for T in (1, 30, 200, 1100)]
    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def worker(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for n in range(12):
                    i = (n + k) % len(xs)
                    got = step(xs[i])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(p, q) for p, q in zip(got, want[i])):
                        wrong.append((k, n))
        except Exception as e:   # a thread's failure has to reach the test
            wrong.append((k, repr(e)))

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("T,K", [(3, 16), (130, 16), (130, 32768)])
def test_largest_channels(nv, T, K):
    """N at its limit (K at its limit: 32768 channels), the last channels among the rest."""
    N = 1 << 24 if K == 16 else 1 << 15
    g = torch.Generator(device="cuda").manual_seed(T)
    a = torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int8, device="cuda")
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
    sa = torch.rand(T, generator=g, device="cuda") + 0.1
    sw = torch.rand(N, generator=g, device="cuda") + 0.1
    out = nv.nvfp4_int8_matmul(a, sa, w, sw)
    for n0 in (0, N // 2 - 64, N - 4096):
        n1 = n0 + 4096
        ref = (a.double() @ w[n0:n1].double().t()) * sa.double()[:, None] * sw[n0:n1].double()
        assert ((out[:, n0:n1].double() - ref).abs() <= (B + 2.0 ** -22) * ref.abs()).all()
