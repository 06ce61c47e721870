"""The device-side failure path on the GPU, made to happen on purpose without a fault.

Every wait in the library's kernels is bounded by wall-clock time.  The test hook
nvfp4_selftest_wait_timeout runs each kind of wait (an mbarrier phase no thread arrives at,
bulk-copy bytes that never land, a grid-wide counter no CTA advances) with a 2 ms limit and
nothing to complete it: the kernel must return on its own, record bit 1 in the flag, and
leave the context usable, so that the next forward on the same workspace runs, matches the
oracle and clears the flag."""
import time

import pytest
import torch

import synth
from helpers import Layer, compare_moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_quantized_moe_nvfp4_b200 as m
    return m


@pytest.mark.parametrize("kind", [0, 1, 2], ids=["mbarrier", "bulk_bytes", "counter"])
def test_wait_gives_up_and_context_survives(nv, kind):
    E, H, I, K, T = 8, 192, 128, 4, 3
    layer = Layer(E, H, I, seed=31)
    x = synth.activations_bf16(T, H, 31)
    ids, w = synth.routing(T, E, K, seed=31)
    ws = nv.alloc_moe_workspace(T, H, I, E, K)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    nv.nvfp4_selftest_wait_timeout(ws, kind, 2_000_000)     # 2 ms
    flag = nv.moe_nvfp4_read_error_flag(ws)                 # synchronises: the kernel ended
    elapsed = time.perf_counter() - t0
    assert flag == 2
    assert elapsed < 1.0
    for path in (nv.PATH_GEMV, nv.PATH_GEMM):
        out = nv.moe_nvfp4_forward(x.cuda(), ids.cuda(), w.cuda(), *layer.dev, workspace=ws,
                                   path=path)
        assert nv.moe_nvfp4_read_error_flag(ws) == 0
        ref, ref64, _ = layer.oracle_forward(x, ids, w)
        compare_moe(out, ref, ref64)


def lost_or_right(got, want):
    """Each element is what the call gives or NaN; the share that is NaN."""
    gone = got.isnan()
    assert torch.equal(got[~gone], want[~gone])
    return float(gone.float().mean())


# few tokens: every column tile of the split kernel, one CTA and several a cluster (each cluster
# loses a part of every tile); many tokens: pairs of CTAs, whose first tiles are there
@pytest.mark.parametrize("T,H,I", [(1, 2048, 72), (17, 64, 136), (40, 1024, 2056),
                                   (4100, 136, 2056)])
def test_a_lost_tile_of_the_gated_projection_is_nan(nv, T, H, I):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    w = (torch.randn(2 * I, H, generator=g) * H ** -0.5).bfloat16().cuda()
    gu = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    h = nv.moe_nvfp4_gate_up(x, w, gu=gu)
    a, b = torch.full_like(h, 7), torch.full_like(gu, 7)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    nv.nvfp4_selftest_gate_up_timeout(x, w, a, b, flag)
    assert int(flag) == 2 and time.perf_counter() - t0 < 1.0
    for got, want in ((a, h), (b, gu)):
        share = lost_or_right(got, want)
        assert share == 1 if T < 100 else 0.5 < share < 0.9, share
    assert torch.equal(nv.moe_nvfp4_gate_up(x, w), h)   # the context goes on


@pytest.mark.parametrize("T,N,K", [(1, 1000, 2064), (17, 264, 128), (40, 4096, 1040),
                                   (4100, 4104, 272)])
def test_a_lost_tile_of_the_8_bit_product_is_nan(nv, T, N, K):
    g = torch.Generator().manual_seed(T)
    a, w = (torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).cuda() for n in (T, N))
    sa, sw = torch.rand(T, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    want = nv.nvfp4_int8_matmul(a, sa, w, sw)
    got = torch.full_like(want, 7)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    nv.nvfp4_selftest_int8_matmul_timeout(a, sa, w, sw, got, flag)
    assert int(flag) == 2 and time.perf_counter() - t0 < 1.0
    share = lost_or_right(got, want)
    assert share == 1 if T < 100 else 0.5 < share < 0.9, share
    assert torch.equal(nv.nvfp4_int8_matmul(a, sa, w, sw), want)
