"""Grouped and 4-bit products on whole numbers: every sum is exact in fp32 in any
order, so one product left out, taken twice or scaled wrongly shows, and so does
an output that was not written."""
import numpy as np
import pytest
import torch

import decode_gemm_bf16_b200 as uw
from tests import expert_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert uw.uw_last_device_status() == 0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(M, K, seed, step=1.0):
    """Whole numbers from -3 to 3, times a power of two: exact in BF16, in two 8-bit halves and in 4 bits."""
    return (torch.randint(-3, 4, (M, K), generator=_gen(seed), device="cuda") * step).to(torch.bfloat16)


def _weights(E, N, K, seed):
    """Whole numbers from -3 to 3, every block of 32 times 1, 2 or 4: exact in BF16 and in 4 bits; below 2^24 in sums of K < 2^17."""
    w = torch.randint(-3, 4, (E, N, K), generator=_gen(seed), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    s = torch.randint(0, 3, (E, N, K // 32), generator=_gen(seed + 1), device="cuda").to(torch.bfloat16)
    return w * torch.exp2(s).repeat_interleave(32, -1)


def _offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def _nan(*shape, f32):
    return torch.full(shape, float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")


def _same(y, ref):
    ref = ref.to(y.dtype)   # an exact sum, rounded once
    bad = ~(y == ref)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}: {y[bad][0]} for {ref[bad][0]}"


def _mx_gemm_is_exact(M, N, K, xmx, seed=0):
    X, W = _rows(M, K, seed), _weights(1, N, K, seed + 1)[0]
    Wm = uw.uw_mx_quantize(W)
    assert torch.equal(uw.uw_mx_dequantize(Wm), W)
    ref = X.double() @ W.double().T
    for f32 in (True, False):
        _same(uw.uw_mx_gemm(uw.uw_mx_quantize(X) if xmx else X, Wm, out=_nan(M, N, f32=f32), out_f32=f32), ref)
        assert uw.uw_last_device_status() == 0


def _grouped_is_exact(sizes, N, K, mx, up, gather, seed=0):
    E, R = len(sizes), int(sum(sizes))
    T = max(1, R // 3) if gather else R
    X = _rows(T, K, seed, 2.0 ** -6 if up else 1.0)
    rows = torch.randint(0, T, (R,), generator=_gen(seed), device="cuda").int() if gather else None
    W = [_weights(E, N, K, seed + 2 + 2 * i) for i in range(2 if up else 1)]
    off = _offsets(sizes)
    y = uw.uw_gemm_grouped(X, uw.uw_mx_quantize(W[0]) if mx else W[0], off, rows=rows,
                           up=(uw.uw_mx_quantize(W[1]) if mx else W[1]) if up else None, out=_nan(R, N, f32=True), out_f32=True)
    assert uw.uw_last_device_status() == 0
    Xs = (X if rows is None else X[rows.long()]).double()
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        g, *u = [Xs[lo:hi] @ w[e].double().T for w in W]
        if up:   # exact sums through the SwiGLU
            zero = torch.zeros_like(g)
            U.check(y[lo:hi], U.swiglu_ref(g, u[0]), U.swiglu_tolerance(g, u[0], zero, zero))
        else:
            _same(y[lo:hi], g)


# ---------------------------------------------------------------- few tiles left over, few k steps
@pytest.mark.parametrize("M,N,K,xmx", [(337, 14336, 4096, False), (400, 14336, 4096, False), (448, 14336, 4096, False),
                                       (1500, 4096, 4096, False), (150, 9728, 2560, False), (112, 85, 2560, False),
                                       (256, 28672, 8192, True), (375, 9626, 6976, True)])
def test_mx_gemm_parts_of_few_steps(M, N, K, xmx):
    _mx_gemm_is_exact(M, N, K, xmx)


@pytest.mark.parametrize("sizes,N,K,up", [([256], 256, 2048, False), ([256], 19200, 4096, False), ([130, 0, 126], 9472, 2048, False),
                                          ([130, 126], 4800, 2048, True)])
@pytest.mark.parametrize("mx", [False, True])
def test_grouped_parts_of_few_steps(sizes, N, K, up, mx):
    _grouped_is_exact(sizes, N, K, mx, up, True)


# ---------------------------------------------------------------- pairs of CTAs that have nothing to do
@pytest.mark.parametrize("M,N,K,xmx", [(100, 40, 128, False), (65, 300, 2048, False), (1, 64, 64, True), (200, 520, 512, True)])
def test_most_pairs_idle(M, N, K, xmx):
    """A tile or a few among 74 pairs, call after call: a pair leaves right after it has started."""
    X, W = _rows(M, K, 1), _weights(1, N, K, 2)[0]
    Xq, Wm = uw.uw_mx_quantize(X) if xmx else X, uw.uw_mx_quantize(W)
    out = _nan(M, N, f32=True)
    for i in range(600):
        if i % 100 == 0:
            out.fill_(float("nan"))
        uw.uw_mx_gemm(Xq, Wm, out=out, out_f32=True)
    _same(out, X.double() @ W.double().T)


def test_most_pairs_idle_bf16():
    _grouped_is_exact([0, 70, 0, 65], 200, 320, False, False, False)
    X, W, off = _rows(135, 320, 1), _weights(4, 200, 320, 2), _offsets([0, 70, 0, 65])
    y = uw.uw_gemm_grouped(X, W, off, out_f32=True)
    for _ in range(600):
        z = uw.uw_gemm_grouped(X, W, off, out_f32=True)
    assert torch.equal(y, z)
    empty = _offsets([0, 0, 0, 0])    # no pair has a tile
    for _ in range(200):
        out = uw.uw_gemm_grouped(X, W, empty, out=y, out_f32=True)
    assert torch.equal(out, z)


# ---------------------------------------------------------------- scales of two weights
@pytest.mark.parametrize("sizes,N,K", [([130, 70, 0, 200], 200, 384), ([100] * 5, 64, 128), ([300], 1000, 2048), ([0, 90, 85], 129, 1152),
                                       ([20, 30], 200, 1152), ([1, 2, 3], 328, 2048), ([60, 50], 1408, 640)])
def test_scales_of_gate_and_up(sizes, N, K):
    """Blocks of 32 weights scaled by 1, 2 or 4 at random, in gate and in up: single CTAs and pairs, rings of odd length,
    an odd multiple of 128 along K, half a scale tile of rows, experts without slots."""
    for seed in range(3):
        _grouped_is_exact(sizes, N, K, True, True, seed % 2 == 0, seed=100 * seed)


def test_many_stages_of_gate_and_up():
    _grouped_is_exact([40] * 16, 704, 4096, True, True, True, seed=5)
    _grouped_is_exact([180, 230, 97, 400], 1408, 4096, True, True, True, seed=6)


# ---------------------------------------------------------------- waits that run out
_EXPIRED_CHILD = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
import decode_gemm_bf16_b200 as uw
from tests import test_gpu_experts_exact as E

def product(M, N, K, mx, up):
    X, W = E._rows(M, K, 1), E._weights(1, N, K, 2)
    Wq = uw.uw_mx_quantize(W) if mx else W
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    y = uw.uw_gemm_grouped(X, Wq, off, up=Wq if up else None, out_f32=True)
    return y, X.double() @ W[0].double().T

for case in ((4, 640, 8192, False, False), (4, 640, 8192, True, False), (4, 640, 8192, True, True), (4, 640, 8256, True, False),
             (256, 256, 4096, False, False), (200, 300, 8192, True, False), (200, 300, 8192, True, True)):
    product(*case)                        # cut along k: the joining worker waits in vain
    print("expired", uw.uw_last_device_status())
    y, ref = product(100, 200, 128, case[3], False)   # too short to be cut
    print("after", uw.uw_last_device_status(), int((y.double() == ref).all()))
"""


def test_waits_that_run_out_are_reported_and_harm_nothing():
    """Partial sums that nobody publishes (the UW_DEBUG_SKIP_TAGS hook): single CTAs and pairs, BF16 and 4-bit weights, gate
    and up, end with UW_ERR_TIMEOUT, and the next call is right.  In a child process: hook and limit stay out of the others."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, UW_TIMEOUT_MS="20", UW_DEBUG_SKIP_TAGS="1")
    r = subprocess.run([sys.executable, "-c", _EXPIRED_CHILD, root], env=env, capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-3000:]
    lines = r.stdout.strip().splitlines()
    assert lines[0::2] == ["expired 7"] * 7 and lines[1::2] == ["after 0 1"] * 7, r.stdout


def test_small_rebuilt_tiles_on_two_streams():
    """K an odd multiple of 64 and few rows (the least shared memory of all forms), tiles cut along k, on two streams at once."""
    cases = []
    for seed, (M, N, K) in enumerate([(3, 700, 4160), (16, 900, 2112), (1, 2000, 8256)]):
        X, W = _rows(M, K, seed), _weights(1, N, K, seed + 5)[0]
        cases.append((X, uw.uw_mx_quantize(W), X.double() @ W.double().T))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(60):
        for j, s in enumerate(streams):
            X, W, ref = cases[(i + j) % 3]
            with torch.cuda.stream(s):
                got.append((uw.uw_mx_gemm(X, W, out_f32=True), ref))
    torch.cuda.synchronize()
    for y, ref in got:
        _same(y, ref)
