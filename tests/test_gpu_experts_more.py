"""Router logits at the ends of the range, SwiGLU where its denominator is near the largest number."""
import math

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


# ---------------------------------------------------------------- router
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(14, 48, 6), (200, 48, 6), (3000, 60, 4), (2500, 256, 8), (400, 300, 5), (40, 1000, 12)])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route_ends_of_the_range(T, E, k, score, renorm, dtype):
    """Infinities, the largest and the lowest number, masked and NaN logits: one CTA, a warp a token, eight lanes a token."""
    x = (torch.randn(T, E, generator=_gen(T), device="cuda") * 2).to(dtype)
    fin = torch.finfo(dtype)
    x[torch.rand(T, E, generator=_gen(2), device="cuda") < 0.3] = -math.inf
    for r, t in enumerate(range(0, T, 14)):       # (sets of rows, the last may be short)
        rows = x[t:t + 14]
        for i, row in enumerate(rows):
            if i == 0:
                row[9] = math.inf                 # all the weight
            elif i == 1:
                row[10:13] = math.inf             # equal shares
            elif i == 2:
                row[7], row[20] = fin.max, math.inf   # infinity is above every number
            elif i == 3:
                row[5:9] = fin.max
            elif i == 4:
                row[:] = fin.min
            elif i == 5:
                row[:] = -math.inf
                row[3] = fin.min
            elif i == 6:
                row[:] = math.inf
            elif i == 7:
                row[:k] = math.nan
            elif i == 8:
                row[:] = math.nan
                row[E - 1] = math.inf
            elif i == 9:
                row[:] = -math.inf
    r = uw.uw_route(x, k, score=score, renorm=renorm)
    ids, w, offsets, rows, pos = U.route_ref(x.double().cpu().numpy(), k, score, renorm, 1.0)
    for got, want, name in ((r.ids, ids, "ids"), (r.offsets, offsets, "offsets"), (r.rows, rows, "rows"), (r.pos, pos, "pos")):
        assert np.array_equal(got.cpu().numpy(), want), name
    got = r.weights.double().cpu().numpy()
    # finite logits that carry weight are within 32 of each other: exp off by 2 ulps, its argument by 2^-24 32; the sum of
    # E terms by (E/32 + 5) 2^-24, divisions by 1; weights below the normal range by their spacing
    assert np.isfinite(got).all()
    assert (np.abs(got - w) <= (2 * 32 + 16 + E / 16) * 2.0 ** -24 * np.abs(w) + 2.0 ** -126).all(), float(np.abs(got - w).max())


# ---------------------------------------------------------------- SwiGLU
def test_swiglu_where_the_denominator_nears_the_largest_number():
    """silu(g) for g from -86 to -88.5 is about g e^g, 1e-36 to 1e-37; times an up projection of 2^123 it is of order 1."""
    K, N, g = 64, 64, [-86.0, -87.0, -87.5, -88.0, -88.5, -30.0, 3.0, 0.0, -0.0, 88.0, 120.0]
    X = torch.zeros(len(g), K, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = torch.tensor(g, device="cuda")
    X[:, 1] = 1.0
    W = torch.zeros(2, 1, N, K, dtype=torch.bfloat16, device="cuda")
    W[0, :, :, 0] = 1.0
    W[1, :, :, 1] = 2.0 ** 123
    off = torch.tensor([0, len(g)], dtype=torch.int32, device="cuda")
    y = uw.uw_gemm_grouped(X, W[0], off, up=W[1], out_f32=True)
    gd, ud = X.double() @ W[0, 0].double().T, X.double() @ W[1, 0].double().T
    zero = torch.zeros_like(gd)
    ref, tol = U.swiglu_ref(gd, ud), U.swiglu_tolerance(gd, ud, zero, zero)
    over = ref > torch.finfo(torch.float32).max     # 88 2^123 = 2^129.5 and 120 2^123 pass the type's range
    assert over.any(1).tolist() == [False] * 9 + [True] * 2 and y[over].isposinf().all()
    U.check(y[~over], ref[~over], tol[~over])


def test_swiglu_beyond_the_exponential():
    """e^-g past the largest number: 0, as with the plain formula in fp32; infinities and NaN as it gives them."""
    K, N, g = 64, 64, [-89.0, -1000.0, -3e38, 3e38, math.inf, -math.inf, math.nan]
    X = torch.zeros(len(g), K, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = torch.tensor(g, device="cuda")
    X[:, 1] = 1.0
    W = torch.zeros(2, 1, N, K, dtype=torch.bfloat16, device="cuda")
    W[0, :, :, 0] = 1.0
    W[1, :, :, 1] = 1.0
    W[1, :, :, 0] = 0.0
    off = torch.tensor([0, len(g)], dtype=torch.int32, device="cuda")
    y = uw.uw_gemm_grouped(X[:4], W[0], torch.tensor([0, 4], dtype=torch.int32, device="cuda"), up=W[1], out_f32=True)
    assert (y[:3] == 0).all() and torch.equal(y[3], X[3, 0].float().expand(N))
    z = uw.uw_gemm_grouped(X, W[0], off, up=W[1], out_f32=True)
    assert torch.equal(z[:4], y) and z[4:].isnan().all()   # (an infinity of X times the up weight 0 is NaN)
