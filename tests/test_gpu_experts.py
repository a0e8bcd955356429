"""The microscaled 4-bit form and the expert layer against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import decode_gemm_bf16_b200 as uw
from tests import expert_util as U

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(*shape, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=_gen(seed), device="cuda") * scale).to(torch.bfloat16)


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert uw.uw_last_device_status() == 0


# ---------------------------------------------------------------- quantisation
def _special_rows(K):
    """Values at and beside every border of the rounding, extremes of the range, zeros of both signs, NaN, infinities."""
    t = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.9375, 4, 0, -0.0, -0.25, -0.75, -5.0625])
    rows = []
    for s in (-134, -133, -127, -126, -100, -3, 0, 1, 60, 120, 125):
        r = np.zeros(K)
        r[:16] = t * 2.0 ** s
        r[16:32] = t * 2.0 ** s * (1 + 2.0 ** -7)
        r[32:48] = -t * 2.0 ** s * (1 - 2.0 ** -8)
        rows.append(r)
    for bad in (np.nan, np.inf, -np.inf):
        r = np.linspace(-3, 3, K)
        r[40] = bad
        rows.append(r)
    rows.append(np.zeros(K))
    rows.append(np.full(K, -0.0))
    return np.stack(rows)


@pytest.mark.parametrize("rows,K", [(1, 64), (1, 4096), (3, 192), (37, 320), (127, 64), (128, 256), (129, 512), (300, 1088)])
@pytest.mark.parametrize("f32", [False, True])
def test_mx_quantize_bytes_and_values(rows, K, f32):
    x = torch.randn(rows, K, generator=_gen(rows + K), device="cuda") * torch.exp2(
        torch.randint(-20, 20, (rows, 1), generator=_gen(rows), device="cuda").float())
    x = x if f32 else x.to(torch.bfloat16)
    m = uw.uw_mx_quantize(x)
    code, sb = U.mx_quantize_ref(x.double().cpu().numpy())
    packed, tiles = U.pack_ref(code, sb)
    assert np.array_equal(m.codes.cpu().numpy(), packed)
    assert np.array_equal(m.scales.cpu().numpy().ravel(), tiles)      # bytes past the matrix are 0
    want = torch.from_numpy(U.mx_values_ref(code, sb)).cuda()
    assert torch.equal(uw.uw_mx_dequantize(m).double(), want)
    assert torch.equal(uw.uw_mx_dequantize(m, out_f32=True).double(), want)


@pytest.mark.parametrize("f32", [False, True])
def test_mx_quantize_borders(f32):
    x = torch.from_numpy(_special_rows(128)).float().cuda()
    x = x if f32 else x.to(torch.bfloat16)
    m = uw.uw_mx_quantize(x)
    code, sb = U.mx_quantize_ref(x.double().cpu().numpy())
    packed, tiles = U.pack_ref(code, sb)
    assert np.array_equal(m.codes.cpu().numpy(), packed)
    assert np.array_equal(m.scales.cpu().numpy().ravel(), tiles)
    want = torch.from_numpy(U.mx_values_ref(code, sb)).cuda()
    for got in (uw.uw_mx_dequantize(m).double(), uw.uw_mx_dequantize(m, out_f32=True).double()):
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))
    again = uw.uw_mx_quantize(uw.uw_mx_dequantize(m)[:11])   # what is held comes back as it was
    assert torch.allclose(uw.uw_mx_dequantize(again), uw.uw_mx_dequantize(m)[:11], rtol=0, atol=0, equal_nan=True)


def test_mx_batch_and_strides():
    x = _bf16(3, 70, 192, seed=4)
    m = uw.uw_mx_quantize(x)
    assert m.shape == (3, 70, 192) and m.batch == 3
    each = [uw.uw_mx_quantize(x[i].contiguous()) for i in range(3)]
    assert torch.equal(m.codes, torch.stack([e.codes for e in each]))
    assert torch.equal(m.scales, torch.cat([e.scales for e in each]))
    wide = torch.zeros(70, 200, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:195] = x[0]
    assert torch.equal(uw.uw_mx_quantize(wide[:, 3:195]).codes, each[0].codes)
    turned = x[0].t().contiguous().t()
    assert torch.equal(uw.uw_mx_quantize(turned).codes, each[0].codes)
    empty = uw.uw_mx_quantize(x[0, :0])
    assert empty.shape == (0, 192) and uw.uw_mx_dequantize(empty).shape == (0, 192)


def test_mx_quantize_past_32_bits():
    """2^32 values in a batch: byte offsets of the last matrix pass 32 bits."""
    batch, rows, K = 9, 65536, 8192
    x = torch.zeros(batch, rows, K, dtype=torch.bfloat16, device="cuda")
    tail = _bf16(130, K, seed=9)
    x[-1, -130:] = tail
    m = uw.uw_mx_quantize(x)
    one = uw.uw_mx_quantize(tail)
    assert torch.equal(m.codes[-1, -130:], one.codes)
    back = uw.uw_mx_dequantize(m)
    assert torch.equal(back[-1, -130:], uw.uw_mx_dequantize(one)) and not back[0, 0].any()


# ---------------------------------------------------------------- products of 4-bit weights
@pytest.mark.parametrize("N,K", [(128, 256), (64, 64), (200, 320), (1000, 1024), (264, 2112), (7, 128)])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 100, 128, 129, 256, 300])
@pytest.mark.parametrize("xmx", [False, True])
def test_mx_gemm(N, K, M, xmx):
    X = _bf16(M, K, seed=M)
    W = uw.uw_mx_quantize(_bf16(N, K, seed=N, scale=0.02))
    Xq = uw.uw_mx_quantize(X) if xmx else X
    Xv = (uw.uw_mx_dequantize(Xq, out_f32=True) if xmx else X).double()
    Wv = uw.uw_mx_dequantize(W, out_f32=True).double()
    ref, tol = Xv @ Wv.T, U.product_tolerance(Xv.abs() @ Wv.abs().T, K)
    if not xmx:
        tol = tol + U.split_tolerance(Xv, Wv)
    for f32 in (False, True):
        out = torch.full((M, N), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        y = uw.uw_mx_gemm(Xq, W, out=out, out_f32=f32)
        U.check(y, ref, tol)
        assert torch.equal(y, uw.uw_mx_gemm(Xq, W, out_f32=f32))   # the same bits again


@pytest.mark.parametrize("xmx", [False, True])
@pytest.mark.parametrize("M", [1, 40, 1000])
def test_mx_gemm_full_size(M, xmx):
    N, K = 14336, 4096
    X = _bf16(M, K, seed=M)
    W = uw.uw_mx_quantize(_bf16(N, K, seed=2, scale=0.02))
    Xq = uw.uw_mx_quantize(X) if xmx else X
    Xv = (uw.uw_mx_dequantize(Xq, out_f32=True) if xmx else X).double()
    Wv = uw.uw_mx_dequantize(W, out_f32=True).double()
    tol = U.product_tolerance(Xv.abs() @ Wv.abs().T, K)
    U.check(uw.uw_mx_gemm(Xq, W), Xv @ Wv.T, tol if xmx else tol + U.split_tolerance(Xv, Wv))


@pytest.mark.parametrize("xmx", [False, True])
def test_mx_gemm_scale_extremes(xmx):
    """Scales from 2^-127 to 2^100 by row, a NaN block, and zeros: exact small sums."""
    N, K, M = 160, 128, 20
    code = np.random.default_rng(1).integers(0, 16, (N, K)).astype(np.uint8)
    sb = np.repeat(np.linspace(0, 227, N).astype(np.uint8)[:, None], K // 32, 1)
    packed, tiles = U.pack_ref(code, sb)
    W = uw.MxMatrix(torch.from_numpy(packed).cuda(), torch.from_numpy(tiles).cuda())
    X = torch.randint(-3, 4, (M, K), generator=_gen(3), device="cuda").to(torch.bfloat16)
    Xq = uw.uw_mx_quantize(X) if xmx else X
    Xv = (uw.uw_mx_dequantize(Xq, out_f32=True) if xmx else X).double()
    Wv = torch.from_numpy(U.mx_values_ref(code, sb)).cuda()
    y = uw.uw_mx_gemm(Xq, W, out_f32=True)
    # sums of small integers times one power of two: exact, but for results below the normal range, which may be flushed
    ref = Xv @ Wv.T
    assert torch.equal(torch.where(ref.abs() >= 2.0 ** -126, y.double(), 0.0), torch.where(ref.abs() >= 2.0 ** -126, ref, 0.0))
    assert (y.double() - ref).abs()[ref.abs() < 2.0 ** -126].max() <= 2.0 ** -126
    sb[5, 1] = 255
    W = uw.MxMatrix(*(torch.from_numpy(a).cuda() for a in U.pack_ref(code, sb)))
    y2 = uw.uw_mx_gemm(Xq, W, out_f32=True)
    assert y2[:, 5].isnan().all()
    y2[:, 5] = y[:, 5]
    assert torch.equal(y, y2)


@pytest.mark.parametrize("K", [128, 320, 1024])
def test_mx_gemm_rows_of_wide_range(K):
    """Values from 2^-30 to 2^30 in one block, outlier channels, rows near the ends of the range; NaN and infinity stay in their row."""
    N, M = 130, 24
    X = torch.randn(M, K, generator=_gen(1), device="cuda") * torch.exp2(torch.randint(-30, 31, (M, K), generator=_gen(2), device="cuda").float())
    X[3] = torch.randn(K, generator=_gen(3), device="cuda") * 2.0 ** 100
    X[4] = torch.randn(K, generator=_gen(4), device="cuda") * 2.0 ** -100
    X[5] = 0
    X[6, ::32] = 2.0 ** 110
    X = X.to(torch.bfloat16)
    W = uw.uw_mx_quantize(_bf16(N, K, seed=N, scale=0.02))
    Xv, Wv = X.double(), uw.uw_mx_dequantize(W, out_f32=True).double()
    tol = U.product_tolerance(Xv.abs() @ Wv.abs().T, K) + U.split_tolerance(Xv, Wv) + 1e-38
    y = uw.uw_mx_gemm(X, W, out_f32=True)
    U.check(y, Xv @ Wv.T, tol)
    X[7, 5], X[8, 40], X[9, 70] = math.nan, math.inf, -math.inf
    z = uw.uw_mx_gemm(X, W, out_f32=True)
    for r in range(M):
        if r in (7, 8, 9):
            w = Wv[:, {7: 5, 8: 40, 9: 70}[r]]
            assert not z[r][w != 0].isfinite().any()
        else:
            assert torch.equal(y[r], z[r])


# ---------------------------------------------------------------- router
ROUTES = [(1, 1, 1), (1, 4, 4), (7, 8, 2), (16, 64, 6), (33, 128, 8), (100, 33, 5), (130, 256, 8), (600, 160, 32),
          (1000, 1000, 10), (37, 1024, 3), (5000, 60, 4)]


def _check_route(logits, k, score, renorm, scale=1.0):
    r = uw.uw_route(logits, k, score=score, renorm=renorm, scale=scale)
    ids, w, offsets, rows, pos = U.route_ref(logits.double().cpu().numpy(), k, score, renorm, scale)
    for got, want, name in ((r.ids, ids, "ids"), (r.offsets, offsets, "offsets"), (r.rows, rows, "rows"), (r.pos, pos, "pos")):
        assert np.array_equal(got.cpu().numpy(), want), name
    # exp is off by 2 ulps, its argument (fp32, |x| < 2^8 apart) by 2^-24 |x|; a sum of E terms by (E/32 + 5) 2^-24; a division by 1
    E = logits.shape[1]
    err = np.abs(r.weights.double().cpu().numpy() - w)
    spread = float(torch.nan_to_num(logits.double(), 0, 0, 0).abs().max())
    assert (err <= (2 * spread + 16 + E / 16) * 2.0 ** -24 * np.abs(w) + 1e-44).all(), float(err.max())
    return r


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route(T, E, k, score, renorm):
    x = torch.randn(T, E, generator=_gen(T + E), device="cuda") * 2
    _check_route(x, k, score, renorm, 2.5 if renorm else 1.0)
    _check_route(x.to(torch.bfloat16), k, score, renorm)     # many ties


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masks_and_extremes(score, renorm):
    T, E, k = 200, 48, 6
    x = torch.randn(T, E, generator=_gen(1), device="cuda")
    x[torch.rand(T, E, generator=_gen(2), device="cuda") < 0.5] = -math.inf
    x[::7] = -math.inf                       # nothing to choose
    x[3, :] = -math.inf
    x[3, 11] = 0.5                           # one choice
    x[5, :4] = math.nan
    x[6] = math.nan
    x[8, 9] = math.inf
    x[9, 10:13] = math.inf                   # equal shares
    x[10] = torch.finfo(torch.float32).min
    x[11] = torch.finfo(torch.float32).max
    x[12] = 0.0
    x[12, ::2] = -0.0                        # equal: by index
    x[13] = -200.0                           # sigmoid of all is 0 in fp32
    x[13, 4] = -201.0
    if score == "sigmoid":
        x[13] = -1000.0
    r = uw.uw_route(x, k, score=score, renorm=renorm)
    ids, w, offsets, rows, pos = U.route_ref(x.double().cpu().numpy(), k, score, renorm, 1.0)
    for got, want in ((r.ids, ids), (r.offsets, offsets), (r.rows, rows), (r.pos, pos)):
        assert np.array_equal(got.cpu().numpy(), want)
    got = r.weights.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - w) <= 64 * 2.0 ** -24 * np.abs(w) + 1e-37).all()
    assert r.ids[12].tolist() == list(range(k))


@pytest.mark.parametrize("E,k", [(40, 8), (64, 32), (32, 32), (300, 5)])
def test_route_logits_that_differ_in_their_last_bits(E, k):
    """Neighbours a few units in the last place apart, equal ones among them, also at the border of the choice."""
    bits = torch.randint(0, 40, (257, E), generator=_gen(E), device="cuda").int()
    x = (torch.full((257, E), 1.5, device="cuda").view(torch.int32) + bits).view(torch.float32)
    x[::2] = -x[::2]
    _check_route(x, k, "softmax", True)
    y = torch.randn(257, E, generator=_gen(1), device="cuda")
    order = y.sort(dim=1, descending=True).values
    if k < E:
        edge = order[:, k - 1:k]
        y = torch.where(y == order[:, k:k + 1], (edge.view(torch.int32) - 1).view(torch.float32), y)   # beside the last choice
    _check_route(y, k, "sigmoid", False)


def test_route_empty_and_all_masked():
    r = uw.uw_route(torch.empty(0, 8, device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 9 and r.ids.shape == (0, 2) and r.rows.shape == (0,)
    r = uw.uw_route(torch.full((50, 8), -math.inf, device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 9 and (r.rows == -1).all() and (r.pos == -1).all() and (r.weights == 0).all()


def test_route_same_bits_and_strides():
    x = torch.randn(3000, 128, generator=_gen(5), device="cuda").to(torch.bfloat16)
    a = uw.uw_route(x, 8)
    wide = torch.zeros(3000, 300, dtype=torch.bfloat16, device="cuda")
    wide[:, 7:135] = x
    for b in (uw.uw_route(x, 8), uw.uw_route(wide[:, 7:135], 8)):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


# ---------------------------------------------------------------- grouped products
def _offsets(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def _grouped_case(sizes, N, K, mx, up, gather, seed=0, T=None):
    E, R = len(sizes), int(sum(sizes))
    W = [_bf16(E, N, K, seed=seed + 10 + i, scale=0.05) for i in range(2 if up else 1)]
    if mx:
        W = [uw.uw_mx_quantize(w) for w in W]
        Wv = [uw.uw_mx_dequantize(w, out_f32=True).double() for w in W]
    else:
        Wv = [w.double() for w in W]
    T = (T or max(1, R // 2)) if gather else R
    X = _bf16(T, K, seed=seed)
    rows = torch.randint(0, T, (R,), generator=_gen(seed), device="cuda").int() if gather else None
    off = _offsets(sizes)
    ref, tol = U.grouped_ref(X.double(), Wv[0], off.cpu(), rows, Wv[1] if up else None, mx)
    return X, W, off, rows, ref, tol


GROUPS = [[1], [5, 0, 3], [0, 0, 1, 0], [16, 17, 15], [130, 1, 0, 64, 300], [257, 256, 255], [1] * 40, [3, 700, 2],
          [0] * 30 + [20] + [0] * 33]


@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("N,K", [(128, 64), (200, 320), (72, 1024)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(sizes, N, K, mx, up, gather):
    X, W, off, rows, ref, tol = _grouped_case(sizes, N, K, mx, up, gather)
    for f32 in (False, True):
        out = torch.full((int(off[-1]), N), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        y = uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1] if up else None, out=out, out_f32=f32)
        U.check(y, ref, tol)
        assert torch.equal(y, uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1] if up else None, out_f32=f32))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([40, 8, 90, 3], 1001, 576), ([600, 900, 30], 13, 192), ([2] * 9, 4100, 2048)])
def test_grouped_odd_outputs(sizes, N, K, mx, up):
    """N not a multiple of 8 (element stores), many tiles and cut tiles."""
    X, W, off, rows, ref, tol = _grouped_case(sizes, N, K, mx, up, True)
    U.check(uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1] if up else None), ref, tol)


@pytest.mark.parametrize("mx", [False, True])
def test_grouped_leaves_rows_outside_the_offsets(mx):
    sizes, N, K = [5, 0, 21, 2], 136, 256
    X, W, off, rows, ref, tol = _grouped_case(sizes, N, K, mx, True, True)
    lead, tail, R = 3, 50, 28
    rows = torch.cat([torch.full((lead,), -1), rows.cpu(), torch.full((tail,), -1)]).int().cuda()
    out = torch.full((lead + R + tail, N), 7.0, dtype=torch.bfloat16, device="cuda")
    uw.uw_gemm_grouped(X, W[0], off + lead, rows=rows, up=W[1], out=out)
    U.check(out[lead:lead + R], ref, tol)
    assert (out[:lead] == 7).all() and (out[lead + R:] == 7).all()


def test_grouped_ignores_what_no_slot_reads():
    """NaN in rows of X behind the last slot and in experts without slots reach nothing."""
    sizes, N, K = [9, 0, 30], 130, 192
    X, W, off, _, ref, tol = _grouped_case(sizes, N, K, False, False, False)
    X = torch.cat([X, torch.full((40, K), float("nan"), dtype=torch.bfloat16, device="cuda")])
    W[0][1] = float("nan")
    y = uw.uw_gemm_grouped(X, W[0], off)
    U.check(y[:39], ref, tol)


def test_grouped_bad_offsets_and_rows_are_reported():
    X, W, off, rows, ref, tol = _grouped_case([6, 10, 4], 128, 128, False, False, True)
    bad = rows.clone()
    bad[3], bad[15] = -1, 10 ** 9
    y = uw.uw_gemm_grouped(X, W[0], off, rows=bad)
    assert uw.uw_last_device_status() == 8
    keep = [i for i in range(20) if i not in (3, 15)]
    U.check(y[keep], ref[keep], tol[keep])
    for o in ([0, 6, 16, 2 ** 30], [0, 16, 6, 20], [-5, 6, 16, 20]):
        uw.uw_gemm_grouped(X, W[0], torch.tensor(o, dtype=torch.int32, device="cuda"), rows=rows)
        assert uw.uw_last_device_status() == 8


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("fill", [0x00, 0xFF, "random"])
def test_grouped_workspace_contents_do_not_matter(mx, fill):
    X, W, off, rows, ref, tol = _grouped_case([3, 2, 1], 400, 2048, mx, True, True)
    n = uw.uw_gemm_grouped_workspace(6, W[0], W[1], gathered=True)
    ws = (torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda") if fill == "random"
          else torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
    for _ in range(3):
        U.check(uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1], ws=ws), ref, tol)


# ---------------------------------------------------------------- combination
@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (5, 2, 4096), (33, 8, 1000), (100, 9, 13), (64, 32, 7), (700, 3, 520)])
@pytest.mark.parametrize("in32", [False, True])
@pytest.mark.parametrize("out32", [False, True])
def test_combine(T, k, N, in32, out32):
    Z = torch.randn(T * k, N, generator=_gen(T), device="cuda")
    Z = Z if in32 else Z.to(torch.bfloat16)
    pos = torch.randperm(T * k, generator=_gen(k), device="cuda").int().view(T, k)
    pos[torch.rand(T, k, generator=_gen(3), device="cuda") < 0.2] = -1
    pos[T // 2] = -1
    w = torch.rand(T, k, generator=_gen(4), device="cuda")
    y = uw.uw_combine(Z, pos, w, out_f32=out32)
    p = torch.where(pos >= 0, w, 0.0).double()[..., None] * Z.double()[pos.clamp(min=0).long()]
    # k multiply-adds, each off by half a step of a sum that stays below the sum of magnitudes
    U.check(y, p.sum(1), k * 2.0 ** -24 * p.abs().sum(1))
    assert (y[T // 2] == 0).all()


def test_combine_skips_untouched_rows_and_reports_bad_positions():
    Z = torch.full((4, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    Z[1] = 2.0
    pos = torch.tensor([[1, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.0], [0.0, 0.0]], device="cuda")
    y = uw.uw_combine(Z, pos, w)
    assert (y[0] == 1).all() and (y[1] == 0).all()
    pos[1, 0] = 4
    y = uw.uw_combine(Z, pos, w)
    assert uw.uw_last_device_status() == 8 and (y[0] == 1).all()


# ---------------------------------------------------------------- a whole layer
def _layer(x, router, gate, up, down, k, **kw):
    logits = uw.uw_dense_gemm(x, router, out_f32=True)
    r = uw.uw_route(logits, k, renorm=True, **kw)
    h = uw.uw_gemm_grouped(x, gate, r.offsets, rows=r.rows, up=up)
    z = uw.uw_gemm_grouped(h, down, r.offsets)
    return uw.uw_combine(z, r.pos, r.weights), r


def _layer_case(T, E, N, K, mx, seed=0):
    x = _bf16(T, K, seed=seed)
    router = _bf16(E, K, seed=seed + 1, scale=0.05)
    ws = [_bf16(E, N, K, seed=seed + 2, scale=0.04), _bf16(E, N, K, seed=seed + 3, scale=0.04), _bf16(E, K, N, seed=seed + 4, scale=0.04)]
    return x, router, [uw.uw_mx_quantize(w) for w in ws] if mx else ws


def _layer_ref(x, ws, mx, r):
    v = [uw.uw_mx_dequantize(w, out_f32=True).double() if mx else w.double() for w in ws]
    T, K = x.shape
    y, tol = torch.zeros(T, K, dtype=torch.float64, device="cuda"), torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(r.ids.shape[1]):
            e = int(r.ids[t, j])
            if e < 0:
                continue
            xs = x[t:t + 1].double()
            g, u = xs @ v[0][e].T, xs @ v[1][e].T
            h = U.swiglu_ref(g, u)
            dg, du = (U.product_tolerance(xs.abs() @ w.abs().T, K) + (U.split_tolerance(xs, w) if mx else 0) for w in (v[0][e], v[1][e]))
            dh = U.swiglu_tolerance(g, u, dg, du)
            dh = dh + 2.0 ** -8 * (h.abs() + dh)                          # h is rounded to BF16
            z = h @ v[2][e].T
            dz = dh @ v[2][e].abs().T + U.product_tolerance((h.abs() + dh) @ v[2][e].abs().T, h.shape[1])
            if mx:
                dz = dz + U.split_tolerance(h.abs() + dh, v[2][e])
            dz = dz + 2.0 ** -8 * (z.abs() + dz)                          # so is z
            w = float(r.weights[t, j])
            y[t] += w * z[0]
            tol[t] += w * dz[0] + 2.0 ** -20 * w * (z.abs() + dz)[0]
    return y, tol


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 9, 70])
def test_expert_layer(T, mx):
    x, router, ws = _layer_case(T, 12, 320, 256, mx)
    y, r = _layer(x, router, *ws, 3)
    U.check(y, *_layer_ref(x, ws, mx, r))


@pytest.mark.parametrize("mx", [False, True])
def test_expert_layer_in_a_graph(mx):
    """Captured once, replayed on new inputs (other groups), beside eager calls on another stream."""
    x, router, ws = _layer_case(24, 8, 256, 512, mx)
    _layer(x, router, *ws, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        y, r = _layer(x, router, *ws, 2)
    other = _bf16(24, 512, seed=77)
    for seed in range(4):
        x.copy_(_bf16(24, 512, seed=50 + seed))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            z, rz = _layer(other, router, *ws, 2)
        torch.cuda.synchronize()
        want, rw = _layer(x, router, *ws, 2)
        assert torch.equal(y, want) and torch.equal(r.ids, rw.ids)
        again, _ = _layer(other, router, *ws, 2)
        assert torch.equal(z, again)


def test_calls_on_a_given_stream():
    s = torch.cuda.Stream()
    x, router, ws = _layer_case(16, 8, 256, 512, True)
    torch.cuda.synchronize()
    want, r0 = _layer(x, router, *ws, 2)
    logits = uw.uw_dense_gemm(x, router, out_f32=True)
    torch.cuda.synchronize()
    r = uw.uw_route(logits, 2, renorm=True, stream=s)
    h = uw.uw_gemm_grouped(x, ws[0], r.offsets, rows=r.rows, up=ws[1], stream=s)
    z = uw.uw_gemm_grouped(h, ws[2], r.offsets, stream=s.cuda_stream)
    y = uw.uw_combine(z, r.pos, r.weights, stream=s)
    q = uw.uw_mx_gemm(uw.uw_mx_quantize(x, stream=s), uw.uw_mx_quantize(_bf16(64, 512, seed=3), stream=s), stream=s)
    s.synchronize()
    assert torch.equal(y, want) and q.isfinite().all()


@pytest.mark.parametrize("mx", [False, True])
def test_full_size_experts(mx):
    """Four experts of the benchmark's MLP shape, decoding and a prompt, sampled outputs."""
    E, N, K = 4, 14336, 4096
    for sizes in ([2, 0, 5, 1], [700, 3, 0, 321]):
        X, W, off, rows, ref, tol = _grouped_case(sizes, N, K, mx, True, True, T=64)
        U.check(uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1]), ref, tol)


# ---------------------------------------------------------------- drawn shapes, large ones, calls at once
@pytest.mark.parametrize("seed", range(24))
def test_grouped_drawn(seed):
    rng = np.random.default_rng(seed)
    E = int(2 ** rng.uniform(0, 6.5))
    R = int(2 ** rng.uniform(0, 10.5))
    p = np.arange(1, E + 1) ** -rng.uniform(0, 2)
    sizes = rng.multinomial(R, p / p.sum()).tolist()
    N, K = int(2 ** rng.uniform(0, 9.5)), 64 * int(rng.integers(1, 20))
    mx, up, gather = (bool(v) for v in rng.integers(0, 2, 3))
    X, W, off, rows, ref, tol = _grouped_case(sizes, N, K, mx, up, gather, seed=seed)
    f32 = bool(rng.integers(0, 2))
    U.check(uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1] if up else None, out_f32=f32), ref, tol)


@pytest.mark.parametrize("E", [257, 1024])
@pytest.mark.parametrize("mx", [False, True])
def test_grouped_many_experts(E, mx):
    sizes = [(e * 7919) % 5 if e % 3 else 0 for e in range(E)]
    X, W, off, rows, ref, tol = _grouped_case(sizes, 72, 128, mx, True, True)
    U.check(uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1]), ref, tol)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("R", [200, 2000, 9000])
def test_grouped_rounds_and_cut_tiles(mx, up, R):
    """Every way of sharing out tiles: fewer than workers, whole rounds, a rest cut in parts (long K)."""
    for N, K in ((1000, 4096), (2304, 1024)):
        X, W, off, rows, ref, tol = _grouped_case([R // 2, 0, R - R // 2], N, K, mx, up, False)
        U.check(uw.uw_gemm_grouped(X, W[0], off, up=W[1] if up else None), ref, tol)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([1, 0, 17, 5], 520, 8192), ([1, 0, 17, 5], 520, 8256), ([4] * 8, 2600, 4096),
                                       ([4] * 8, 2600, 4160)])
def test_grouped_small_tiles_cut_in_ranges(mx, up, sizes, N, K):
    """A long K with few tiles, or a few behind a whole round: workers share tiles of few slots; the same bits every time."""
    X, W, off, rows, ref, tol = _grouped_case(sizes, N, K, mx, up, True)
    y = uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1] if up else None)
    U.check(y, ref, tol)
    for _ in range(3):
        assert torch.equal(y, uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1] if up else None))


def test_grouped_outputs_past_32_bits():
    """2.3e9 outputs: the last slots' addresses pass 2^31 elements and 2^32 bytes."""
    R, N, K = 70000, 32768, 64
    X = _bf16(R, K, seed=1)
    W = _bf16(2, N, K, seed=2, scale=0.1)
    off = torch.tensor([0, 100, R], dtype=torch.int32, device="cuda")
    y = uw.uw_gemm_grouped(X, W, off)
    for lo, hi, e in ((0, 100, 0), (100, 300, 1), (R - 130, R, 1)):
        ref = X[lo:hi].double() @ W[e].double().T
        U.check(y[lo:hi], ref, U.product_tolerance(X[lo:hi].double().abs() @ W[e].double().abs().T, K))
    z = uw.uw_combine(y, torch.tensor([[R - 1, 5], [-1, R - 2]], dtype=torch.int32, device="cuda"),
                      torch.tensor([[0.5, 0.25], [9.0, 1.0]], device="cuda"), out_f32=True)
    want = torch.stack([0.5 * y[R - 1].double() + 0.25 * y[5].double(), y[R - 2].double()])
    U.check(z, want, 2.0 ** -22 * (y[R - 1].double().abs() + y[5].double().abs() + y[R - 2].double().abs()).expand(2, N))


@pytest.mark.parametrize("mx", [False, True])
def test_grouped_weights_past_32_bits(mx):
    """17 experts of 14336 x 16384 (4e9 weights): the last ones' addresses pass 2^31 elements and 2^32 bytes."""
    E, N, K = 17, 14336, 16384
    W = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    g = _gen(5)
    for e in range(E):
        W[e] = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16) * 0.01
    off = torch.tensor([0] + [3] * 15 + [5, 8], dtype=torch.int32, device="cuda")
    X = _bf16(8, K, seed=3)
    Wm = uw.uw_mx_quantize(W) if mx else W
    y = uw.uw_gemm_grouped(X, Wm, off)
    for lo, hi, e in ((0, 3, 0), (3, 5, 15), (5, 8, 16)):
        w = (uw.uw_mx_dequantize(uw.uw_mx_quantize(W[e])) if mx else W[e]).double()
        x = X[lo:hi].double()
        tol = U.product_tolerance(x.abs() @ w.abs().T, K) + (U.split_tolerance(x, w) if mx else 0)
        U.check(y[lo:hi], x @ w.T, tol)


def test_calls_at_once_on_two_streams():
    """Small and large tiles, 4-bit and BF16, on two streams at the same time: each as alone."""
    cases = [_grouped_case([3, 0, 20], 300, 512, True, True, True, seed=1), _grouped_case([700, 300, 5], 500, 1024, False, False, True, seed=2),
             _grouped_case([150, 300], 384, 2048, True, False, False, seed=3), _grouped_case([1, 2], 2000, 4096, False, True, False, seed=4)]
    x = _bf16(333, 512, seed=9)
    call = lambda c: uw.uw_gemm_grouped(c[0], c[1][0], c[2], rows=c[3], up=c[1][1] if len(c[1]) > 1 else None)  # noqa: E731
    alone = [call(c) for c in cases]
    route = uw.uw_route(x.float(), 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i in range(12):
        for s in (0, 1):
            with torch.cuda.stream(streams[s]):
                got[s].append((call(cases[(i + 2 * s) % 4]), uw.uw_route(x.float(), 4), uw.uw_mx_dequantize(uw.uw_mx_quantize(x))))
    torch.cuda.synchronize()
    for s in (0, 1):
        for i, (y, r, q) in enumerate(got[s]):
            assert torch.equal(y, alone[(i + 2 * s) % 4])
            assert all(torch.equal(a, b) for a, b in zip(r, route))
            assert torch.equal(q, got[0][0][2])


def test_python_refusals():
    X, W, off, rows, _, _ = _grouped_case([3, 2], 64, 128, False, True, True)
    M = uw.uw_mx_quantize(W[0])
    bad = [lambda: uw.uw_gemm_grouped(X.float(), W[0], off, rows=rows),
           lambda: uw.uw_gemm_grouped(X[:, :64], W[0], off, rows=rows),
           lambda: uw.uw_gemm_grouped(X, W[0], off[:2], rows=rows),
           lambda: uw.uw_gemm_grouped(X, W[0], off.long(), rows=rows),
           lambda: uw.uw_gemm_grouped(X, W[0], off.cpu(), rows=rows),
           lambda: uw.uw_gemm_grouped(X, W[0], off, rows=rows.view(1, -1)),
           lambda: uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=M),
           lambda: uw.uw_gemm_grouped(X, W[0], off, rows=rows, up=W[1][:, :32]),
           lambda: uw.uw_gemm_grouped(X, W[0].transpose(1, 2), off, rows=rows),
           lambda: uw.uw_gemm_grouped(X, W[0], off, rows=rows, out=torch.empty(5, 63, dtype=torch.bfloat16, device="cuda")),
           lambda: uw.uw_gemm_grouped(X, W[0], off, rows=rows, out=torch.empty(5, 64, device="cuda")),
           lambda: uw.uw_mx_gemm(X, uw.uw_mx_quantize(W[0][0, :, :64].contiguous())),
           lambda: uw.uw_mx_quantize(X[0]), lambda: uw.uw_mx_quantize(X.half()),
           lambda: uw.MxMatrix(M.codes, M.scales[:-1]), lambda: uw.MxMatrix(M.codes.float(), M.scales),
           lambda: uw.uw_route(X, 2, score="relu"), lambda: uw.uw_route(X[0], 2), lambda: uw.uw_route(X.half(), 2),
           lambda: uw.uw_combine(X, off, off), lambda: uw.uw_combine(X, rows.view(-1, 1), rows.view(-1, 1)),
           lambda: uw.uw_combine(X[0], rows.view(-1, 1), rows.view(-1, 1).float())]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for f, status in ((lambda: uw.uw_gemm_grouped(X, W[0], off, rows=rows, ws=small), 5), (lambda: uw.uw_mx_gemm(X, uw.uw_mx_quantize(W[0][0]), ws=small), 5),
                      (lambda: uw.uw_route(X, 40), 2), (lambda: uw.uw_route(X, 0), 1), (lambda: uw.uw_mx_quantize(_bf16(4, 96)), 2),
                      (lambda: uw.uw_mx_gemm(X, M), 2)):
        with pytest.raises(uw.UnweightError) as ei:
            f()
        assert ei.value.status == status
