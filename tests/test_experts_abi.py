"""The microscaled 4-bit form and the expert layer without a GPU: sizes, the
layout's formula, refusals (nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import decode_gemm_bf16_b200 as uw
from decode_gemm_bf16_b200 import build as uwbuild
from tests import expert_util as U

A = 0x10000   # an aligned address that is never read


@pytest.fixture(scope="module")
def L():
    uwbuild.build()
    return uw.lib()


def test_mx_sizes(L):
    assert uw.uw_mx_bytes(1, 128, 256) == (128 * 128, 1024)
    assert uw.uw_mx_bytes(3, 129, 320) == (3 * 129 * 160, 3 * 2 * 2 * 1024)
    assert uw.uw_mx_bytes(0, 5, 64)[0] == 0
    for bad, status in (((1, 4, 96), 2), ((1, 4, 0), 2), ((1, 4, 32), 2), ((-1, 4, 64), 1), ((1, -4, 64), 1),
                        ((1, 1 << 26, 64), 2), ((1 << 31, 1 << 20, 64), 2)):
        with pytest.raises(uw.UnweightError) as ei:
            uw.uw_mx_bytes(*bad)
        assert ei.value.status == status, bad


def test_scale_tiles_hold_every_byte_once():
    for rows, K in ((1, 64), (130, 320), (256, 512)):
        at, size = U.scale_at(rows, K)
        assert len(np.unique(at)) == at.size and at.min() >= 0 and at.max() < size


def test_plain_quantiser_against_its_definition():
    x = np.random.default_rng(0).standard_normal((8, 64)).astype(np.float32).astype(np.float64)
    code, sb = U.mx_quantize_ref(x)
    v = U.mx_values_ref(code, sb)
    s = np.ldexp(1.0, sb.astype(int) - 127).repeat(32, 1)
    a = np.abs(x).reshape(8, 2, 32).max(-1).repeat(32, 1)
    assert ((a / s >= 4) & (a / s < 8)).all()
    inside = np.abs(x) / s <= 6
    assert (np.abs(v - x)[inside] <= s[inside]).all() and (np.abs(v / s)[~inside] == 6).all()


def _mx(batch=1, rows=128, K=256, codes=A, scales=A):
    return uw.MxDesc(codes, scales, batch, rows, K)


def test_mx_refusals(L):
    q = L.uw_mx_quantize
    assert q(None, 0, 1, 4, 64, A, A, None) == 1 and q(A, 0, 1, 4, 64, None, A, None) == 1
    assert q(A + 2, 0, 1, 4, 64, A, A, None) == 1 and q(A, 0, 1, 4, 64, A, A + 8, None) == 1
    assert q(A, 0, 1, 4, 64, A + 16, A, None) == 1
    assert q(A, 0, 1, 4, 100, A, A, None) == 2
    assert q(None, 0, 1, 0, 64, None, None, None) == 0 and q(None, 0, 0, 4, 64, None, None, None) == 0
    d = L.uw_mx_dequantize
    assert d(None, A, 0, None) == 1 and d(ctypes.byref(_mx(codes=0)), A, 0, None) == 1
    assert d(ctypes.byref(_mx()), None, 0, None) == 1 and d(ctypes.byref(_mx(K=96)), A, 0, None) == 2
    assert d(ctypes.byref(_mx(rows=0, codes=0, scales=0)), None, 0, None) == 0


def test_mx_gemm_refusals(L):
    r, g = ctypes.byref, L.uw_mx_gemm
    big = 1 << 30
    n = ctypes.c_size_t()
    assert L.uw_mx_gemm_workspace(4, 128, 256, 0, r(n)) == 0 and n.value > 0
    assert L.uw_mx_gemm_workspace(0, 128, 256, 0, r(n)) == 0 and n.value == 0
    assert L.uw_mx_gemm_workspace(4, 128, 96, 0, r(n)) == 2 and L.uw_mx_gemm_workspace(-1, 128, 256, 0, r(n)) == 1
    assert L.uw_mx_gemm_workspace(4, 128, 256, 0, None) == 1
    assert g(A, None, 4, None, A, 0, A, big, None) == 1
    assert g(None, None, 4, r(_mx()), A, 0, A, big, None) == 1                    # neither X
    assert g(A, r(_mx(rows=4)), 4, r(_mx()), A, 0, A, big, None) == 1             # both
    assert g(A + 2, None, 4, r(_mx()), A, 0, A, big, None) == 1
    assert g(A, None, 4, r(_mx()), A + 4, 0, A, big, None) == 1
    assert g(A, None, -1, r(_mx()), A, 0, A, big, None) == 1
    assert g(A, None, 4, r(_mx(batch=2)), A, 0, A, big, None) == 2
    assert g(None, r(_mx(rows=5)), 4, r(_mx()), A, 0, A, big, None) == 2          # rows of X
    assert g(None, r(_mx(rows=4, K=512)), 4, r(_mx()), A, 0, A, big, None) == 2   # K of X
    assert g(A, None, 4, r(_mx()), A, 0, None, 0, None) == 5
    assert g(A, None, 4, r(_mx()), A, 0, A + 16, big, None) == 5
    assert g(A, None, 4, r(_mx()), A, 0, A, 64, None) == 5
    assert g(None, None, 0, r(_mx()), None, 0, None, 0, None) == 0


def test_route_refusals(L):
    n = ctypes.c_size_t()
    for T, E, k, want in ((-1, 8, 2, 1), (4, 0, 1, 1), (4, 8, 0, 1), (4, 8, 9, 2), (4, 1025, 2, 2), (4, 64, 33, 2), (1 << 30, 8, 2, 2)):
        assert L.uw_route_workspace(T, E, k, ctypes.byref(n)) == want, (T, E, k)
        assert L.uw_route(A, 1, T, E, k, 0, 0, 1.0, A, A, A, A, A, A, 1 << 30, None) == want
    assert L.uw_route_workspace(1000, 8, 2, ctypes.byref(n)) == 0 and n.value > 0
    args = [A, 1, 1000, 8, 2, 0, 0, 1.0, A, A, A, A, A, A, 1 << 30, None]
    for i, v, want in ((0, None, 1), (0, A + 2, 1), (5, 2, 1), (8, None, 1), (9, None, 1), (10, None, 1), (11, None, 1),
                       (12, None, 1), (12, A + 2, 1), (13, None, 5), (13, A + 128, 5), (14, 16, 5)):
        a = list(args)
        a[i] = v
        assert L.uw_route(*a) == want, (i, v)


def _group(**kw):
    a = uw.GroupArgs()
    d = dict(X=A, x_rows=16, rows=None, slots=16, offsets=A, E=4, N=128, K=256, W=A, up=None, Y=A, workspace=A,
             workspace_bytes=1 << 30)
    d.update(kw)
    for k, v in d.items():
        setattr(a, k, ctypes.pointer(v) if isinstance(v, uw.MxDesc) else v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(slots=-1), 1), (dict(E=0), 1), (dict(E=1025), 2), (dict(N=0), 2), (dict(K=96), 2), (dict(K=0), 2),
    (dict(E=1024, N=1 << 22), 2), (dict(slots=0x7FFFFFFF), 2), (dict(X=None), 1), (dict(X=A + 2), 1), (dict(W=None), 1),
    (dict(W=A + 8), 1), (dict(up=A + 8), 1), (dict(Y=None), 1), (dict(Y=A + 4), 1), (dict(offsets=None), 1),
    (dict(offsets=A + 2), 1), (dict(rows=A + 2), 1), (dict(x_rows=15), 1), (dict(x_rows=0, rows=A), 1),
    (dict(workspace=None), 5), (dict(workspace=A + 64), 5), (dict(workspace_bytes=1000), 5),
    (dict(W_mx=_mx(batch=4)), 1), (dict(W=None, W_mx=_mx(batch=3)), 2), (dict(W=None, W_mx=_mx(batch=4, rows=64)), 2),
    (dict(W=None, W_mx=_mx(batch=4, K=512)), 2), (dict(W=None, W_mx=_mx(batch=4, codes=0)), 1),
    (dict(W=None, up_mx=_mx(batch=4)), 1), (dict(W=None, W_mx=_mx(batch=4), up_mx=_mx(batch=5)), 2)])
def test_grouped_refusals(L, kw, want):
    assert L.uw_gemm_grouped(ctypes.byref(_group(**kw)), None) == want


def test_grouped_no_slots_and_workspace(L):
    n = ctypes.c_size_t()
    assert L.uw_gemm_grouped(None, None) == 1
    assert L.uw_gemm_grouped(ctypes.byref(_group(slots=0, X=None, Y=None, offsets=None, workspace=None)), None) == 0
    assert L.uw_gemm_grouped_workspace(ctypes.byref(_group(slots=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert L.uw_gemm_grouped_workspace(ctypes.byref(_group()), ctypes.byref(n)) == 0 and n.value > 0
    assert L.uw_gemm_grouped_workspace(ctypes.byref(_group(K=32)), ctypes.byref(n)) == 2
    assert L.uw_gemm_grouped_workspace(ctypes.byref(_group()), None) == 1


def test_combine_refusals(L):
    args = [A, 0, 8, A, A, 4, 2, 64, A, 0, None]
    for i, v, want in ((0, None, 1), (0, A + 2, 1), (2, -1, 1), (3, None, 1), (4, None, 1), (5, -1, 1), (6, 0, 1), (6, 33, 2),
                       (7, -1, 1), (8, None, 1), (8, A + 8, 1), (5, 1 << 31, 2)):
        a = list(args)
        a[i] = v
        assert L.uw_combine(*a) == want, (i, v)
    args[5] = 0
    assert L.uw_combine(*args) == 0


def test_python_refusals_without_a_device():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: uw.uw_mx_quantize(x), lambda: uw.uw_route(x, 2), lambda: uw.uw_combine(x, x, x),
                 lambda: uw.uw_gemm_grouped(x, x, x), lambda: uw.MxMatrix(x, x), lambda: uw.uw_route(x, 2, score="other"),
                 lambda: uw.uw_mx_quantize(None)):
        with pytest.raises(ValueError):
            call()
