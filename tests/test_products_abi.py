"""Host-side checks of the fp8 and grouped products (no GPU needed): every refusal the
header documents, before anything is enqueued, and the oracle functions the GPU tests
compare with, pinned by hand."""
import numpy as np
import pytest
import torch

import input_adaptive_reduced_colnorm_b200 as rmm
import oracle
from input_adaptive_reduced_colnorm_b200 import build as rmm_build

OK, INVALID, UNSUPPORTED = range(3)
P16 = 0x10000  # aligned fake device addresses (never dereferenced)
P_MIS = 0x10002


@pytest.fixture(scope="module")
def L():
    rmm_build.build()
    return rmm.lib()


def test_quantize_refusals(L):
    def q(X=P16, n=4, d=256, ldx=256, Xq=P16, ldq=256, sx=P16, lds=4):
        return L.rmm_quantize_fp8(X, n, d, ldx, Xq, ldq, sx, lds, None)
    assert q(n=-1) == INVALID
    assert q(d=0) == INVALID
    assert q(X=None) == INVALID
    assert q(Xq=None) == INVALID
    assert q(sx=None) == INVALID
    assert q(ldx=248) == INVALID       # ldx < d
    assert q(ldq=240) == INVALID
    assert q(lds=3) == INVALID         # lds < n
    assert q(X=P_MIS) == UNSUPPORTED
    assert q(sx=P16 + 1) == UNSUPPORTED
    assert q(ldx=260) == UNSUPPORTED   # not a multiple of 8
    assert q(ldq=264) == UNSUPPORTED   # not a multiple of 16
    assert q(d=(1 << 24) + 1, ldx=1 << 25, ldq=1 << 25) == UNSUPPORTED
    assert q(n=0, X=None, Xq=None, sx=None) == OK


def test_quantize_weight_refusals(L):
    def q(W=P16, g=2, ws=256 * 512, d=256, m=512, ldw=512, Wq=P16, qs=256 * 512, ldq=512, sw=P16):
        return L.rmm_quantize_fp8_weight(W, g, ws, d, m, ldw, Wq, qs, ldq, sw, None)
    assert q(g=0) == INVALID
    assert q(d=0) == INVALID
    assert q(m=0) == INVALID
    assert q(W=None) == INVALID
    assert q(sw=None) == INVALID
    assert q(ldw=504) == INVALID
    assert q(ldq=496) == INVALID
    assert q(ws=255 * 512) == INVALID          # matrices overlap
    assert q(qs=255 * 512) == INVALID
    assert q(ldw=516, ws=1 << 20) == UNSUPPORTED
    assert q(ldq=520, qs=1 << 20) == UNSUPPORTED
    assert q(ws=(1 << 20) + 4) == UNSUPPORTED
    assert q(Wq=P_MIS) == UNSUPPORTED
    assert q(g=1 << 30, ws=256 * 512, qs=256 * 512) == UNSUPPORTED  # too many blocks


def test_linear_fp8_refusals(L):
    def f(X=P16, n=8, d=256, ldx=256, sx=P16, lds=8, W=P16, m=512, ldw=512, sw=P16, Y=P16, ldy=512):
        return L.rmm_linear_fp8(X, n, d, ldx, sx, lds, W, m, ldw, sw, Y, ldy, None)
    assert f(n=-1) == INVALID
    assert f(d=0) == INVALID
    assert f(m=0) == INVALID
    assert f(X=None) == INVALID
    assert f(W=None) == INVALID
    assert f(Y=None) == INVALID
    assert f(sx=None) == INVALID
    assert f(sw=None) == INVALID
    assert f(ldx=240) == INVALID
    assert f(ldw=496) == INVALID
    assert f(ldy=504) == INVALID
    assert f(lds=7) == INVALID
    assert f(X=P_MIS) == UNSUPPORTED
    assert f(ldx=264) == UNSUPPORTED
    assert f(ldw=520) == UNSUPPORTED
    assert f(ldy=516) == UNSUPPORTED
    assert f(sw=P_MIS) == UNSUPPORTED
    assert f(m=(1 << 31) - 1, ldw=1 << 31, ldy=1 << 31) == UNSUPPORTED
    assert f(n=0, X=None, Y=None, sx=None) == OK


def test_grouped_refusals(L):
    def g(X=P16, n=8, d=256, ldx=256, W=P16, groups=4, ws=256 * 512, m=512, ldw=512, off=P16, Y=P16, ldy=512):
        return L.rmm_grouped_linear(X, n, d, ldx, W, groups, ws, m, ldw, off, Y, ldy, None)
    assert g(groups=0) == INVALID
    assert g(off=None) == INVALID
    assert g(X=None) == INVALID
    assert g(ws=256 * 504) == INVALID     # the groups' weights overlap
    assert g(ldx=248) == INVALID
    assert g(groups=1025) == UNSUPPORTED
    assert g(ws=256 * 512 + 4) == UNSUPPORTED
    assert g(ldx=260) == UNSUPPORTED
    assert g(off=P_MIS) == UNSUPPORTED
    assert g(Y=P_MIS) == UNSUPPORTED
    assert g(n=0, X=None, Y=None) == OK

    def h(X=P16, n=8, d=256, ldx=256, sx=P16, lds=8, W=P16, groups=4, ws=256 * 512, m=512, ldw=512, sw=P16, off=P16,
          Y=P16, ldy=512):
        return L.rmm_grouped_linear_fp8(X, n, d, ldx, sx, lds, W, groups, ws, m, ldw, sw, off, Y, ldy, None)
    assert h(off=None) == INVALID
    assert h(lds=7) == INVALID
    assert h(sw=None) == INVALID
    assert h(groups=2000) == UNSUPPORTED
    assert h(ldw=520, ws=1 << 20) == UNSUPPORTED  # e4m3 rows in steps of 16 bytes
    assert h(ws=256 * 512 + 8) == UNSUPPORTED
    assert h(n=0, X=None, Y=None, sx=None) == OK


def test_binding_refuses_cpu_tensors():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    X, W = torch.zeros((4, 16), dtype=bf), torch.zeros((2, 16, 8), dtype=bf)
    Xq, Wq = X.to(f8), W.to(f8)
    sx, sw, off = torch.ones((1, 4)), torch.ones((2, 1, 1)), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: rmm.quantize_fp8(X), lambda: rmm.quantize_fp8_weight(W),
                 lambda: rmm.linear_fp8(Xq, sx, Wq[0], sw[0]), lambda: rmm.grouped_linear(X, W, off),
                 lambda: rmm.grouped_linear_fp8(Xq, sx, Wq, sw, off)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_oracle_e4m3_rounding():
    """Against torch's conversion on every bf16 value up to 448, and by hand at ties."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits.float()) & (bits.float().abs() <= 448)].float()
    assert np.array_equal(oracle.e4m3_round(x.numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    got = oracle.e4m3_round([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 464.0, 1e9, -460.0])
    assert got.tolist() == [16.0, 20.0, 0.0, 2.0 ** -8, 448.0, 448.0, -448.0]


def test_oracle_quantize_by_hand():
    X = np.zeros((2, 130))
    X[0, 3], X[0, 4], X[0, 129] = 896.0, -34.0, 3.0
    q, s = oracle.quantize_fp8(X)
    assert s.tolist() == [[2.0, 1.0], [np.float32(3.0) / np.float32(448.0), 1.0]]
    assert q[0, 3] == 448.0 and q[0, 4] == -16.0 and q[0, 129] == 448.0 and not q[1].any()
    qw, sw = oracle.quantize_fp8_weight(X.T)
    assert sw.tolist() == [[2.0], [np.float32(3.0) / np.float32(448.0)]]
    assert np.array_equal(qw[:, 0], q[0])
    assert np.array_equal(oracle.fp8_widen(q, s)[0, [3, 4]], [896.0, -32.0])


def test_oracle_grouped_by_hand():
    X = np.arange(8.0).reshape(4, 2)
    W = [np.eye(2), 2 * np.eye(2), 3 * np.eye(2)]
    Y = oracle.grouped_product(X, W, [1, 1, 3, 2], np.full((4, 2), 9.0))
    assert Y.tolist() == [[9, 9], [4, 6], [8, 10], [9, 9]]  # group 0 empty, group 2's end clamped to its start


def test_contraction_limit(L):
    """A contraction past 2^24 would keep a tile's epilogue waiting for most of the limit of its waits."""
    d = 1 << 24
    f = lambda d: L.rmm_linear_fp8(P16, 0, d, 1 << 25, P16, 1, P16, 16, 16, P16, P16, 16, None)  # noqa: E731
    g = lambda d: L.rmm_grouped_linear(P16, 0, d, 1 << 25, P16, 2, 1 << 30, 16, 16, P16, P16, 16, None)  # noqa: E731
    assert f(d) == OK and g(d) == OK
    assert f(d + 1) == UNSUPPORTED and g(d + 1) == UNSUPPORTED


def test_in_place_is_refused(L):
    """An output that is an input: refused before anything is enqueued."""
    P2 = 0x20000
    assert L.rmm_quantize_fp8(P16, 4, 256, 256, P16, 512, P2, 4, None) == INVALID
    assert b"Xq must not be X" in L.rmm_last_error()
    assert L.rmm_quantize_fp8_weight(P16, 1, 0, 256, 256, 256, P16, 0, 512, P2, None) == INVALID
    assert b"Wq must not be W" in L.rmm_last_error()
    for X, W, Y in ((P16, P2, P16), (P2, P16, P16)):
        assert L.rmm_linear_fp8(X, 8, 256, 256, P2, 8, W, 512, 512, P2, Y, 512, None) == INVALID
        assert b"Y must not be X or W" in L.rmm_last_error()
        assert L.rmm_grouped_linear(X, 8, 256, 256, W, 2, 1 << 20, 512, 512, P2, Y, 512, None) == INVALID
        assert b"Y must not be X or W" in L.rmm_last_error()
