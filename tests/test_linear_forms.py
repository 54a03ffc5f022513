"""GPU: which calls of the fused and grouped linears multiply exactly and which round the weights to fp16
(and so report a range), and what infinities become in either form, as include/awq.h states it."""
import math

import pytest
import torch

import fused_reference as R

pytestmark = pytest.mark.gpu

LIVE = 64           # columns of X that are not zero: y = LIVE 2^-14 15 60000 = 3515.625


def _big(N, K, G, lead=()):
    """Codes 15, zero points 0, scales 60000: every weight is beyond fp16."""
    q, s, z = R.packed(1, 1, K, G, True)
    wide = [t.expand(*lead, N, t.shape[-1]) for t in (torch.full_like(q, -1), torch.full_like(s, 60000.0), torch.zeros_like(z))]
    return tuple(t.contiguous() for t in wide)


def _rows(M, K):
    X = torch.zeros(M, K, dtype=torch.float16, device="cuda")
    X[:, :LIVE] = 2.0 ** -14
    return X


def _expect(lib, y, exact):
    torch.cuda.synchronize()
    if exact:
        lib.device_error()
        want = LIVE * 2.0 ** -14 * 15 * 60000
        assert ((y.double() - want).abs() <= R.HALF * want * 1.01).all()
    else:
        with pytest.raises(lib.AWQError) as e:
            lib.device_error()
        assert e.value.status == lib.AWQ_ERR_RANGE


@pytest.mark.parametrize("M,N,K,G,exact", [
    (1, 64, 128, 128, True), (8, 64, 4096, 32, True), (4, 64, 12288, 32, True), (2, 64, 28672, 32, True),
    (1, 64, 59392, 32, True), (8, 64, 12288, 32, True), (16, 64, 2048, 32, True), (9, 40, 2048, 256, True),
    (8, 32832, 4224, 128, True),
    # K no multiple of 128, whatever the rows; too many rows; N K beyond 2^27; rows beyond shared memory
    (1, 64, 160, 32, False), (1, 64, 2880, 64, False), (8, 64, 96, 32, False), (17, 64, 128, 128, False),
    (9, 32832, 4224, 128, False), (1, 64, 131072, 128, False),
])
def test_range_of_the_fused_linear(lib, M, N, K, G, exact):
    y = lib.linear_fused(_rows(M, K), *_big(N, K, G), G, True)
    _expect(lib, y, exact)


@pytest.mark.parametrize("E,per,N,K,G,exact", [
    (4, 8, 64, 1024, 128, True), (4, 1, 64, 256, 32, True), (1, 8, 64, 4096, 32, True),
    (4, 9, 64, 1024, 128, False), (4, 1, 64, 96, 32, False), (64, 3, 2048, 512, 32, False),
])
def test_range_of_the_grouped_linear(lib, E, per, N, K, G, exact):
    offsets = torch.arange(0, E * per + 1, per, dtype=torch.int32, device="cuda")
    y = lib.linear_grouped(_rows(E * per, K), *_big(N, K, G, (E,)), offsets, None, G, True)
    _expect(lib, y, exact)


@pytest.mark.parametrize("M,K,exact", [(1, 512, True), (3, 512, True), (16, 512, True), (3, 480, False), (20, 512, False),
                                       (150, 4096, False), (40, 14336, False)])
@pytest.mark.parametrize("zp", [True, False])
def test_infinities_of_a_row(lib, M, K, exact, zp):
    """One infinity, two of opposite signs and a NaN, in three rows."""
    N, G = 300, 32
    w = R.packed(30, N, K, G, zp)
    X = R.activations(31, M, K)
    clean = lib.linear_fused(X, *w, G, zp)
    bad = sorted({0, M // 2, M - 1})
    X2 = X.clone()
    X2[bad[0], 7] = math.inf
    if M > 1:
        X2[bad[1], 7], X2[bad[1], K - 1] = -math.inf, math.inf
        X2[bad[-1], 40] = math.nan
    y = lib.linear_fused(X2, *w, G, zp)
    torch.cuda.synchronize()
    lib.device_error()
    keep = [m for m in range(M) if m not in bad]
    assert torch.equal(y[keep], clean[keep])
    W = R.dequantised(w, G)
    for m in bad:
        want = (W * X2[m].double()).sum(1).half()
        assert not torch.isfinite(want).any()
        if exact:
            assert torch.isnan(y[m]).all()
        else:
            assert torch.equal(y[m].nan_to_num(nan=1.0), want.nan_to_num(nan=1.0))
