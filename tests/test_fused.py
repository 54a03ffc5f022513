"""GPU: the fused linear, the expert-grouped linear, routing and combination against plain fp64
implementations (tests/fused_reference.py derives the bounds)."""
import math
import os
import subprocess
import sys

import pytest
import torch

import fused_reference as R

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _finish(lib):
    torch.cuda.synchronize()
    lib.device_error()


# (M, N, K, G, zero_point, activation, gated, bias, residual)
LINEAR = [
    (1, 256, 128, 128, True, None, False, False, False),
    (1, 4096, 4096, 128, True, None, False, False, True),
    (1, 28672, 1024, 128, True, "silu", True, False, False),
    (2, 1, 32, 32, True, None, False, True, True),
    (2, 2, 96, 32, False, "silu", True, True, True),
    (3, 37, 96, 32, True, "relu", False, True, False),
    (4, 130, 2048 + 256, 256, False, "gelu", False, False, True),
    (5, 74, 1024, 64, True, "gelu_tanh", True, True, False),
    (7, 515, 14336, 128, True, None, False, True, True),
    (8, 1022, 4096, 32, True, "silu", True, False, True),
    (8, 96, 14336, 256, True, None, False, False, False),
    (9, 257, 160, 32, True, "silu", False, True, True),
    (9, 260, 4096, 128, True, "silu", True, False, True),
    (15, 1030, 2048, 64, False, None, False, True, True),
    (16, 512, 8192, 256, True, "relu", True, True, False),
    (16, 4096, 4096, 128, True, None, False, False, True),
    (17, 700, 1024, 64, False, "gelu", True, True, True),
    (31, 384, 4096, 256, True, "relu", True, False, False),
    (33, 129, 448, 64, True, None, False, True, False),
    (64, 4096, 14336, 64, False, None, False, True, True),
    (65, 258, 1024, 32, True, "gelu_tanh", True, False, True),
    (128, 640, 512, 128, True, "silu", False, False, True),
    (129, 510, 8192, 128, True, None, False, True, False),
    (192, 256, 320, 64, True, "silu", True, True, True),
    (193, 1000, 1024, 128, True, "gelu", False, True, True),
    (500, 333, 2048, 128, False, None, False, False, False),
    (2048, 1026, 512, 128, True, "silu", True, False, True),
    # a product of two halves without an activation; rows too long for shared memory
    (4, 66, 256, 128, True, None, True, True, True),
    (40, 130, 256, 64, False, None, True, False, False),
    (1, 40, 131072, 128, True, None, False, False, True),
    (3, 40, 262144, 256, True, None, False, True, False),
]


def _case(c, seed):
    M, N, K, G, zp, act, gated, bias, residual = c
    w = R.packed(seed, N, K, G, zp)
    X = R.activations(seed + 1, M, K)
    n = N // 2 if gated else N
    g = torch.Generator().manual_seed(seed + 2)
    b = torch.randn(N, generator=g).half().cuda() if bias else None
    r = torch.randn(M, n, generator=g).half().cuda() if residual else None
    return w, X, b, r


@pytest.mark.parametrize("c", LINEAR, ids=lambda c: "-".join(map(str, c)))
def test_linear_fused(lib, c):
    M, N, K, G, zp, act, gated, _, _ = c
    w, X, b, r = _case(c, 10)
    y = lib.linear_fused(X, *w, G, zp, bias=b, activation=act, gated=gated, residual=r)
    _finish(lib)
    ref, bound = R.linear64(X, w, G, b, act, gated, r)
    R.assert_close(y, ref, bound, gated)


@pytest.mark.parametrize("M", [1, 6, 11, 70, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_fused_strided_rows_and_guard_bands(lib, M, gated):
    """Rows of larger tensors: only the result's elements are written; the residual may be the
    result itself."""
    N, K, G = 202, 384, 128
    n = N // 2 if gated else N
    w = R.packed(20, N, K, G, True)
    X = R.activations(21, M, K)
    wide = torch.full((M, K + 40), NAN, dtype=torch.float16, device="cuda")
    wide[:, 8:8 + K] = X
    buf = torch.full((M + 2, n + 7), NAN, dtype=torch.float16, device="cuda")
    y = buf[1:M + 1, 3:3 + n]
    res = R.activations(22, M, n)
    y.copy_(res)
    out = lib.linear_fused(wide[:, 8:8 + K], *w, G, True, activation="silu", gated=gated, residual=y, out=y)
    _finish(lib)
    assert out is y
    ref, bound = R.linear64(X, w, G, None, "silu", gated, res)
    R.assert_close(y, ref, bound, gated)
    buf[1:M + 1, 3:3 + n] = NAN
    assert torch.isnan(buf).all()


@pytest.mark.parametrize("M", [3, 12, 150])
def test_linear_fused_rows_do_not_mix(lib, M):
    """NaN and infinities of one row stay in it; -inf, +inf and NaN come out as the formula says."""
    N, K, G = 300, 512, 64
    w = R.packed(30, N, K, G, True)
    X = R.activations(31, M, K)
    clean = lib.linear_fused(X, *w, G, True).clone()
    X2 = X.clone()
    X2[1, 5] = NAN
    X2[M - 1, 7] = float("inf")
    y = lib.linear_fused(X2, *w, G, True)
    _finish(lib)
    keep = [m for m in range(M) if m not in (1, M - 1)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[1]).all()
    assert not torch.isfinite(y[M - 1]).any()


def test_linear_fused_overflow_to_inf(lib):
    """An output beyond fp16 rounds to infinity."""
    N, K, G = 64, 128, 128
    q, s, z = R.packed(40, N, K, G, True)
    X = torch.full((16, K), 60000.0, dtype=torch.float16, device="cuda")
    y = lib.linear_fused(X, torch.full_like(q, -1), torch.full_like(s, 2.0), torch.zeros_like(z), G, True)
    _finish(lib)
    assert torch.isinf(y).all() and (y > 0).all()


def test_linear_fused_range_flag(lib):
    """More than 16 rows: weights beyond fp16 are flagged, as in linear_gemm.  Few rows: they multiply
    in fp32 exactly, without a limit (K a multiple of 128)."""
    N, K, G = 64, 128, 128
    q, s, z = R.packed(40, N, K, G, True)
    big = (torch.full_like(q, -1), torch.full_like(s, 60000.0), torch.zeros_like(z))
    lib.linear_fused(torch.full((17, K), 2.0 ** -10, dtype=torch.float16, device="cuda"), *big, G, True)
    with pytest.raises(lib.AWQError) as e:
        lib.device_error()
    assert e.value.status == lib.AWQ_ERR_RANGE
    lib.device_error()
    y = lib.linear_fused(torch.full((8, K), 2.0 ** -14, dtype=torch.float16, device="cuda"), *big, G, True)
    _finish(lib)
    want = 2.0 ** -14 * 15 * 60000 * K          # 7031.25
    assert ((y.double() - want).abs() <= R.HALF * want * 1.01).all()


def test_linear_fused_agrees_with_linear_gemm(lib):
    """Without an epilogue it is the linear of the other entry points (fp32 sums in another order)."""
    w = R.packed(45, 512, 1024, 128, True)
    for M in (1, 8, 40, 300):
        X = R.activations(46, M, 1024)
        a, b = lib.linear_fused(X, *w, 128, True), lib.linear_gemm(X, *w, 128, True)
        _finish(lib)
        ref, bound = R.linear64(X, w, 128)
        R.assert_close(a, ref, bound)
        assert ((a.double() - b.double()).abs() <= 2 * bound).all()


def test_empty_calls(lib):
    w = R.packed(50, 64, 128, 64, True)
    X = torch.empty(0, 128, dtype=torch.float16, device="cuda")
    assert lib.linear_fused(X, *w, 64, True).shape == (0, 64)
    we = R.packed(51, 64, 128, 64, True, lead=(4,))
    r = lib.moe_route(torch.empty(0, 4, device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 5 and r.rows.shape == (0,)
    y = lib.linear_grouped(X, *we, r.offsets, r.rows, 64, True)
    assert y.shape == (0, 64)
    assert lib.moe_combine(y, r.weights, r.positions).shape == (0, 64)
    some = lib.moe_combine(y, torch.zeros(3, 2, device="cuda"), torch.full((3, 2), -1, dtype=torch.int32, device="cuda"))
    _finish(lib)
    assert not some.any()


# ---------------------------------------------------------------------------
# grouped
# ---------------------------------------------------------------------------

def _grouped(seed, counts, N, K, G, zp, act, gated, bias, gather, T=None, gap=0):
    """Inputs of a grouped call with the given rows per expert, `gap` rows before the first expert's
    and behind the last's."""
    E, n_rows = len(counts), sum(counts) + 2 * gap
    w = R.packed(seed, N, K, G, zp, lead=(E,))
    g = torch.Generator().manual_seed(seed + 3)
    b = torch.randn(E, N, generator=g).half().cuda() if bias else None
    T = T or max(1, n_rows // 2)
    rows = torch.randint(0, T, (n_rows,), generator=g, dtype=torch.int32).cuda() if gather else None
    X = R.activations(seed + 4, T if gather else n_rows, K)
    offsets = torch.tensor([gap + sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32, device="cuda")
    return w, X, b, rows, offsets, n_rows


def _check_grouped(y, X, w, G, b, rows, offsets, act, gated, rms=True):
    o = offsets.tolist()
    for e in range(len(o) - 1):
        a, z = o[e], o[e + 1]
        if a == z:
            continue
        x = X[rows[a:z].long()] if rows is not None else X[a:z]
        we = tuple(None if t is None else t[e] for t in w)
        ref, bound = R.linear64(x, we, G, None if b is None else b[e], act, gated)
        R.assert_close(y[a:z], ref, bound, gated, rms=rms and (z - a) * ref.shape[1] >= 4096)


GROUPED = [
    # counts, N, K, G, zero_point, activation, gated, bias, gather
    ([1], 256, 128, 128, True, None, False, False, False),
    ([1, 0, 1], 130, 256, 64, True, "silu", True, False, True),
    ([0, 3, 0, 0, 5, 1, 0, 8], 512, 512, 128, True, "silu", True, True, True),
    ([2] * 7, 37, 96, 32, False, "relu", False, True, True),
    ([9, 8, 7, 16, 17, 0, 25], 258, 1024, 64, True, "gelu", True, False, True),
    ([40, 0, 1, 33], 515, 2048, 128, True, None, False, True, False),
    ([70, 64, 65, 3], 384, 512, 256, False, "gelu_tanh", True, True, True),
    ([200, 1, 129, 0, 131], 300, 1024, 128, True, "silu", True, False, True),
    ([191, 193, 384, 385], 256, 448, 64, True, None, False, False, False),
    ([300, 0, 0, 0], 1024, 256, 32, True, "silu", True, True, True),
    ([1] * 64, 256, 1024, 128, True, "silu", True, False, True),
    ([3] * 100 + [0] * 27 + [50], 64, 128, 32, True, "silu", True, False, True),
    ([1] * 1024, 64, 64, 32, True, None, False, False, True),
]


@pytest.mark.parametrize("c", GROUPED, ids=lambda c: f"E{len(c[0])}-R{sum(c[0])}-" + "-".join(map(str, c[1:])))
@pytest.mark.parametrize("gap", [0, 3])
def test_linear_grouped(lib, c, gap):
    counts, N, K, G, zp, act, gated, bias, gather = c
    w, X, b, rows, offsets, n_rows = _grouped(60, counts, N, K, G, zp, act, gated, bias, gather, gap=gap)
    n = N // 2 if gated else N
    buf = torch.full((n_rows + 2, n + 5), NAN, dtype=torch.float16, device="cuda")
    y = buf[1:1 + n_rows, 2:2 + n]
    out = lib.linear_grouped(X, *w, offsets, rows, G, zp, bias=b, activation=act, gated=gated, out=y)
    _finish(lib)
    assert out is y
    _check_grouped(y, X, w, G, b, rows, offsets, act, gated)
    y[gap:n_rows - gap] = NAN                 # everything else is as it was
    assert torch.isnan(buf).all()


MANY_EXPERTS = [
    # rows of an expert below, K, G, zero_point, activation, gated, bias: 64-row units (2048 / 1024 codes a row) or
    # 16-row tiles, by length; K / G odd, even and a multiple of 8
    (4, 512, 128, True, None, False, True),
    (4, 896, 128, True, "silu", True, False),
    (4, 896, 32, True, "relu", False, True),
    (4, 1408, 128, True, "silu", True, True),
    (4, 1408, 64, False, None, False, False),
    (11, 2048, 128, True, "gelu", True, True),
    (11, 2048, 64, True, None, False, True),
    (11, 1152, 32, True, "silu", True, False),
    (21, 640, 128, True, "silu", True, True),
    (41, 640, 64, True, None, False, True),
]


@pytest.mark.parametrize("c", MANY_EXPERTS, ids=lambda c: "-".join(map(str, c)))
def test_linear_grouped_many_experts(lib, c):
    """Uneven shares of 64 experts: none, one, above 4 and above 8 rows (a second set), above a tile's."""
    below, K, G, zp, act, gated, bias = c
    counts = [5 * e % below for e in range(64)]
    w, X, b, rows, offsets, n_rows = _grouped(66, counts, 770, K, G, zp, act, gated, bias, True, gap=2)
    y = lib.linear_grouped(X, *w, offsets, rows, G, zp, bias=b, activation=act, gated=gated,
                           out=torch.full((n_rows, 385 if gated else 770), NAN, dtype=torch.float16, device="cuda"))
    _finish(lib)
    _check_grouped(y, X, w, G, b, rows, offsets, act, gated)
    assert torch.isnan(y[:2]).all() and torch.isnan(y[-2:]).all()


@pytest.mark.parametrize("M", [1, 4, 6, 8, 13])
@pytest.mark.parametrize("N,K,G,act,gated", [(38003, 256, 128, "relu", False), (75842, 1152, 64, "silu", True),
                                             (38002, 1408, 32, None, False)])
def test_linear_fused_many_rows_of_weights(lib, M, N, K, G, act, gated):
    """64-row units with bias and residual, ragged in rows and in codes."""
    c = (M, N, K, G, True, act, gated, True, True)
    w, X, b, r = _case(c, 69)
    y = lib.linear_fused(X, *w, G, True, bias=b, activation=act, gated=gated, residual=r)
    _finish(lib)
    ref, bound = R.linear64(X, w, G, b, act, gated, r)
    R.assert_close(y, ref, bound, gated)


@pytest.mark.parametrize("M", [1, 5, 8, 14])
@pytest.mark.parametrize("K,G", [(640, 128), (640, 64), (896, 32), (1408, 128), (11008, 128)])
def test_linear_fused_lengths_of_scale_rows(lib, M, K, G):
    """Rows of 5, 10, 28, 11 and 86 scales: read by halves and by words."""
    w = R.packed(67, 130, K, G, True)
    X = R.activations(68, M, K)
    y = lib.linear_fused(X, *w, G, True)
    _finish(lib)
    ref, bound = R.linear64(X, w, G, None, None, False, None)
    R.assert_close(y, ref, bound, False)


@pytest.mark.parametrize("counts", [[2, 0, 3], [40, 9, 0], [150, 200, 30]])
@pytest.mark.parametrize("gather", [False, True])
def test_linear_grouped_strided_rows(lib, counts, gather):
    """X as columns of a wider tensor, in place and gathered (with and without the copy)."""
    N, K, G = 130, 384, 128
    w, X, b, rows, offsets, n_rows = _grouped(65, counts, N, K, G, True, "relu", False, True, gather, T=70)
    wide = torch.full((X.shape[0], K + 24), NAN, dtype=torch.float16, device="cuda")
    wide[:, 16:16 + K] = X
    y = lib.linear_grouped(wide[:, 16:16 + K], *w, offsets, rows, G, True, bias=b, activation="relu")
    _finish(lib)
    _check_grouped(y, X, w, G, b, rows, offsets, "relu", False)


@pytest.mark.parametrize("n_rows", [5, 40, 300])
def test_linear_grouped_bad_tables_stay_in_bounds(lib, n_rows):
    """Row numbers outside X count as rows of zeros; offsets outside 0..R are clamped."""
    N, K, G, E, T = 128, 256, 64, 3, 7
    w = R.packed(70, N, K, G, True, lead=(E,))
    X = R.activations(71, T, K)
    bias = torch.randn(E, N, generator=torch.Generator().manual_seed(5)).half().cuda()
    rows = torch.arange(n_rows, dtype=torch.int32, device="cuda") % T
    rows[1], rows[2], rows[n_rows - 1] = -1, T, 2 ** 31 - 1
    offsets = torch.tensor([-5, n_rows // 2, n_rows // 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    buf = torch.full((n_rows + 2, N), NAN, dtype=torch.float16, device="cuda")
    y = buf[1:1 + n_rows]
    lib.linear_grouped(X, *w, offsets, rows, G, True, bias=bias, out=y)
    _finish(lib)
    assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all()
    X0 = torch.cat((X, torch.zeros(1, K, dtype=torch.float16, device="cuda")))
    good = torch.where((rows < 0) | (rows >= T), T, rows)
    _check_grouped(y, X0, w, G, bias, good, torch.tensor([0, n_rows // 2, n_rows // 2, n_rows]), None, False)
    # a falling table: nothing outside Y is written, rows that no expert owns stay
    for table in ([n_rows, 0, 0, 0], [3, 2, 1, 0], [n_rows, n_rows, n_rows, n_rows]):
        buf.fill_(NAN)
        lib.linear_grouped(X, *w, torch.tensor(table, dtype=torch.int32, device="cuda"), rows, G, True, bias=bias, out=y)
        _finish(lib)
        assert torch.isnan(buf).all()


@pytest.mark.parametrize("ws", ["own", "none", "short", "given"])
def test_linear_grouped_gather_workspace(lib, ws):
    """Many gathered rows: with the copy into a workspace and without, rows outside X zero in both."""
    counts, N, K, G, E = [150, 0, 131, 90], 258, 512, 64, 4
    w, X, _, rows, offsets, n_rows = _grouped(77, counts, N, K, G, True, "silu", True, False, True, T=60, gap=5)
    rows[7], rows[160], rows[n_rows - 6] = -3, 60, 2 ** 30
    y = torch.full((n_rows, N // 2), NAN, dtype=torch.float16, device="cuda")
    kw = {}
    if ws != "own":
        size = {"none": 0, "short": n_rows * K * 2 - 256, "given": n_rows * K * 2 + 256}[ws]
        kw = dict(workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
    lib.linear_grouped(X, *w, offsets, rows, G, True, activation="silu", gated=True, out=y, **kw)
    _finish(lib)
    X0 = torch.cat((X, torch.zeros(1, K, dtype=torch.float16, device="cuda")))
    _check_grouped(y, X0, w, G, None, torch.where((rows < 0) | (rows >= 60), 60, rows), offsets, "silu", True)
    assert torch.isnan(y[:5]).all() and torch.isnan(y[n_rows - 5:]).all()


def test_linear_grouped_equals_the_dense_product(lib):
    """One expert with every row is linear_fused."""
    for M in (1, 5, 8, 20, 100, 400):
        w = R.packed(75, 384, 512, 128, True)
        X = R.activations(76, M, 512)
        a = lib.linear_fused(X, *w, 128, True, activation="silu", gated=True)
        b = lib.linear_grouped(X, *(t[None].contiguous() for t in w),
                               torch.tensor([0, M], dtype=torch.int32, device="cuda"), None, 128, True,
                               activation="silu", gated=True)
        _finish(lib)
        ref, bound = R.linear64(X, w, 128, None, "silu", True)
        R.assert_close(a, ref, bound, True)
        R.assert_close(b, ref, bound, True)


# ---------------------------------------------------------------------------
# routing and combination
# ---------------------------------------------------------------------------

# fp32 weights: expf is off by at most a few units (2^-22 relative with the argument's rounding of
# |l - top| <= 2^7 by half a unit), the sum of E terms by E 2^-24
def _weight_bound(E):
    return 2.0 ** -16 + E * 2.0 ** -24


def _check_route(r, logits, k, scoring, renorm):
    w, experts, offsets, rows, positions = R.route64(logits, k, scoring, renorm)
    assert r.experts.tolist() == experts
    assert r.offsets.tolist() == offsets
    assert r.rows.tolist() == rows
    assert r.positions.tolist() == positions
    w = torch.tensor(w, dtype=torch.float64).reshape(len(experts), k)
    got = r.weights.double().cpu()
    assert torch.isfinite(got).all()
    assert ((got - w).abs() <= _weight_bound(logits.shape[1]) * w + 2.0 ** -126).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 7, 7), (31, 33, 4), (32, 64, 6), (33, 128, 8), (100, 5, 1),
                                   (256, 16, 2), (257, 60, 4), (1000, 200, 10), (700, 257, 32), (300, 1024, 32),
                                   (5000, 8, 2), (13000, 40, 7), (12300, 130, 3), (12288, 9, 2), (9216, 64, 8), (9215, 64, 8),
                                   (6144, 72, 4), (6143, 72, 4), (33, 8, 2), (161, 32, 4)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_moe_route(lib, T, E, k, half, scoring, renorm):
    g = torch.Generator().manual_seed(T * 31 + E)
    x = 3 * torch.randn(T, E, generator=g)
    if E > 2:      # masks: single experts, and whole tokens
        x[torch.rand(T, E, generator=g) < 0.1] = -math.inf
        x[torch.rand(T, generator=g) < 0.1] = -math.inf
    x = x.half() if half else x
    r = lib.moe_route(x.cuda(), k, scoring=scoring, renormalize=renorm)
    torch.cuda.synchronize()
    _check_route(r, x, k, scoring, renorm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_moe_route_special_logits(lib, dtype, scoring, renorm):
    """Ties, signed zeros, the lowest finite value, infinities and NaN."""
    low, inf = torch.finfo(dtype).min, math.inf
    rows = [[0, 0, 0, 0, 0], [-0.0, 0.0, -0.0, 1, 1], [low] * 5, [low, low, 3, low, low], [-inf] * 5,
            [-inf, 2, -inf, -inf, -inf], [inf, 1, inf, 0, 0], [inf] * 5, [NAN, 1, NAN, 2, NAN], [NAN] * 5,
            [-inf, low, inf, NAN, 0], [-60, -61, -62, -80, -90], [60, 61, 62, 80, 90]]
    x = torch.tensor(rows, dtype=dtype)
    r = lib.moe_route(x.cuda(), 3, scoring=scoring, renormalize=renorm)
    torch.cuda.synchronize()
    _check_route(r, x, 3, scoring, renorm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(104, 5), (104, 70), (6500, 70)])
def test_moe_route_special_logits_of_many_tokens(lib, dtype, scoring, T, E):
    """The same rows where tokens are shared out to blocks, by warps and by four lanes."""
    low, inf = torch.finfo(dtype).min, math.inf
    rows = [[0, 0, 0, 0, 0], [-0.0, 0.0, -0.0, 1, 1], [low] * 5, [low, low, 3, low, low], [-inf] * 5,
            [-inf, 2, -inf, -inf, -inf], [inf, 1, inf, 0, 0], [inf] * 5, [NAN, 1, NAN, 2, NAN], [NAN] * 5,
            [-inf, low, inf, NAN, 0], [-60, -61, -62, -80, -90], [60, 61, 62, 80, 90]]
    x = torch.full((T, E), -inf, dtype=dtype)
    at = torch.randperm(E, generator=torch.Generator().manual_seed(E))[:5]
    x[:, at] = torch.tensor(rows, dtype=dtype).repeat(T // len(rows) + 1, 1)[:T]
    r = lib.moe_route(x.cuda(), 3, scoring=scoring, renormalize=True)
    torch.cuda.synchronize()
    _check_route(r, x, 3, scoring, True)


def test_moe_route_strided_logits_and_given_outputs(lib):
    T, E, k = 600, 24, 3
    x = torch.randn(T, E + 9, generator=torch.Generator().manual_seed(3)).cuda()
    guard = 17

    def buf(n, dtype):
        return torch.full((n + 2 * guard,), -7, dtype=dtype, device="cuda")
    b = [buf(T * k, torch.float32), buf(T * k, torch.int32), buf(E + 1, torch.int32), buf(T * k, torch.int32),
         buf(T * k, torch.int32)]
    v = [t[guard:-guard] for t in b]
    out = lib.MoeRoute(v[0].view(T, k), v[1].view(T, k), v[2], v[3], v[4].view(T, k))
    r = lib.moe_route(x[:, 4:4 + E], k, out=out)
    torch.cuda.synchronize()
    _check_route(r, x[:, 4:4 + E], k, "softmax", True)
    for t in b:
        assert (t[:guard] == -7).all() and (t[-guard:] == -7).all()


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (2, 2, 7), (5, 3, 130), (9, 8, 1024), (33, 6, 2054), (64, 5, 4096), (3, 33, 64)])
@pytest.mark.parametrize("residual", [False, True])
def test_moe_combine(lib, T, k, N, residual):
    g = torch.Generator().manual_seed(T + N)
    n_rows = T * k + 3
    Y = torch.randn(n_rows, N, generator=g).half().cuda()
    w = torch.rand(T, k, generator=g).cuda()
    pos = torch.randperm(n_rows, generator=g)[:T * k].reshape(T, k).int().cuda()
    pos[torch.rand(T, k, generator=g).cuda() < 0.2] = -1
    pos[0, 0] = n_rows                         # outside Y: contributes nothing, like -1
    if T > 1:
        pos[1] = -1
    unused = torch.ones(n_rows, dtype=torch.bool)
    used = pos[(pos >= 0) & (pos < n_rows)].long().cpu()
    unused[used] = False
    Y[unused.cuda()] = NAN                     # rows that no slot names are not read
    w[(pos < 0) | (pos >= n_rows)] = NAN       # nor the weights of slots without a row
    r = torch.randn(T, N, generator=g).half().cuda() if residual else None
    out = lib.moe_combine(Y, w, pos, residual=r)
    torch.cuda.synchronize()
    ok = (pos >= 0) & (pos < n_rows)
    terms = torch.where(ok[..., None], w.double()[..., None] * Y.double()[pos.long().clamp(0, n_rows - 1)], 0.0)
    ref = terms.sum(1) + (r.double() if residual else 0)
    size = terms.abs().sum(1) + (r.double().abs() if residual else 0)
    bound = (k + 2) * 2.0 ** -24 * size + R.HALF * ref.abs() * (1 + 2.0 ** -10) + 2.0 ** -24
    assert ((out.double() - ref).abs() <= bound).all()
    # strided and misaligned rows, in place on the residual
    if residual:
        buf = torch.full((T + 2, N + 3), NAN, dtype=torch.float16, device="cuda")
        o = buf[1:T + 1, 1:N + 1]
        o.copy_(r)
        lib.moe_combine(Y, w, pos, residual=o, out=o)
        torch.cuda.synchronize()
        assert torch.equal(o, out)
        o.fill_(NAN)
        assert torch.isnan(buf).all()


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

def _layer(lib, X, logits, gate_up, down, k, G, zp, stream=None, out=None):
    r = lib.moe_route(logits, k, stream=stream)
    h = lib.linear_grouped(X, *gate_up, r.offsets, r.rows, G, zp, activation="silu", gated=True, stream=stream)
    y = lib.linear_grouped(h, *down, r.offsets, None, G, zp, stream=stream)
    return lib.moe_combine(y, r.weights, r.positions, residual=X, stream=stream, out=out), r


def _layer64(X, r, gate_up, down, G, h16):
    """The layer from the kernel's own routing and its rounded hidden rows (h16 by row)."""
    out, size = X.double().clone(), X.double().abs()
    o = r.offsets.tolist()
    y = torch.zeros(r.rows.shape[0], X.shape[1], dtype=torch.float64, device="cuda")
    b = torch.zeros_like(y)
    for e in range(len(o) - 1):
        if o[e] < o[e + 1]:
            y[o[e]:o[e + 1]], b[o[e]:o[e + 1]] = R.linear64(h16[o[e]:o[e + 1]], tuple(None if t is None else t[e] for t in down), G)
    bound = torch.zeros_like(out)
    for j in range(r.weights.shape[1]):
        p = r.positions[:, j].long()
        ok = (p >= 0)
        w = r.weights[:, j].double()[:, None]
        out += torch.where(ok[:, None], w * y[p.clamp_min(0)], 0.0)
        size += torch.where(ok[:, None], (w * y[p.clamp_min(0)]).abs(), 0.0)
        bound += torch.where(ok[:, None], w * b[p.clamp_min(0)], 0.0)
    k = r.weights.shape[1]
    bound = bound + (k + 2) * 2.0 ** -24 * size
    return out, bound + R.HALF * (out.abs() + bound) + 2.0 ** -24


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (6, 8, 2), (40, 16, 4), (300, 6, 2)])
@pytest.mark.parametrize("zp", [True, False])
def test_moe_layer(lib, T, E, k, zp):
    """Routing, both grouped products and the combination as a layer runs them, some tokens padded."""
    H, F, G = 512, 384, 64
    gate_up = R.packed(90, 2 * F, H, G, zp, lead=(E,), scale=0.005)
    down = R.packed(91, H, F, G, zp, lead=(E,), scale=0.005)
    X = R.activations(92, T, H)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(8)).cuda()
    if T > 2:
        logits[T - 2:] = -math.inf
    out, r = _layer(lib, X, logits, gate_up, down, k, G, zp)
    _finish(lib)
    _check_route(r, logits, k, "softmax", True)
    h = lib.linear_grouped(X, *gate_up, r.offsets, r.rows, G, zp, activation="silu", gated=True)
    _check_grouped(h, X, gate_up, G, None, r.rows, r.offsets, "silu", True)
    ref, bound = _layer64(X, r, gate_up, down, G, h)
    assert ((out.double() - ref).abs() <= bound).all()
    if T > 2:
        assert torch.equal(out[T - 2:], X[T - 2:])     # padded tokens pass through


@pytest.mark.parametrize("T", [2, 50])
def test_moe_layer_captured_and_replayed(lib, T):
    """A captured layer follows new logits and inputs on replay; two graphs run at once on two
    streams give what they give alone."""
    E, k, H, F, G = 8, 2, 256, 128, 64
    gate_up = R.packed(95, 2 * F, H, G, True, lead=(E,), scale=0.01)
    down = R.packed(96, H, F, G, True, lead=(E,), scale=0.01)
    X = [R.activations(97 + i, T, H) for i in range(2)]
    logits = [torch.randn(T, E, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    eager = [[_layer(lib, X[i], logits[j], gate_up, down, k, G, True)[0].clone() for j in range(2)] for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs, ins, streams = [], [], [], []
    for i in range(2):
        x, l = X[i].clone(), logits[i].clone()
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _layer(lib, x, l, gate_up, down, k, G, True)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            o, _ = _layer(lib, x, l, gate_up, down, k, G, True)
        graphs.append(g), outs.append(o), ins.append((x, l)), streams.append(s)
    for swap in (False, True, False):
        for i in range(2):
            ins[i][1].copy_(logits[1 - i if swap else i])
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        lib.device_error()
        for i in range(2):
            assert torch.equal(outs[i], eager[i][1 - i if swap else i])


FIRST_CALL = """
import sys; sys.path[:0] = ["tests", "."]
import torch
import fused_reference as R
from bit_weight_only_linear_b200 import awq
w = [R.packed(1, 256, 1024, 128, True), R.packed(2, 256, 1024, 128, True, lead=(4,))]
X = {m: R.activations(m, m, 1024) for m in (2, 61, 300)}
logits = {m: torch.randn(m, 4, generator=torch.Generator().manual_seed(m)).cuda() for m in X}
def calls(m):
    r = awq.moe_route(logits[m], 2)
    h = awq.linear_grouped(X[m], *w[1], r.offsets, r.rows, 128, True)
    return [awq.linear_fused(X[m], *w[0], 128, True), awq.moe_combine(h, r.weights, r.positions)]
torch.cuda.synchronize()
outs = {}
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for m in X:
        outs[m] = calls(m)
g.replay()
torch.cuda.synchronize()
awq.device_error()
for m in X:
    assert all(torch.equal(a, b) for a, b in zip(outs[m], calls(m))), m
print("captured")
"""


def test_first_calls_inside_a_capture(lib):
    """A process whose first call of every form is a captured one."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_dense_mlp_on_a_side_stream(lib):
    """gate_up and down as linear_fused pairs on a stream of their own, behind a copy on it."""
    M, H, F, G = 20, 512, 640, 128
    gate_up, down = R.packed(100, 2 * F, H, G, True, scale=0.005), R.packed(101, H, F, G, True, scale=0.005)
    src = R.activations(102, M, H)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    X = torch.zeros_like(src)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        X.copy_(src)
    h = lib.linear_fused(X, *gate_up, G, True, activation="silu", gated=True, stream=s)
    y = lib.linear_fused(h, *down, G, True, residual=X, stream=s)
    s.synchronize()
    _finish(lib)
    ref, bound = R.linear64(src, gate_up, G, None, "silu", True)
    R.assert_close(h, ref, bound, True)
    ref, bound = R.linear64(h, down, G, None, None, False, src)
    R.assert_close(y, ref, bound)


def test_results_do_not_change_from_call_to_call(lib):
    E, k, T, H, F, G = 8, 2, 90, 1024, 512, 128
    gate_up = R.packed(110, 2 * F, H, G, True, lead=(E,), scale=0.01)
    X = R.activations(111, T, H)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(9)).cuda()
    first = None
    for _ in range(10):
        r = lib.moe_route(logits, k)
        h = lib.linear_grouped(X, *gate_up, r.offsets, r.rows, G, True, activation="silu", gated=True)
        d = [lib.linear_fused(X[:m], *(t[0].contiguous() for t in gate_up), G, True) for m in (1, 8, 16, 90)]
        now = [t.clone() for t in (*r, h, *d)]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
    _finish(lib)
