"""GPU: what the binding of the fused / grouped linears, routing and combination refuses."""
import pytest
import torch

import fused_reference as R

pytestmark = pytest.mark.gpu


def _t(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_linear_fused_refusals(lib):
    w = R.packed(1, 64, 256, 64, True)
    X = _t(4, 256)
    bad = [
        lambda: lib.linear_fused(X.float(), *w, 64, True),                       # type
        lambda: lib.linear_fused(X[0], *w, 64, True),                            # dimensions
        lambda: lib.linear_fused(_t(4, 512), *w, 64, True),                      # K
        lambda: lib.linear_fused(_t(256, 4).T, *w, 64, True),                    # columns, not rows
        lambda: lib.linear_fused(_t(1, 256).expand(4, 256), *w, 64, True),       # overlapping rows
        lambda: lib.linear_fused(X, *w, 128, True),                              # scales of another group size
        lambda: lib.linear_fused(X, *w, 48, True),
        lambda: lib.linear_fused(X, w[0], w[1], None, 64, True),                 # zeros missing
        lambda: lib.linear_fused(X, *w, 64, False),                              # zeros too many
        lambda: lib.linear_fused(X, *w, 64, True, activation="tanh"),
        lambda: lib.linear_fused(X, *w, 64, True, bias=_t(63)),
        lambda: lib.linear_fused(X, *w, 64, True, bias=_t(64).float()),
        lambda: lib.linear_fused(X, *w, 64, True, bias=_t(64).cpu()),
        lambda: lib.linear_fused(X, *w, 64, True, gated=True, residual=_t(4, 64)),
        lambda: lib.linear_fused(X, *w, 64, True, residual=_t(1, 64).expand(4, 64)),
        lambda: lib.linear_fused(X, *w, 64, True, out=_t(4, 65)),
        lambda: lib.linear_fused(X, *w, 64, True, out=_t(64, 4).T),
        lambda: lib.linear_fused(X, *(t[:63] for t in w), 64, True, gated=True),  # odd N
        lambda: lib.linear_fused(X, w[0][None], w[1], w[2], 64, True),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for x in (_t(4, 264)[:, 4:260], _t(4, 260)[:, :256]):                        # rows off 16 bytes
        with pytest.raises(lib.AWQError) as e:
            lib.linear_fused(x, *w, 64, True)
        assert e.value.status == lib.AWQ_ERR_INVALID_ARG


def test_linear_grouped_refusals(lib):
    w = R.packed(2, 64, 256, 64, True, lead=(3,))
    X, o = _t(4, 256), _t(4, dtype=torch.int32)
    for f in [
        lambda: lib.linear_grouped(X, *w, o[:3], None, 64, True),
        lambda: lib.linear_grouped(X, *w, o.long(), None, 64, True),
        lambda: lib.linear_grouped(X, *w, o.cpu(), None, 64, True),
        lambda: lib.linear_grouped(X, *w, o, _t(4, dtype=torch.int64), 64, True),
        lambda: lib.linear_grouped(X, *w, o, _t(8, dtype=torch.int32)[::2], 64, True),
        lambda: lib.linear_grouped(X, *w, o, None, 64, True, bias=_t(64)),
        lambda: lib.linear_grouped(X, *w, o, None, 64, True, out=_t(5, 64)),
        lambda: lib.linear_grouped(X, w[0][0], w[1][0], w[2][0], o, None, 64, True),
        lambda: lib.linear_grouped(X, w[0], w[1][:2], w[2], o, None, 64, True),
    ]:
        with pytest.raises(ValueError):
            f()


def test_route_and_combine_refusals(lib):
    l = _t(4, 8, dtype=torch.float32)
    for f in [
        lambda: lib.moe_route(l.double(), 2), lambda: lib.moe_route(l[0], 2), lambda: lib.moe_route(l.T, 2),
        lambda: lib.moe_route(l, 2, scoring="max"),
        lambda: lib.moe_combine(_t(8, 16), l[:, :2].contiguous(), _t(4, 2, dtype=torch.int64)),
        lambda: lib.moe_combine(_t(8, 16), l[:, :3].contiguous(), _t(4, 2, dtype=torch.int32)),
        lambda: lib.moe_combine(_t(8, 16), _t(4, 2), _t(4, 2, dtype=torch.int32)),
        lambda: lib.moe_combine(_t(8, 16), l[:, :2].contiguous(), _t(4, 2, dtype=torch.int32), residual=_t(4, 15)),
    ]:
        with pytest.raises(ValueError):
            f()
    for k in (0, 9):
        with pytest.raises(lib.AWQError):
            lib.moe_route(l, k)
    with pytest.raises(lib.AWQError) as e:
        lib.moe_route(_t(1000, 8, dtype=torch.float32), 2, workspace=_t(16, dtype=torch.uint8))
    assert e.value.status == 3


def test_workspaces_refused(lib):
    """A workspace elsewhere than on the device, or in pieces; a top_k that no tensor could hold."""
    w = R.packed(3, 64, 256, 64, True, lead=(2,))
    X, o = _t(4, 256), _t(3, dtype=torch.int32)
    l = _t(1000, 8, dtype=torch.float32)
    for ws in (torch.zeros(1 << 16, dtype=torch.uint8), _t(1 << 16, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError):
            lib.linear_grouped(X, *w, o, _t(4, dtype=torch.int32), 64, True, workspace=ws)
        with pytest.raises(ValueError):
            lib.moe_route(l, 2, workspace=ws)
    for k in (-1, 1 << 40):
        with pytest.raises(lib.AWQError):
            lib.moe_route(l, k)
