"""CPU: sizes at the end of the 32-bit range are refused, not turned into other sizes (nothing is launched)."""
import pytest

from test_fused_refusals import FAKE, UNSUPPORTED, _cfg, _combine, _fused, _grouped, clib  # noqa: F401

LAST = 2 ** 31 - 1


@pytest.mark.parametrize("call", [_fused, _grouped])
@pytest.mark.parametrize("G", [32, 128, 256])
def test_rows_of_weights_too_long(clib, call, G):
    K = 2 ** 31 - 256 if G == 256 else 2 ** 31 - G
    assert call(clib, K=K, ldx=K, c=_cfg(g=G)) == UNSUPPORTED


@pytest.mark.parametrize("N", [65535 * 128 + 1, LAST - 127, LAST - 126, LAST])
def test_combined_rows_too_wide(clib, N):
    assert _combine(clib, N=N, ldy=N, ldo=N, o=FAKE) == UNSUPPORTED


@pytest.mark.parametrize("E", [1, 8, 128, 1024])
def test_the_bindings_shortcuts_follow_the_library(clib, E):
    """Below these counts the binding asks for no workspace without asking the library: the library must need
    none there, and one from there on."""
    from bit_weight_only_linear_b200 import awq
    T, R = awq._ROUTE_SINGLE, awq._GATHER_MIN_SHARE * E
    assert all(clib.awq_moe_route_workspace_bytes(t, E) == 0 for t in range(T + 1))
    assert clib.awq_moe_route_workspace_bytes(T + 1, E) > 0
    assert all(clib.awq_linear_grouped_workspace_bytes(r, E, 128) == 0 for r in range(R))
    assert clib.awq_linear_grouped_workspace_bytes(R, E, 128) > 0
