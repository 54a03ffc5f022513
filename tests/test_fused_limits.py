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
