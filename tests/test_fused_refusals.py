"""CPU: the fused / grouped linears, routing and combination refuse bad arguments before anything
is launched (no GPU is needed: every call below fails its checks, or has nothing to do)."""
import pytest
import torch

FAKE = 0x10000      # 16-byte aligned, never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def clib():
    from bit_weight_only_linear_b200 import awq, build
    build.build()
    return awq.load_library()


def _cfg(g=128, zp=1, bits=4):
    from bit_weight_only_linear_b200.awq import QuantConfig
    return QuantConfig(bits, g, zp)


def _fused(clib, **kw):
    a = dict(X=FAKE, M=4, ldx=256, q=FAKE, s=FAKE, z=FAKE, N=64, K=256, c=_cfg(), b=0, act=0, gated=0, r=0, ldr=0,
             Y=FAKE, ldy=64)
    a.update(kw)
    return clib.awq_linear_fused(a["X"], a["M"], a["ldx"], a["q"], a["s"], a["z"], a["N"], a["K"], a["c"], a["b"],
                                 a["act"], a["gated"], a["r"], a["ldr"], a["Y"], a["ldy"], None)


def _grouped(clib, **kw):
    a = dict(X=FAKE, T=4, ldx=256, rows=0, R=4, o=FAKE, E=3, q=FAKE, s=FAKE, z=FAKE, N=64, K=256, c=_cfg(), b=0, act=0,
             gated=0, Y=FAKE, ldy=64, ws=0, wb=0)
    a.update(kw)
    return clib.awq_linear_grouped(a["X"], a["T"], a["ldx"], a["rows"], a["R"], a["o"], a["E"], a["q"], a["s"], a["z"],
                                   a["N"], a["K"], a["c"], a["b"], a["act"], a["gated"], a["Y"], a["ldy"],
                                   a["ws"], a["wb"], None)


@pytest.mark.parametrize("call", [_fused, _grouped])
@pytest.mark.parametrize("kw,status", [
    (dict(c=_cfg(bits=3)), UNSUPPORTED), (dict(c=_cfg(g=48)), UNSUPPORTED), (dict(c=_cfg(zp=2)), INVALID),
    (dict(K=200), INVALID), (dict(N=0), INVALID), (dict(N=-64), INVALID), (dict(X=0), INVALID), (dict(X=FAKE + 2), INVALID),
    (dict(q=0), INVALID), (dict(q=FAKE + 8), INVALID), (dict(s=0), INVALID), (dict(s=FAKE + 2), INVALID),
    (dict(z=0), INVALID), (dict(z=FAKE + 4), INVALID), (dict(Y=0), INVALID), (dict(Y=FAKE + 1), INVALID),
    (dict(b=FAKE + 1), INVALID), (dict(act=-1), INVALID), (dict(act=5), INVALID), (dict(gated=2), INVALID),
    (dict(gated=1, N=63, ldy=64), INVALID), (dict(ldx=255), INVALID), (dict(ldx=248), INVALID), (dict(ldx=257), INVALID),
    (dict(ldy=63), INVALID), (dict(gated=1, ldy=31), INVALID),
])
def test_linear_argument_errors(clib, call, kw, status):
    assert call(clib, **kw) == status


def test_fused_only(clib):
    assert _fused(clib, M=-1) == INVALID
    assert _fused(clib, r=FAKE, ldr=63) == INVALID
    assert _fused(clib, r=FAKE + 1, ldr=64) == INVALID
    assert _fused(clib, M=0, X=0, Y=0) == OK
    assert _fused(clib, M=(1 << 30) + 1) == UNSUPPORTED
    assert _fused(clib, N=0x7ffffe01, ldy=0x7ffffe01) == UNSUPPORTED


def test_grouped_only(clib):
    assert _grouped(clib, R=-1) == INVALID
    assert _grouped(clib, T=-1) == INVALID
    assert _grouped(clib, E=0) == INVALID
    assert _grouped(clib, E=1025) == INVALID
    assert _grouped(clib, o=0) == INVALID
    assert _grouped(clib, o=FAKE + 2) == INVALID
    assert _grouped(clib, rows=FAKE + 2) == INVALID
    assert _grouped(clib, R=5) == INVALID                       # rows of X missing
    assert _grouped(clib, T=0, rows=FAKE) == INVALID
    assert _grouped(clib, ws=FAKE + 8, wb=1 << 20) == INVALID
    assert clib.awq_linear_grouped_workspace_bytes(100, 8, 4096) == 0          # few rows are gathered in place
    assert clib.awq_linear_grouped_workspace_bytes(8000, 8, 4096) == 8000 * 8192
    assert clib.awq_linear_grouped_workspace_bytes(-1, 8, 4096) == 0
    assert _grouped(clib, E=1024, N=1 << 22, ldy=1 << 22) == UNSUPPORTED
    assert _grouped(clib, R=(1 << 30) + 1, T=1 << 30, rows=FAKE) == UNSUPPORTED
    assert _grouped(clib, R=0, T=0, X=0, Y=0) == OK


def _route(clib, **kw):
    a = dict(l=FAKE, half=0, T=4, ld=8, E=8, k=2, sc=0, rn=1, w=FAKE, e=FAKE, o=FAKE, r=FAKE, p=FAKE, ws=0, wb=0)
    a.update(kw)
    return clib.awq_moe_route(a["l"], a["half"], a["T"], a["ld"], a["E"], a["k"], a["sc"], a["rn"], a["w"], a["e"], a["o"],
                              a["r"], a["p"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0, k=1), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(ld=7), INVALID),
    (dict(half=2), INVALID), (dict(sc=2), INVALID), (dict(sc=-1), INVALID), (dict(rn=2), INVALID),
    (dict(E=1025, ld=1025), UNSUPPORTED), (dict(E=64, ld=64, k=33), UNSUPPORTED), (dict(T=(1 << 22) + 1), UNSUPPORTED),
    (dict(l=0), INVALID), (dict(w=0), INVALID), (dict(e=0), INVALID), (dict(o=0), INVALID), (dict(r=0), INVALID),
    (dict(p=0), INVALID), (dict(l=FAKE + 2), INVALID), (dict(l=FAKE + 1, half=1), INVALID), (dict(w=FAKE + 2), INVALID),
    (dict(p=FAKE + 1), INVALID), (dict(ws=FAKE + 8, wb=1 << 20), INVALID),
])
def test_route_argument_errors(clib, kw, status):
    assert _route(clib, **kw) == status


def _combine(clib, **kw):
    a = dict(Y=FAKE, R=4, ldy=64, w=FAKE, p=FAKE, T=2, k=2, N=64, r=0, ldr=0, o=FAKE, ldo=64)
    a.update(kw)
    return clib.awq_moe_combine(a["Y"], a["R"], a["ldy"], a["w"], a["p"], a["T"], a["k"], a["N"], a["r"], a["ldr"], a["o"],
                                a["ldo"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INVALID), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(N=0), INVALID), (dict(ldy=63), INVALID),
    (dict(ldo=63), INVALID), (dict(r=FAKE, ldr=63), INVALID), (dict(Y=0), INVALID), (dict(Y=FAKE + 1), INVALID),
    (dict(r=FAKE + 1, ldr=64), INVALID), (dict(o=0), INVALID), (dict(o=FAKE + 1), INVALID), (dict(w=0), INVALID),
    (dict(w=FAKE + 2), INVALID), (dict(p=0), INVALID), (dict(p=FAKE + 2), INVALID), (dict(T=0, w=0, p=0, o=0), OK),
])
def test_combine_argument_errors(clib, kw, status):
    assert _combine(clib, **kw) == status


def test_binding_refuses_cpu_tensors():
    from bit_weight_only_linear_b200 import awq
    x = torch.zeros(2, 128, dtype=torch.float16)
    q = torch.zeros(8, 16, dtype=torch.int32)
    s = torch.zeros(8, 1, dtype=torch.float16)
    for f in (lambda: awq.linear_fused(x, q, s, None, 128, False),
              lambda: awq.linear_grouped(x, q[None], s[None], None, torch.zeros(2, dtype=torch.int32), None, 128, False),
              lambda: awq.moe_route(torch.zeros(2, 4), 2),
              lambda: awq.moe_combine(x, torch.zeros(2, 1), torch.zeros(2, 1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            f()
