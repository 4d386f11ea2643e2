"""Refusals of the decode entries: the C ABI with fake device addresses, before
any HIP call, and the Python wrappers on host tensors (no GPU needed)."""

import pytest

import mxfp4_activation_amd as wush
from mxfp4_activation_amd import _lib

A = 1 << 20  # fake device address: never dereferenced
B = A * 64
EINVAL, EALIGN, EUNSUPPORTED, OK = _lib.WUSH_EINVAL, _lib.WUSH_EALIGN, _lib.WUSH_EUNSUPPORTED, _lib.WUSH_OK


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_linear_w4_refusals(fmt):
    lib = wush.load()
    G = 16 if fmt == 1 else 32

    def f(fmt=fmt, X=A, ldx=4 * G, T=None, c=A * 2, s=A * 3, g=A * 4, M=2, N=8, K=4 * G, Y=B, ot=0, ws=None, n=0):
        return lib.wush_linear_w4(fmt, X, ldx, T, c, s, g, M, N, K, Y, ot, ws, n, None)

    assert f(M=0) == OK and f(N=0) == OK
    assert f(fmt=3) == EUNSUPPORTED
    assert f(ot=2) == EINVAL
    assert f(M=-1) == EINVAL and f(N=-1) == EINVAL
    assert f(K=G // 2) == EINVAL and f(K=0) == EINVAL
    assert f(X=None) == EINVAL and f(c=None) == EINVAL and f(s=None) == EINVAL and f(Y=None) == EINVAL
    assert f(ldx=4 * G - 8) == EINVAL
    assert f(ldx=4 * G + 4) == EALIGN
    assert f(X=A + 8) == EALIGN
    assert f(c=A * 2 + 4) == EALIGN
    assert f(Y=B + 2) == EALIGN
    assert f(T=A * 5) == EINVAL  # workspace missing
    assert b"workspace" in lib.wush_last_error()
    need = lib.wush_linear_w4_workspace(2, 4 * G, 0)
    assert need == 2 * 3 * 2 * 4 * G
    assert f(T=A * 5, ws=B * 2, n=need - 1) == EINVAL
    assert f(T=A * 5, ws=B * 2 + 8, n=need) == EALIGN
    assert f(T=A * 5 + 2, ws=B * 2, n=need) == EALIGN
    assert f(T=A * 5, ws=B, n=need) == EINVAL  # workspace overlaps Y
    assert f(T=A * 5, ws=A, n=need) == EINVAL  # workspace overlaps X
    assert f(Y=A) == EINVAL and f(Y=A * 2) == EINVAL and f(Y=A * 3) == EINVAL
    if fmt == 1:
        assert f(g=None) == EINVAL
        assert f(g=A * 4 + 2) == EALIGN
        assert f(Y=A * 4) == EINVAL
    if fmt == 2:
        assert f(s=A * 3 + 1) == EALIGN
    assert lib.wush_linear_w4_workspace(0, 64, 0) == 0


def test_moe_w4_refusals():
    lib = wush.load()

    def f(fmt=0, X=A, ldx=64, r=A * 2, gc=A * 3, gs=A * 4, gg=None, ti=None, dc=A * 5, ds=A * 6, dg=None, tm=None, M=2,
          E=4, k=2, H=64, I=32, Y=B, ot=0, ids=B * 2, w=B * 3, ws=B * 4, n=1 << 20):
        return lib.wush_moe_w4(fmt, X, ldx, r, gc, gs, gg, ti, dc, ds, dg, tm, M, E, k, 1, H, I, Y, ot, ids, w, ws, n,
                               None)

    assert f(M=0) == OK
    assert f(fmt=5) == EUNSUPPORTED
    assert f(ot=7) == EINVAL
    assert f(M=-1) == EINVAL
    assert f(E=0) == EINVAL and f(E=1025) == EINVAL
    assert f(k=0) == EINVAL and f(k=5) == EINVAL and f(E=64, k=33) == EINVAL
    assert f(H=48) == EINVAL and f(I=40) == EINVAL and f(H=1 << 25) == EINVAL
    for name in ("X", "r", "gc", "gs", "dc", "ds", "Y", "ids", "w", "ws"):
        assert f(**{name: None}) == EINVAL, name
    assert f(fmt=1, gg=None, dg=A * 8) == EINVAL
    assert f(fmt=1, gg=A * 8, dg=None) == EINVAL
    assert f(X=A + 2) == EALIGN and f(ldx=68) == EALIGN and f(ldx=56) == EINVAL
    assert f(r=A * 2 + 8) == EALIGN and f(gc=A * 3 + 4) == EALIGN and f(ids=B * 2 + 2) == EALIGN
    assert f(ti=A * 7 + 8) == EALIGN and f(tm=A * 7 + 8) == EALIGN
    need = lib.wush_moe_w4_workspace(2, 4, 2, 64, 32, 0, 0)
    assert need > 0 and f(n=need - 1) == EINVAL
    assert lib.wush_moe_w4_workspace(2, 4, 2, 64, 32, 1, 0) > need
    # Tokens beyond 64 reuse the workspace.
    assert lib.wush_moe_w4_workspace(64, 4, 2, 64, 32, 1, 0) == lib.wush_moe_w4_workspace(999, 4, 2, 64, 32, 1, 0)
    assert f(Y=A) == EINVAL and f(ids=A * 3) == EINVAL and f(w=B) == EINVAL and f(ws=A * 5) == EINVAL


def test_token_logprobs_refusals():
    lib = wush.load()

    def f(L=A, t=0, ld=100, R=4, V=100, tg=A * 2, top=5, lp=B, en=B * 2, ti=B * 3, tl=B * 4, ws=B * 5, n=1 << 20):
        return lib.wush_token_logprobs(L, t, ld, R, V, tg, top, lp, en, ti, tl, ws, n, None)

    assert f(R=0) == OK
    assert f(t=3) == EINVAL and f(t=-1) == EINVAL
    assert f(R=-1) == EINVAL and f(V=0) == EINVAL and f(V=1 << 31) == EINVAL
    assert f(top=-1) == EINVAL and f(top=33) == EINVAL
    assert f(ld=99) == EINVAL
    for name in ("L", "tg", "lp", "en", "ti", "tl"):
        assert f(**{name: None}) == EINVAL, name
    assert f(L=A + 2) == EALIGN and f(t=1, L=A + 1) == EALIGN and f(tg=A * 2 + 4) == EALIGN and f(lp=B + 2) == EALIGN
    assert f(V=100000, ld=100000, ws=None, n=0) == EINVAL  # several workgroups share a row: workspace
    assert lib.wush_token_logprobs_workspace(4, 100, 0, 5) == 0
    assert f(lp=A) == EINVAL and f(en=B) == EINVAL and f(ti=A * 2) == EINVAL


def test_wrappers_refuse_host_tensors_and_bad_names():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        wush.linear_w4("mxfp4", x, c, s)
    with pytest.raises(ValueError, match="fmt must be"):
        wush.linear_w4("fp4", x, c, s)
    with pytest.raises(ValueError, match="out_dtype"):
        wush.linear_w4("mxfp4", x, c, s, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="bfloat16"):
        wush.linear_w4("mxfp4", x.float(), c, s)
    with pytest.raises(ValueError, match="contiguous rows"):
        wush.linear_w4("mxfp4", torch.zeros(64, 2, dtype=torch.bfloat16).t(), c, s)
    with pytest.raises(TypeError, match="logits must be"):
        wush.token_logprobs(torch.zeros(2, 8, dtype=torch.float64), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="device tensor"):
        wush.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))
