"""Refusals of dflash_logprobs and dflash_logprobs_grad, checked on the host
before any HIP call (no GPU needed)."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
FAR = ctypes.c_void_p(0x7000000000)


@pytest.fixture(scope="module")
def dfl():
    import block_draft_select_amd as m
    return m


def _rows(dfl, R=3, stride=100000, V=100000, dtype=1):
    return dfl.dflash_rows(R, stride, V, dtype)


def _ws(dfl, r):
    n = ctypes.c_size_t(777)
    return dfl.lib.dflash_rows_workspace_bytes(ctypes.byref(r), ctypes.byref(n)), n.value


def _fwd(dfl, r, Z=FAKE, T=None, group=1, M=2, tok=FAKE, logp=FAKE, norm=FAKE, ent=None, N=3, top=FAKE, top_logp=FAKE, ws=FAKE,
         n=1 << 40):
    return dfl.lib.dflash_logprobs(ctypes.byref(r) if r is not None else None, Z, T, group, M, tok, logp, norm, ent, N, top,
                                   top_logp, ws, n, None)


def _grad(dfl, r, Z=FAKE, T=None, group=1, M=2, tok=FAKE, g=FAKE, ge=None, norm=FAKE, ent=None, dZ=FAR, stride=100000):
    return dfl.lib.dflash_logprobs_grad(ctypes.byref(r) if r is not None else None, Z, T, group, M, tok, g, ge, norm, ent, dZ,
                                        stride, None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), 1), (dict(V=0), 1), (dict(dtype=2), 1), (dict(stride=99999), 1), (dict(R=4194305), 2),
    (dict(V=2097153, stride=2097153), 2), (dict(stride=(1 << 40) + 1), 2), (dict(R=4194304, stride=1 << 21, V=1 << 21), 2),
])
def test_bad_rows(dfl, kw, status):
    r = _rows(dfl, **kw)
    assert _fwd(dfl, r) == status and _grad(dfl, r) == status
    assert dfl.lib.dflash_last_error() != b""


def test_bad_arguments(dfl):
    r = _rows(dfl)
    assert _fwd(dfl, None) == 1 and _grad(dfl, None) == 1
    for kw in (dict(Z=None), dict(Z=ODD), dict(tok=None), dict(logp=None), dict(norm=None), dict(M=-1), dict(M=1025), dict(group=0),
               dict(group=-2), dict(N=-1), dict(N=33), dict(top=None), dict(top_logp=None)):
        assert _fwd(dfl, r, **kw) == 1, kw
    for kw in (dict(Z=None), dict(Z=ODD), dict(tok=None), dict(g=None), dict(norm=None), dict(M=-1), dict(M=1025), dict(group=0),
               dict(dZ=None), dict(dZ=ODD), dict(stride=99999), dict(stride=(1 << 40) + 1), dict(ge=FAKE)):
        assert _grad(dfl, r, **kw) in (1, 2), kw
    assert _grad(dfl, r, ge=FAKE) == 1 and b"entropy" in dfl.lib.dflash_last_error()


def test_workspaces(dfl):
    r = _rows(dfl, V=151936, stride=151936)  # few long rows: several segments
    assert _fwd(dfl, r, ws=None) == 3 and _fwd(dfl, r, ws=ctypes.c_void_p(0x10008)) == 3 and _fwd(dfl, r, n=16) == 3


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("V", [1, 5000, 8193, 16384, 32000, 151936, 2097152])
def test_a_workspace_serves_fewer_rows_too(dfl, dtype, V):
    last = 0
    for R in sorted({1, 2, 3, 7, 8, 31, 41, 64, 100, 128, 195, 342, 683, 1023, 1024, 1025, 2047, 2048, 4097}):
        r = _rows(dfl, R=R, stride=V, V=V, dtype=dtype)
        status, n = _ws(dfl, r)
        assert status == 0 and n >= last
        last = n
        for N in (0, 1, 32):
            # few long rows need one; a call that needs none would be launched here
            if R < 64 and V * (2 if dtype else 4) > 262144:
                assert _fwd(dfl, r, N=N, n=0) == 3
                assert int(dfl.lib.dflash_last_error().split(b"need ")[1].split()[0]) <= n, (R, V)


def test_overlapping_gradients_are_refused(dfl):
    r = _rows(dfl, R=3, stride=120, V=100)
    at = lambda e: ctypes.c_void_p(0x100000 + 2 * e)  # noqa: E731
    for e, stride in ((1, 120), (99, 120), (-50, 120), (0, 121), (119, 120), (240, 100)):
        assert _grad(dfl, r, Z=at(0), dZ=at(e), stride=stride) == 1, (e, stride)
        assert b"overlaps" in dfl.lib.dflash_last_error()


@pytest.mark.parametrize("at", [0, 100, 3 * 240 - 42, -4])
def test_outputs_over_their_rows_are_refused(dfl, at):
    # 3 rows of 100 bf16 logits, 240 bytes apart: 680 bytes
    r = _rows(dfl, R=3, stride=120, V=100)
    rows_, there, away = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100000 + at), ctypes.c_void_p(0x7000000000)
    out = dict(Z=rows_, tok=away, logp=away, norm=away, top=away, top_logp=away)
    for name in ("logp", "norm", "ent", "top", "top_logp"):
        assert _fwd(dfl, r, **{**out, name: there}) == 1, name
        assert b"overlaps Z" in dfl.lib.dflash_last_error()
    given = dict(Z=away, dZ=rows_, stride=120, tok=away, g=away, norm=away, ge=away, ent=away)
    for name in ("T", "tok", "g", "norm", "ge", "ent"):
        assert _grad(dfl, r, **{**given, name: there}) == 1, name
        assert b"dZ overlaps" in dfl.lib.dflash_last_error()


def test_empty_calls_launch_nothing(dfl):
    r = _rows(dfl, R=0)
    assert _fwd(dfl, r, Z=None, tok=None, logp=None, norm=None, top=None, top_logp=None, ws=None, n=0) == 0
    assert _grad(dfl, r, Z=None, tok=None, g=None, norm=None, dZ=None) == 0
    assert _fwd(dfl, r, M=-1) == 1 and _fwd(dfl, r, N=99) == 1  # but a wrong call is wrong


def test_binding_refusals(dfl):
    z = torch.zeros(4, 10)
    r = dfl.rows(z)
    tok, lp, norm = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 2)
    ws = torch.zeros(64, dtype=torch.uint8)
    for a, b in ((tok, None), (None, lp), (tok, torch.zeros(4, 3)), (tok.long(), lp), (tok, lp.double())):
        with pytest.raises((ValueError, TypeError)):
            dfl.dflash_logprobs(r, z, a, b, norm, ws)
        with pytest.raises((ValueError, TypeError)):
            dfl.dflash_logprobs_grad(r, z, a, b, norm, z)
    with pytest.raises(ValueError, match="device tensor"):
        dfl.dflash_logprobs(r, z, tok, lp, norm, ws)
    with pytest.raises(ValueError, match="together"):
        dfl.dflash_logprobs(r, z, None, None, norm, ws, top_idx=tok)
    for group in (0, -1, 1 << 31):
        with pytest.raises(ValueError, match="group"):
            dfl.dflash_logprobs(r, z, None, None, norm, ws, group=group)
        with pytest.raises(ValueError, match="group"):
            dfl.dflash_logprobs_grad(r, z, None, None, norm, z, group=group)
