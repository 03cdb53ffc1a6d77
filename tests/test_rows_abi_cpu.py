"""Refusals of the operators on logit rows, checked on the host before any
HIP call (no GPU needed), and the binding's description of row tensors."""

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


def _rows(dfl, R=3, stride=100, V=100, dtype=1):
    return dfl.dflash_rows(R, stride, V, dtype)


def _ws(dfl, r):
    n = ctypes.c_size_t(777)
    return dfl.lib.dflash_rows_workspace_bytes(ctypes.byref(r), ctypes.byref(n)), n.value


def _flt(dfl, group=1):
    return dfl.dflash_filters(None, None, None, None, group)


def _sample(dfl, r, Z=FAKE, f="on", u=FAKE, token=FAKE, ws=FAKE, n=1 << 40):
    f = _flt(dfl) if f == "on" else f
    return dfl.lib.dflash_sample(ctypes.byref(r) if r is not None else None, Z, ctypes.byref(f) if f is not None else None,
                                 u, token, None, None, ws, n, None)


def _filter(dfl, r, Z=FAKE, out=FAR, stride=100, ws=FAKE, n=1 << 40, f="on"):
    f = _flt(dfl) if f == "on" else f
    return dfl.lib.dflash_filter(ctypes.byref(r), Z, ctypes.byref(f), 0.0, out, stride, None, ws, n, None)


def _distill(dfl, r, S=FAKE, K=4, tau=1.0, idx=FAKE, t=FAKE, t_lse=None, lse=FAKE, rest=None, ws=FAKE, n=1 << 40):
    return dfl.lib.dflash_distill(ctypes.byref(r), S, K, tau, idx, t, t_lse, None, FAKE, lse, rest, ws, n, None)


def _grad(dfl, r, S=FAKE, K=4, tau=1.0, idx=FAKE, t=FAKE, t_lse=None, lse=FAKE, rest=None, dS=FAR, stride=100):
    return dfl.lib.dflash_distill_grad(ctypes.byref(r), S, K, tau, idx, t, t_lse, None, None, lse, rest, dS, stride, None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), 1), (dict(V=0), 1), (dict(V=-5), 1), (dict(dtype=2), 1), (dict(stride=99), 1), (dict(stride=-100), 1),
    (dict(R=4194305), 2), (dict(V=2097153, stride=2097153), 2), (dict(stride=(1 << 40) + 1), 2),
])
def test_bad_rows_are_refused_everywhere(dfl, kw, status):
    r = _rows(dfl, **kw)
    assert _ws(dfl, r) == (status, 777)
    assert dfl.lib.dflash_last_error() != b""
    assert _sample(dfl, r) == status
    assert _filter(dfl, r) == status
    assert _distill(dfl, r) == status
    assert _grad(dfl, r) == status


def test_limits_are_accepted(dfl):
    assert _ws(dfl, _rows(dfl, R=1, stride=2097152, V=2097152, dtype=0))[0] == 0
    assert _ws(dfl, _rows(dfl, R=4194304, stride=8, V=8))[0] == 0
    assert _ws(dfl, _rows(dfl, R=1, stride=0, V=100))[0] == 0  # one row: the stride does not matter
    assert _ws(dfl, _rows(dfl, R=4194304, stride=1 << 21, V=1 << 21))[0] == 2  # more blocks than a launch holds


def test_null_rows_and_filters(dfl):
    r = _rows(dfl)
    assert dfl.lib.dflash_rows_workspace_bytes(None, ctypes.byref(ctypes.c_size_t())) == 1
    assert dfl.lib.dflash_rows_workspace_bytes(ctypes.byref(r), None) == 1
    assert _sample(dfl, None) == 1
    assert _sample(dfl, r, f=None) == 1
    assert b"filters is NULL" in dfl.lib.dflash_last_error()
    assert _sample(dfl, r, f=_flt(dfl, 0)) == 1
    assert _filter(dfl, r, f=_flt(dfl, -3)) == 1


def test_pointers_and_workspaces(dfl):
    r = _rows(dfl)
    for kw in (dict(Z=None), dict(Z=ODD), dict(u=None), dict(token=None)):
        assert _sample(dfl, r, **kw) == 1, kw
    for kw in (dict(Z=None), dict(out=None), dict(out=ODD), dict(stride=99)):
        assert _filter(dfl, r, **kw) == 1, kw
    for kw in (dict(S=None), dict(idx=None), dict(t=None), dict(lse=None)):
        assert _distill(dfl, r, **kw) == 1, kw
        assert _grad(dfl, r, **kw) == 1, kw
    assert _grad(dfl, r, dS=None) == 1 and _grad(dfl, r, stride=10) == 1
    need = _ws(dfl, r)[1]
    for call in (_sample, _filter, _distill):
        assert call(dfl, r, ws=None) == 3
        assert call(dfl, r, ws=ctypes.c_void_p(0x10008)) == 3
    assert _sample(dfl, r, n=16) == 3 and _filter(dfl, r, n=16) == 3 and _distill(dfl, r, n=0) == 3
    assert need > 16


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("V", [1, 33, 5000, 16384, 32000, 151936, 262144, 2097152])
def test_a_workspace_serves_fewer_rows_too(dfl, dtype, V):
    # what a call asks for (its refusal says so) stays within the workspace of
    # as many rows or more
    last = 0
    for R in sorted({1, 2, 3, 7, 8, 31, 41, 42, 64, 100, 128, 195, 196, 341, 342, 512, 513, 1023, 1024, 1025, 2048, 4097}):
        r = _rows(dfl, R=R, stride=V, V=V, dtype=dtype)
        status, n = _ws(dfl, r)
        assert status == 0 and n >= last
        last = n
        for call in (_sample, _distill):
            assert call(dfl, r, n=0) == 3
            assert int(dfl.lib.dflash_last_error().split(b"need ")[1].split()[0]) <= n, (R, V)


@pytest.mark.parametrize("kw", [dict(K=-1), dict(K=1025), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
                                dict(tau=float("inf")), dict(tau=1e-40), dict(t_lse=FAKE), dict(rest=FAKE)])
def test_bad_distill_arguments(dfl, kw):
    r = _rows(dfl)
    assert _distill(dfl, r, **kw) == 1
    assert _grad(dfl, r, **kw) == 1


def test_overlapping_outputs_are_refused(dfl):
    r = _rows(dfl, R=3, stride=120, V=100)
    base = 0x100000
    at = lambda e: ctypes.c_void_p(base + 2 * e)  # noqa: E731
    for call, out in ((_filter, "out"), (_grad, "dS")):
        src = {"Z" if call is _filter else "S": at(0)}
        for e, stride in ((1, 120), (99, 120), (-50, 120), (0, 121), (119, 120), (240, 100)):
            assert call(dfl, r, **src, **{out: at(e)}, stride=stride) == 1, (e, stride)
            assert b"overlaps" in dfl.lib.dflash_last_error()


@pytest.mark.parametrize("stride", [0, 100, -7])
def test_one_rows_overlapping_output_is_refused(dfl, stride):
    # one row's stride may be anything, 0 too
    r = _rows(dfl, R=1, stride=stride, V=100)
    at = lambda e: ctypes.c_void_p(0x100000 + 2 * e)  # noqa: E731
    for call, out in ((_filter, "out"), (_grad, "dS")):
        src = {"Z" if call is _filter else "S": at(0)}
        for e in (1, 50, -99):
            for own in (stride, 100):
                assert call(dfl, r, **src, **{out: at(e)}, stride=own) == 1, (e, own)
                assert b"overlaps" in dfl.lib.dflash_last_error()


def test_empty_calls_launch_nothing(dfl):
    r = _rows(dfl, R=0)
    assert _ws(dfl, r) == (0, 0)
    nul = dict(ws=None, n=0)
    assert _sample(dfl, r, Z=None, u=None, token=None, **nul) == 0
    assert _filter(dfl, r, Z=None, out=None, **nul) == 0
    assert _distill(dfl, r, S=None, idx=None, t=None, lse=None, **nul) == 0
    assert _grad(dfl, r, S=None, idx=None, t=None, lse=None, dS=None) == 0


def test_rows_of_tensors(dfl):
    def of(t):
        r = dfl.rows(t)
        return r.R, r.stride, r.V, r.dtype
    z = torch.zeros(4, 6, 10)
    assert of(z) == (24, 10, 10, dfl.F32)
    assert of(z[:, :, :7]) == (24, 10, 7, dfl.F32)
    assert of(z[:, 2].to(torch.bfloat16)) == (4, 10, 10, dfl.BF16)
    assert of(z[:, 2]) == (4, 60, 10, dfl.F32)
    assert of(z[0, 0]) == (1, 10, 10, dfl.F32)
    assert of(z[:1]) == (6, 10, 10, dfl.F32)
    assert of(torch.zeros(0, 10)) == (0, 10, 10, dfl.F32)
    assert of(torch.zeros(5, 1)[:, :1]) == (5, 1, 1, dfl.F32)
    for bad in (z[:, :4], z.transpose(1, 2), z[..., ::2]):
        with pytest.raises(ValueError):
            dfl.rows(bad)
    with pytest.raises(TypeError):
        dfl.rows(z.half())


@pytest.mark.parametrize("group,error", [(1.5, TypeError), (9.0, TypeError), (0, ValueError), (-3, ValueError),
                                         ((1 << 32) + 1, ValueError), (1 << 31, ValueError), (None, TypeError)])
def test_groups_that_are_no_positive_int32_are_refused(dfl, group, error):
    # a group that the call rounded or wrapped would read settings behind their array
    z = torch.zeros(12, 10)
    r = dfl.rows(z)
    with pytest.raises(error, match="group|integer"):
        dfl.dflash_sample(r, z, None, None, None, group=group)
    with pytest.raises(error, match="group|integer"):
        dfl.dflash_filter(r, z, z, None, group=group)


def test_kernel_names(dfl):
    for i, n in enumerate(dfl.KERNELS):
        assert dfl.lib.dflash_kernel_name(i) == n.encode()
    assert dfl.lib.dflash_kernel_name(len(dfl.KERNELS)) == b""
