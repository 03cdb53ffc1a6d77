"""Refusals of dflash_quant_i8, dflash_linear_i8, dflash_logprobs and
dflash_logprobs_grad, each by the check that it is meant for: every array has an
address of its own, far from the others', and the error's text is compared, so
that no other check can stand in.  All of it happens on the host before any HIP
call (no GPU needed).
"""

import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def at(n, off=0):
    """The n-th address, 2^40 bytes from its neighbours, `off` bytes behind it."""
    return ctypes.c_void_p((n + 1 << 40) + off)


Z, TOK, LOGP, NORM, ENT, TOP, TOP_LOGP, WS, T, GE, DZ = (at(i) for i in range(11))
X, Q, SCALE = (at(i) for i in range(3))
XQ, XS, WQ, WSC, Y = (at(i) for i in range(5))


@pytest.fixture(scope="module")
def dfl():
    import block_draft_select_amd as m
    return m


def refused(dfl, status, want, text):
    assert status == want, (status, dfl.lib.dflash_last_error())
    assert text in dfl.lib.dflash_last_error().decode(), dfl.lib.dflash_last_error()


def rows_(dfl, R=3, stride=None, V=151936, dtype=1):  # few long rows: a call with a workspace
    return dfl.dflash_rows(R, V if stride is None else stride, V, dtype)


def fwd(dfl, r, **kw):
    a = dict(Z=Z, T=T, group=1, M=2, tok=TOK, logp=LOGP, norm=NORM, ent=ENT, N=3, top=TOP, top_logp=TOP_LOGP, ws=WS, n=1 << 30)
    a.update(kw)
    return dfl.lib.dflash_logprobs(ctypes.byref(r) if r is not None else None, *a.values(), None)


def grad(dfl, r, **kw):
    a = dict(Z=Z, T=T, group=1, M=2, tok=TOK, g=LOGP, ge=GE, norm=NORM, ent=ENT, dZ=DZ, stride=151936)
    a.update(kw)
    return dfl.lib.dflash_logprobs_grad(ctypes.byref(r) if r is not None else None, *a.values(), None)


def quant(dfl, r, **kw):
    a = dict(X=X, q=Q, stride=112, scale=SCALE)
    a.update(kw)
    return dfl.lib.dflash_quant_i8(ctypes.byref(r) if r is not None else None, *a.values(), None)


def linear(dfl, null=False, **kw):
    d = dict(R=3, xq_stride=112, wq_stride=112, y_stride=50, N=50, H=100, dtype=1)
    a = dict(xq=XQ, xs=XS, wq=WQ, ws=WSC, Y=Y)
    d.update({k: v for k, v in kw.items() if k in d})
    a.update({k: v for k, v in kw.items() if k in a})
    d = dfl.dflash_linear(*d.values())
    return dfl.lib.dflash_linear_i8(None if null else ctypes.byref(d), *a.values(), None)


BAD_ROWS = [(dict(R=-1), INVALID, "R must not be negative"), (dict(V=0), INVALID, "V must be >= 1"), (dict(dtype=2), INVALID, "unknown dtype"),
            (dict(stride=151935), INVALID, "stride must be at least V"), (dict(R=4194305), UNSUPPORTED, "R above DFLASH_ROWS_MAX"),
            (dict(V=2097153), UNSUPPORTED, "V above DFLASH_V_MAX"), (dict(stride=(1 << 40) + 1), UNSUPPORTED, "stride above 2^40"),
            (dict(R=4194304, V=1 << 21), UNSUPPORTED, "too large for one launch")]


@pytest.mark.parametrize("kw,status,text", BAD_ROWS)
def test_rows(dfl, kw, status, text):
    r = rows_(dfl, **kw)
    refused(dfl, fwd(dfl, r), status, text)
    refused(dfl, grad(dfl, r, stride=max(r.V, 1)), status, text)
    refused(dfl, quant(dfl, r, stride=1 << 22), status, text)


def test_no_rows(dfl):
    refused(dfl, fwd(dfl, None), INVALID, "rows is NULL")
    refused(dfl, grad(dfl, None), INVALID, "rows is NULL")
    refused(dfl, quant(dfl, None), INVALID, "rows is NULL")


FORWARD = [(dict(group=0), "group must be"), (dict(group=-2), "group must be"), (dict(M=-1), "M must be in"), (dict(M=1025), "M must be in"),
           (dict(Z=None), "Z is NULL"), (dict(Z=at(0, 1)), "Z is not aligned"), (dict(tok=None), "tok is NULL"), (dict(logp=None), "logp is NULL"),
           (dict(norm=None), "norm is NULL"), (dict(N=-1), "N must be in"), (dict(N=33), "N must be in"), (dict(top=None), "top_idx is NULL"),
           (dict(top_logp=None), "top_logp is NULL")]


@pytest.mark.parametrize("kw,text", FORWARD)
def test_forward(dfl, kw, text):
    refused(dfl, fwd(dfl, rows_(dfl), **kw), INVALID, text)


def test_the_other_arguments_pass(dfl):
    # the workspace is looked at last but for overlaps: what comes before it is in order
    for kw in (dict(), dict(T=None), dict(ent=None), dict(M=0, tok=None, logp=None), dict(N=0, top=None, top_logp=None), dict(Z=at(0, 2)),
               dict(M=1024), dict(N=32), dict(group=1 << 30)):
        refused(dfl, fwd(dfl, rows_(dfl), ws=None, **kw), WORKSPACE, "workspace is NULL")
    refused(dfl, fwd(dfl, rows_(dfl), ws=at(7, 8)), WORKSPACE, "not 16-byte aligned")
    refused(dfl, fwd(dfl, rows_(dfl), n=16), WORKSPACE, "too small")


@pytest.mark.parametrize("name,bytes_", [("logp", 24), ("norm", 24), ("ent", 12), ("top", 36), ("top_logp", 36)])
def test_outputs_over_the_rows(dfl, name, bytes_):
    last = 2 * 3 * 151936 - 2  # of the rows
    for off in (0, last // 4 * 4, 4 - bytes_):
        refused(dfl, fwd(dfl, rows_(dfl), **{name: at(0, off)}), INVALID, "an output overlaps Z")


GRADIENT = [(dict(group=0), INVALID, "group must be"), (dict(M=-1), INVALID, "M must be in"), (dict(M=1025), INVALID, "M must be in"),
            (dict(Z=None), INVALID, "Z is NULL"), (dict(Z=at(0, 1)), INVALID, "Z is not aligned"), (dict(tok=None), INVALID, "tok is NULL"),
            (dict(g=None), INVALID, "grad_logp is NULL"), (dict(norm=None), INVALID, "norm is NULL"),
            (dict(ent=None), INVALID, "grad_entropy needs entropy"), (dict(dZ=None), INVALID, "dZ is NULL"),
            (dict(dZ=at(10, 1)), INVALID, "dZ is not aligned"), (dict(stride=151935), INVALID, "dZ's stride must be at least V"),
            (dict(stride=(1 << 40) + 1), UNSUPPORTED, "dZ's stride is above")]


@pytest.mark.parametrize("kw,status,text", GRADIENT)
def test_gradient(dfl, kw, status, text):
    refused(dfl, grad(dfl, rows_(dfl), **kw), status, text)


@pytest.mark.parametrize("name,bytes_", [("T", 12), ("tok", 24), ("g", 24), ("ge", 12), ("norm", 24), ("ent", 12)])
def test_gradients_over_inputs(dfl, name, bytes_):
    last = 2 * 3 * 151936 - 2
    for off in (0, last // 4 * 4, 4 - bytes_):
        refused(dfl, grad(dfl, rows_(dfl), **{name: at(10, off)}), INVALID, "dZ overlaps an input")
    refused(dfl, grad(dfl, rows_(dfl), dZ=at(0, 2)), INVALID, "dZ overlaps its input")


QUANT = [(dict(X=None), INVALID, "X is NULL"), (dict(X=at(0, 1)), INVALID, "X is not aligned"), (dict(q=None), INVALID, "q is NULL"),
         (dict(q=at(1, 8)), INVALID, "q is not 16-byte aligned"), (dict(stride=96), INVALID, "q's stride must be"),
         (dict(stride=104), INVALID, "q's stride must be"), (dict(stride=-112), INVALID, "q's stride must be"),
         (dict(stride=(1 << 22) + 16), UNSUPPORTED, "q's stride is above"), (dict(scale=None), INVALID, "scale is NULL"),
         (dict(q=at(0, 592)), INVALID, "q overlaps X"), (dict(q=at(0, -320)), INVALID, "q overlaps X"),
         (dict(scale=at(0, 596)), INVALID, "scale overlaps"), (dict(scale=at(0, -8)), INVALID, "scale overlaps"),
         (dict(scale=at(1, 320)), INVALID, "scale overlaps"), (dict(scale=at(1, -8)), INVALID, "scale overlaps")]


@pytest.mark.parametrize("kw,status,text", QUANT)
def test_quant(dfl, kw, status, text):
    refused(dfl, quant(dfl, rows_(dfl, V=100), **kw), status, text)  # 3 rows of 200 bytes, 112 apart in 8 bits


LINEAR = [(dict(null=True), INVALID, "linear is NULL"), (dict(R=-1), INVALID, "R must not be negative"), (dict(N=0), INVALID, "N must be >= 1"),
          (dict(H=0), INVALID, "H must be >= 1"), (dict(dtype=2), INVALID, "unknown dtype"), (dict(R=4194305), UNSUPPORTED, "R above"),
          (dict(N=2097153, y_stride=2097153), UNSUPPORTED, "N above"), (dict(H=65537, xq_stride=65552, wq_stride=65552), UNSUPPORTED, "H above"),
          (dict(y_stride=49), INVALID, "Y's stride must be"), (dict(y_stride=(1 << 40) + 1), UNSUPPORTED, "Y's stride is above"),
          (dict(R=4194304, N=2097152, y_stride=2097152), UNSUPPORTED, "too large for one launch"),
          (dict(xq_stride=96), INVALID, "xq's stride must be"), (dict(xq_stride=104), INVALID, "xq's stride must be"),
          (dict(xq_stride=-112), INVALID, "xq's stride must be"), (dict(xq_stride=(1 << 22) + 16), UNSUPPORTED, "xq's stride is above"),
          (dict(wq_stride=96), INVALID, "wq's stride must be"), (dict(wq_stride=120), INVALID, "wq's stride must be"),
          (dict(wq_stride=1 << 41), UNSUPPORTED, "wq's stride is above"),
          (dict(xq=None), INVALID, "xq is NULL"), (dict(xq=at(0, 8)), INVALID, "xq is not 16-byte aligned"), (dict(xs=None), INVALID, "xs is NULL"),
          (dict(wq=None), INVALID, "wq is NULL"), (dict(wq=at(2, 8)), INVALID, "wq is not 16-byte aligned"), (dict(ws=None), INVALID, "ws is NULL"),
          (dict(Y=None), INVALID, "Y is NULL"), (dict(Y=at(4, 1)), INVALID, "Y is not aligned"),
          (dict(Y=at(4, 2), dtype=0), INVALID, "Y is not aligned")]
# Y of 300 bytes over xq (3 rows, 336 bytes), wq (50, 5600), xs (12) and ws (200)
LINEAR += [(dict(Y=at(n, off)), INVALID, "Y overlaps an input") for n, size in ((0, 336), (2, 5600), (1, 12), (3, 200)) for off in (0, size - 2, -298)]


@pytest.mark.parametrize("kw,status,text", LINEAR)
def test_linear(dfl, kw, status, text):
    refused(dfl, linear(dfl, **kw), status, text)


def test_binding(dfl):
    z, r = torch.zeros(4, 10), dfl.rows(torch.zeros(4, 10))
    tok, lp, norm, ws = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 2), torch.zeros(64, dtype=torch.uint8)
    for a, b in ((tok, None), (None, lp), (tok, torch.zeros(4, 3)), (tok[0, 0], lp[0, 0])):
        with pytest.raises(ValueError, match="tok and logp must be given together"):
            dfl.dflash_logprobs(r, z, a, b, norm, ws)
        with pytest.raises(ValueError, match="tok and grad_logp must be given together"):
            dfl.dflash_logprobs_grad(r, z, a, b, norm, z)
    for a, b in ((tok, None), (None, lp), (tok, torch.zeros(4, 3))):
        with pytest.raises(ValueError, match="top_idx and top_logp must be given together"):
            dfl.dflash_logprobs(r, z, None, None, norm, ws, top_idx=a, top_logp=b)
    for group, error, text in ((0, ValueError, "group must lie"), (1 << 31, ValueError, "group must lie"), (1.0, TypeError, "integer")):
        with pytest.raises(error, match=text):
            dfl.dflash_logprobs(r, z, None, None, norm, ws, group=group)
        with pytest.raises(error, match=text):
            dfl.dflash_logprobs_grad(r, z, None, None, norm, z, group=group)


class _Cpu:
    """A device whose tensors are the host's, so that the checks behind that of the device are reached."""
    index = -1


def test_binding_arrays(dfl):
    # the helpers that every array goes through, by themselves
    v = torch.zeros(8)
    assert dfl._vec(v, "v", torch.float32, 8, _Cpu()) == v.data_ptr() and dfl._vec(None, "v", torch.float32, 8, _Cpu(), True) is None
    with pytest.raises(ValueError, match="tok and logp must be given together"):
        dfl._given(dfl.rows(torch.zeros(4, 10)), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(2, 4), "logp", _Cpu())
    r = dfl.rows(torch.zeros(4, 10))
    for shape, M in (((4, 2), 2), ((4,), 1), ((4, 1), 1), ((4, 0), 0), ((2, 2, 3), 3)):
        assert dfl._given(r, torch.zeros(shape, dtype=torch.int32), torch.zeros(shape), "logp", _Cpu())[0] == M
    z = torch.zeros(4, 10)
    assert dfl._row_tensor(z, "Z", r, _Cpu(), r.stride) == (z.data_ptr(), 10)
    with pytest.raises(ValueError, match="must hold 4 rows of 10"):
        dfl._row_tensor(torch.zeros(4, 9), "Z", r, _Cpu())
    with pytest.raises(ValueError, match="must hold 4 rows of 10"):
        dfl._row_tensor(z.bfloat16(), "Z", r, _Cpu())
    with pytest.raises(ValueError, match="row stride 10, got 12"):
        dfl._row_tensor(torch.zeros(4, 12)[:, :10], "Z", r, _Cpu(), r.stride)
    with pytest.raises(ValueError, match="device tensor"):
        dfl._row_tensor(z, "Z", r, torch.device("cuda:0"))
    q = dfl.i8_rows(3, 100, device="cpu")
    assert dfl._i8(q, "q", 3, 100, _Cpu()) == (q.data_ptr(), 112)
    with pytest.raises(ValueError, match="row stride 128, got 112"):
        dfl._i8(q, "q", 3, 100, _Cpu(), 128)
    with pytest.raises(ValueError, match="shape"):
        dfl._i8(q, "q", 2, 100, _Cpu())
    with pytest.raises(ValueError, match="adjacent"):
        dfl._i8(torch.zeros(100, 3, dtype=torch.int8).t(), "q", 3, 100, _Cpu())
    with pytest.raises(TypeError, match="int8"):
        dfl._i8(q.short(), "q", 3, 100, _Cpu())
