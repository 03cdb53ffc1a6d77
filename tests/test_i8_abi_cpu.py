"""Refusals of dflash_quant_i8 and dflash_linear_i8, checked on the host before
any HIP call (no GPU needed), and the binding's description of 8-bit rows."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
OFF8 = ctypes.c_void_p(0x10008)
FAR = ctypes.c_void_p(0x7000000000)
FAR2 = ctypes.c_void_p(0x6000000000)


@pytest.fixture(scope="module")
def dfl():
    import block_draft_select_amd as m
    return m


def _quant(dfl, r, X=FAKE, q=FAR, stride=112, scale=FAKE):
    return dfl.lib.dflash_quant_i8(ctypes.byref(r) if r is not None else None, X, q, stride, scale, None)


def _lin(dfl, xq=FAKE, xs=FAKE, wq=FAR2, ws=FAKE, Y=FAR, null=False, **kw):
    d = dict(R=3, xq_stride=112, wq_stride=112, y_stride=50, N=50, H=100, dtype=1)
    d.update(kw)
    d = dfl.dflash_linear(*[d[n] for n in ("R", "xq_stride", "wq_stride", "y_stride", "N", "H", "dtype")])
    return dfl.lib.dflash_linear_i8(None if null else ctypes.byref(d), xq, xs, wq, ws, Y, None)


def test_bad_quant_calls(dfl):
    r = dfl.dflash_rows(3, 100, 100, 1)
    assert _quant(dfl, None) == 1
    for kw in (dict(X=None), dict(X=ODD), dict(q=None), dict(q=OFF8), dict(stride=100), dict(stride=96), dict(stride=113), dict(stride=-112),
               dict(scale=None)):
        assert _quant(dfl, r, **kw) == 1, kw
    assert _quant(dfl, r, stride=1 << 41) == 2
    for kw, status in ((dict(R=-1), 1), (dict(V=0), 1), (dict(dtype=3), 1), (dict(R=4194305), 2), (dict(stride=50), 1)):
        d = dict(R=3, stride=100, V=100, dtype=1)
        d.update(kw)
        assert _quant(dfl, dfl.dflash_rows(d["R"], d["stride"], d["V"], d["dtype"])) == status, kw
    for at in (0x10000, 0x10000 + 500, 0x10000 - 300):
        assert _quant(dfl, r, q=ctypes.c_void_p(at // 16 * 16)) == 1
        assert b"overlaps" in dfl.lib.dflash_last_error()
    for kw in (dict(X=ctypes.c_void_p(0x50000), scale=ctypes.c_void_p(0x50000 + 596)), dict(q=ctypes.c_void_p(0x50000), scale=ctypes.c_void_p(0x50000 - 8))):
        assert _quant(dfl, r, **kw) == 1 and b"scale overlaps" in dfl.lib.dflash_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), 1), (dict(R=-1), 1), (dict(N=0), 1), (dict(H=0), 1), (dict(dtype=2), 1), (dict(R=4194305), 2),
    (dict(N=2097153, y_stride=2097153), 2), (dict(H=65537, xq_stride=65552, wq_stride=65552), 2), (dict(xq_stride=96), 1),
    (dict(xq_stride=104), 1), (dict(wq_stride=96), 1), (dict(wq_stride=120), 1), (dict(xq_stride=-112), 1), (dict(y_stride=49), 1),
    (dict(y_stride=(1 << 40) + 1), 2), (dict(xq_stride=(1 << 22) + 16), 2), (dict(wq_stride=1 << 41), 2), (dict(xq=None), 1), (dict(xs=None), 1),
    (dict(wq=None), 1), (dict(ws=None), 1), (dict(Y=None), 1), (dict(xq=OFF8), 1), (dict(wq=OFF8), 1), (dict(Y=ODD), 1),
    (dict(R=4194304, N=2097152, y_stride=2097152), 2),
])
def test_bad_products(dfl, kw, status):
    assert _lin(dfl, **kw) == status
    assert dfl.lib.dflash_last_error() != b""


def test_products_over_their_inputs_are_refused(dfl):
    base = 0x10000
    for at in (base, base + 320, base - 290):  # xq: 2 * 112 + 112 bytes; Y: 300
        assert _lin(dfl, Y=ctypes.c_void_p(at), xs=FAR2, ws=FAR2) == 1 and b"overlaps" in dfl.lib.dflash_last_error()
    assert _lin(dfl, Y=FAR2, xs=FAKE, ws=FAKE) == 1  # the weights
    assert _lin(dfl, xs=FAR, wq=FAR2) == 1 and _lin(dfl, ws=FAR) == 1


def test_empty_calls_launch_nothing(dfl):
    assert _lin(dfl, R=0, xq=None, xs=None, wq=None, ws=None, Y=None) == 0
    assert _quant(dfl, dfl.dflash_rows(0, 100, 100, 1), X=None, q=None, scale=None) == 0
    assert _lin(dfl, R=0, H=0) == 1


def test_i8_rows(dfl):
    for R, H, pitch in ((3, 100, 112), (1, 16, 16), (2, 1, 16), (0, 5, 16)):
        t = dfl.i8_rows(R, H, device="cpu")
        assert t.dtype == torch.int8 and tuple(t.shape) == (R, H) and (R < 2 or t.stride(0) == pitch)


def test_description_of_a_product(dfl):
    x, w = dfl.i8_rows(6, 100, device="cpu"), dfl.i8_rows(9, 100, device="cpu")
    d = dfl.linear_i8(x, w, torch.zeros(2, 3, 11)[:, :, :9])
    assert (d.R, d.N, d.H, d.xq_stride, d.wq_stride, d.y_stride, d.dtype) == (6, 9, 100, 112, 112, 11, dfl.F32)
    for bad in ((x, dfl.i8_rows(9, 99, device="cpu"), torch.zeros(6, 9)), (x, w, torch.zeros(6, 8)), (x, w, torch.zeros(5, 9)),
                (x[0], w, torch.zeros(1, 9))):
        with pytest.raises(ValueError):
            dfl.linear_i8(*bad)
    with pytest.raises(TypeError):
        dfl.linear_i8(x, w, torch.zeros(6, 9, dtype=torch.half))


def test_binding_refusals(dfl):
    X = torch.zeros(3, 100)
    r, s = dfl.rows(X), torch.zeros(3)
    q = dfl.i8_rows(3, 100, device="cpu")
    with pytest.raises(TypeError):
        dfl.dflash_quant_i8(r, X, q.short(), s)
    with pytest.raises(ValueError, match="shape"):
        dfl.dflash_quant_i8(r, X, q[:2], s)
    with pytest.raises(ValueError, match="adjacent"):
        dfl.dflash_quant_i8(r, X, torch.zeros(100, 3, dtype=torch.int8).t(), s)
    with pytest.raises(ValueError, match="device tensor"):
        dfl.dflash_quant_i8(r, X, q, s)
    # rows whose last one does not own the bytes up to a multiple of 16: the check
    # comes after that of the device, so it is called by itself
    with pytest.raises(ValueError, match="multiple of 16"):
        dfl._i8(torch.zeros(1, 100, dtype=torch.int8), "q", 1, 100, _Cpu())
    assert dfl._i8(q, "q", 3, 100, _Cpu())[1] == 112


class _Cpu:
    index = -1  # what get_device() says of a CPU tensor
