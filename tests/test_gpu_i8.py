"""GPU parity of dflash_quant_i8 and dflash_linear_i8 with oracle.i8.

Bars: none.  The 8-bit values, scales and products are defined to the last
bit: sums are whole numbers, each later step is one fp32 operation, and the
result is rounded once to its type.
"""

import sys

import numpy as np
import pytest

from oracle import i8 as O

pytestmark = pytest.mark.gpu


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_select_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def _type(name):
    import torch
    return dict(bf16=torch.bfloat16, f32=torch.float32)[name]


def i8_tensor(a, gap=0):
    """An int8 [R, H] tensor on the GPU in 8-bit rows, `gap` more bytes between them, the bytes behind H of any value."""
    import torch
    R, H = a.shape
    pitch = -(-H // 16) * 16 + gap
    full = torch.randint(-128, 128, (R, pitch), dtype=torch.int8, device="cuda")
    full[:, :H] = torch.from_numpy(a.astype(np.int8)).cuda()
    return full[:, :H]


def check_quant(x, dt, pad=0, shift=0, gap=0, rows_=None):
    import torch
    import block_draft_select_amd as dfl
    R, H = x.shape
    flat = torch.full((R * (H + pad) + shift + 8,), 1e30, dtype=_type(dt), device="cuda")
    v = flat[shift:shift + R * (H + pad)].view(R, H + pad)[:, :H]
    v.copy_(torch.from_numpy(x).to(v.dtype))
    pitch = -(-H // 16) * 16 + gap
    full = torch.full((R, pitch), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((R,), 7.0, dtype=torch.float32, device="cuda")
    dfl.dflash_quant_i8(dfl.rows(v), v, full[:, :H], scale)
    torch.cuda.synchronize()
    q, s, xs = full.cpu().numpy(), scale.cpu().numpy(), v.float().cpu().numpy()
    assert (q[:, H:] == 99).all()  # what lies between rows stays
    for i in range(R) if rows_ is None else rows_:
        wq, wsc = O.quantise(xs[i])
        assert s[i] == wsc or (np.isnan(s[i]) and np.isnan(wsc)), (i, s[i], wsc)
        bad = q[i, :H] != wq
        assert not bad.any(), (i, int(bad.argmax()), xs[i][bad][:3], q[i, :H][bad][:3], wq[bad][:3])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 3, 8, 15, 16, 17, 255, 512, 1003, 1024, 2048, 2049, 4096, 5000, 8192, 16384, 16389, 40000])
def test_quant(dt, H):
    rng = np.random.default_rng(H)
    x = rng.normal(size=(7, H)).astype(np.float32) * np.exp(rng.normal(size=(7, 1))).astype(np.float32)
    x[2] = 0.0
    x[3, H // 2] *= 100
    x[4, H - 1] = np.nan
    x[5, 0] = -np.inf
    x[6] = np.round(x[6] * 8) / 16  # multiples of one step: quotients on the middle
    _say(f"[i8] quant {dt} H={H}")
    check_quant(x, dt, pad=H % 3, shift=H % 5, gap=16 * (H % 2))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quant_middles_and_ends_of_the_range(dt):
    rng = np.random.default_rng(1)
    rows = []
    for e in (-140, -126, -100, -62, -60, -40, 0, 40, 110):
        for top in (127.0, 126.5, 100.0, 1.0):
            k = rng.integers(-253, 254, size=400) * 0.5
            k[0] = top
            k = np.clip(k, -top, top)
            with np.errstate(under="ignore"):
                rows.append((k * 2.0 ** e).astype(np.float32))
    big = rng.normal(size=400).astype(np.float32)
    big[0] = 3.3895313892515355e38
    rows += [big, big * np.float32(1e30), np.full(400, 1.4e-45, np.float32), np.arange(400, dtype=np.float32) * np.float32(1.4e-45)]
    check_quant(np.stack(rows), dt)


def test_quant_near_middles():
    # quotients within a few steps of fp32 of k + 1/2, for scales that are no power of two
    rng = np.random.default_rng(2)
    x = np.zeros((64, 2000), np.float32)
    for i in range(64):
        a = np.float32(np.exp(rng.normal() * 3))
        s = np.float64(np.float32(np.float64(a) / 127.0))
        mid = ((rng.integers(-127, 126, size=1999) + 0.5) * s).astype(np.float32)
        x[i, 1:] = (mid.view(np.int32) + rng.integers(-2, 3, size=1999).astype(np.int32)).view(np.float32)
        x[i, 1:] = np.clip(x[i, 1:], -a, a)
        x[i, 0] = a
    check_quant(x, "f32")


def test_quant_many_rows():
    rng = np.random.default_rng(3)
    x = np.tile(rng.normal(size=(50, 264)).astype(np.float32), (2000, 1))
    check_quant(x, "bf16", rows_=list(range(60)) + [50000, 99999])


def check_linear(R, N, H, dt, seed=0, gaps=(0, 0), pad=0, shift=0, full=False, scales=None):
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(seed)
    lo = -128 if full else -127
    xq, wq = rng.integers(lo, 128, size=(R, H)), rng.integers(lo, 128, size=(N, H))
    if full:
        xq[0], wq[0] = -128, -128  # the largest sum
    xs, ws = scales if scales else (np.exp(rng.normal(size=R)) * 0.01, np.exp(rng.normal(size=N)) * 0.01)
    xs, ws = xs.astype(np.float32), ws.astype(np.float32)
    flat = torch.full((R * (N + pad) + shift + 8,), 777.0, dtype=_type(dt), device="cuda")
    rowsv = flat[shift:shift + R * (N + pad)].view(R, N + pad)
    y = rowsv[:, :N]
    tx, tw = i8_tensor(xq, gaps[0]), i8_tensor(wq, gaps[1])
    d = dfl.linear_i8(tx, tw, y)
    dfl.dflash_linear_i8(d, tx, torch.from_numpy(xs).cuda(), tw, torch.from_numpy(ws).cuda(), y)
    torch.cuda.synchronize()
    assert bool((flat[:shift] == 777.0).all()) and bool((rowsv[:, N:] == 777.0).all()) and bool((flat[shift + R * (N + pad):] == 777.0).all())
    want = O.product(xq, xs, wq, ws)
    want = O.to_bf16(want) if dt == "bf16" else want
    got = y.float().cpu().numpy()
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (R, N, H, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 15, 16, 17, 63, 64, 65, 127, 128, 200, 256, 1003, 2048, 4097])
@pytest.mark.parametrize("R,N", [(1, 1), (1, 333), (16, 48), (17, 100), (33, 50), (70, 130), (129, 257), (300, 200)])
def test_linear(dt, R, N, H):
    _say(f"[i8] linear {dt} {R} x {N} x {H}")
    check_linear(R, N, H, dt, seed=R + N + H, gaps=(16 * (H % 2), 16 * (N % 2)), pad=N % 3, shift=R % 4)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,N,H", [(1, 5003, 2048), (8, 5003, 2048), (64, 5003, 1024), (256, 4096, 512), (257, 4099, 512), (512, 2048, 2048),
                                   (1152, 3001, 640), (2048, 512, 1024), (4, 40, 65536)])
def test_linear_sizes(dt, R, N, H):
    _say(f"[i8] linear {dt} {R} x {N} x {H}")
    check_linear(R, N, H, dt, seed=R, full=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,N,H", [(1, 16400, 200), (1, 70001, 63), (5, 16999, 4097), (16, 16385, 8192), (17, 20001, 1003), (32, 16384, 2048),
                                   (33, 30011, 129), (40, 16417, 1000), (64, 17000, 2048), (64, 140000, 16)])
def test_linear_few_tokens_many_channels(dt, R, N, H):
    _say(f"[i8] linear {dt} {R} x {N} x {H}")
    check_linear(R, N, H, dt, seed=R + N, gaps=(16 * (H % 2), 16 * (N % 2)), pad=N % 3, shift=R % 4)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,N,H,pitch", [(1, 17000, 4001, 4096), (20, 40000, 4096, 4096), (40, 16500, 900, 4096), (64, 5003, 4001, 4096),
                                         (200, 9001, 4001, 4096), (256, 17001, 4096, 4096), (512, 4999, 4001, 4096), (64, 9000, 8100, 8192),
                                         (130, 20011, 100, 4096)])
def test_weights_a_multiple_of_4096_apart(dt, R, N, H, pitch):
    # blocks begin in other places of k there
    _say(f"[i8] linear {dt} {R} x {N} x {H}, weights {pitch} apart")
    check_linear(R, N, H, dt, seed=R + N, gaps=(16, pitch - -(-H // 16) * 16), pad=N % 3)


def test_linear_special_scales():
    R, N = 20, 40
    xs, ws = np.ones(R), np.ones(N)
    xs[3], xs[4], xs[5] = np.nan, 0.0, 3e38
    ws[7], ws[8], ws[9] = np.inf, 1e-42, 3e38
    for dt in ("bf16", "f32"):
        check_linear(R, N, 100, dt, scales=(xs, ws))


@pytest.mark.parametrize("R,N", [(1, 48), (20, 300), (130, 1000), (300, 2000)])
def test_the_longest_rows(R, N):
    # sums of 65536 products of -128 and -128 stay below 2^31
    _say(f"[i8] linear f32 {R} x {N} x 65536")
    check_linear(R, N, 65536, "f32", seed=R, full=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,N,H,strides", [
    (9, 100, 100, (112, 112, 1 << 28)), (9, 16400, 100, (112, 112, 1 << 28)), (300, 300, 64, (64, 64, 1 << 23)),
    (530, 600, 200, (1 << 22, 1 << 22, 600)), (20, 600, 200, (1 << 22, 1 << 22, 600)), (20, 16400, 200, (1 << 22, 1 << 18, 16401))])
def test_products_beyond_32_bit_offsets(dt, R, N, H, strides):
    # the last rows of the result, of the tokens or of the weights begin 2^31 elements and more behind the first
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(R + N)
    xq, wq = rng.integers(-127, 128, size=(R, H)), rng.integers(-127, 128, size=(N, H))
    pitch = -(-H // 16) * 16
    xs, ws = np.exp(rng.normal(size=R)).astype(np.float32), np.exp(rng.normal(size=N)).astype(np.float32)

    def far(rows, stride, width, a, dtype):
        t = torch.empty((rows - 1) * stride + width, dtype=dtype, device="cuda").as_strided((rows, a.shape[1]), (stride, 1))
        t.copy_(torch.from_numpy(a).to(dtype))
        return t

    tx, tw = far(R, strides[0], pitch, xq, torch.int8), far(N, strides[1], pitch, wq, torch.int8)
    y = far(R, strides[2], N, np.full((R, N), 777.0), _type(dt))
    _say(f"[i8] linear {dt} {R} x {N} x {H}, rows {strides} apart")
    dfl.dflash_linear_i8(dfl.linear_i8(tx, tw, y), tx, torch.from_numpy(xs).cuda(), tw, torch.from_numpy(ws).cuda(), y)
    torch.cuda.synchronize()
    want = O.product(xq, xs, wq, ws)
    assert np.array_equal(y.float().cpu().numpy(), O.to_bf16(want) if dt == "bf16" else want)


def test_quant_beyond_32_bit_offsets():
    import torch
    import block_draft_select_amd as dfl
    R, H = 20, 1003
    rng = np.random.default_rng(8)
    x = torch.empty((R - 1) * (1 << 27) + H, dtype=torch.bfloat16, device="cuda").as_strided((R, H), (1 << 27, 1))
    x.copy_(torch.from_numpy(rng.normal(size=(R, H))).to(x.dtype))
    near, q, qn = x.contiguous(), dfl.i8_rows(R, H), dfl.i8_rows(R, H)
    s, sn = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    dfl.dflash_quant_i8(dfl.rows(x), x, q, s)
    dfl.dflash_quant_i8(dfl.rows(near), near, qn, sn)
    far = torch.empty(2000 * (1 << 21), dtype=torch.int8, device="cuda").view(2000, 1 << 21)[:, :H]
    many = near.repeat(100, 1)
    sm = torch.empty(2000, device="cuda")
    dfl.dflash_quant_i8(dfl.rows(many), many, far, sm)
    torch.cuda.synchronize()
    assert torch.equal(q, qn) and torch.equal(s, sn)
    assert torch.equal(far, qn.repeat(100, 1)) and torch.equal(sm, sn.repeat(100))


@pytest.mark.parametrize("R,N,H", [(3, 400, 300), (5, 40000, 300), (40, 20000, 1000), (300, 3000, 500)])
def test_products_on_two_streams_and_in_a_graph(R, N, H):
    import torch
    import block_draft_select_amd as dfl
    ins = []
    for k in range(2):
        x, w = dfl.i8_rows(R, H), dfl.i8_rows(N, H)
        h, m = torch.randn(R, H, device="cuda").bfloat16(), torch.randn(N, H, device="cuda").bfloat16()
        xs, ws, y = torch.empty(R, device="cuda"), torch.empty(N, device="cuda"), torch.empty(R, N, device="cuda")
        ins.append((h, m, x, xs, w, ws, y))

    def step(i):
        h, m, x, xs, w, ws, y = i
        dfl.dflash_quant_i8(dfl.rows(h), h, x, xs)
        dfl.dflash_quant_i8(dfl.rows(m), m, w, ws)
        dfl.dflash_linear_i8(dfl.linear_i8(x, w, y), x, xs, w, ws, y)

    wants = []
    for i in ins:
        step(i)
        torch.cuda.synchronize()
        wants.append(i[-1].clone())
        q = [[O.quantise(r) for r in t.float().cpu().numpy()] for t in (i[0], i[1][:50])]
        want = O.product(*[np.stack([a[j] for a in b]) if j == 0 else np.array([a[j] for a in b]) for b in q for j in (0, 1)])
        assert np.array_equal(i[-1][:, :50].cpu().numpy(), want)
        i[-1].zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                step(ins[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(ins[k][-1], wants[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ins[0])
    for k in range(4):
        ins[0][0].copy_(torch.randn(R, H, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = ins[0][-1].clone()
        step(ins[0])
        torch.cuda.synchronize()
        assert torch.equal(got, ins[0][-1])


def test_empty_product():
    import torch
    import block_draft_select_amd as dfl
    x, w = dfl.i8_rows(0, 100), dfl.i8_rows(5, 100)
    y = torch.empty(0, 5, device="cuda")
    dfl.dflash_linear_i8(dfl.linear_i8(x, w, y), x, torch.empty(0, device="cuda"), w, torch.ones(5, device="cuda"), y)
    torch.cuda.synchronize()


def test_hidden_vectors_to_log_probabilities():
    """As a program runs them: hidden vectors in 8 bits, the head's product, and
    what the head's rows say; against float64 from the 8-bit values."""
    import torch
    import block_draft_select_amd as dfl
    from oracle import rows as RO
    torch.manual_seed(5)
    B, L, H, V = 3, 8, 256, 5003
    h = torch.randn(B, L, H, device="cuda").bfloat16()
    w = torch.randn(V, H, device="cuda").bfloat16() * 0.1
    r_h, r_w = dfl.rows(h), dfl.rows(w)
    xq, wq = dfl.i8_rows(B * L, H), dfl.i8_rows(V, H)
    xs, ws = torch.empty(B * L, device="cuda"), torch.empty(V, device="cuda")
    U = torch.empty(B, L, V, dtype=torch.bfloat16, device="cuda")
    r = dfl.rows(U)
    d = dfl.linear_i8(xq, wq, U)
    work = dfl.rows_workspace(r)
    tok = torch.full((B * L,), -1, dtype=torch.int32, device="cuda")
    u = torch.rand(B * L, dtype=torch.float64, device="cuda")
    logp, norm, ent = torch.empty(B * L, device="cuda"), torch.empty(B * L, 2, device="cuda"), torch.empty(B * L, device="cuda")
    top, top_logp = torch.empty(B * L, 5, dtype=torch.int32, device="cuda"), torch.empty(B * L, 5, device="cuda")

    def step():
        dfl.dflash_quant_i8(r_h, h, xq, xs)
        dfl.dflash_quant_i8(r_w, w, wq, ws)
        dfl.dflash_linear_i8(d, xq, xs, wq, ws, U)
        dfl.dflash_sample(r, U, u, tok, work)
        dfl.dflash_logprobs(r, U, tok, logp, norm, work, entropy=ent, top_idx=top, top_logp=top_logp)

    step()
    torch.cuda.synchronize()
    hq = [O.quantise(x) for x in h.view(-1, H).float().cpu().numpy()]
    hw = [O.quantise(x) for x in w.float().cpu().numpy()]
    want = O.to_bf16(O.product(np.stack([q for q, _ in hq]), np.array([s for _, s in hq]), np.stack([q for q, _ in hw]),
                               np.array([s for _, s in hw])))
    assert np.array_equal(U.view(-1, V).float().cpu().numpy(), want)
    # l is below 9 and E|t| below 13: 9 2^-24 + 13 ln2 1.5 2^-24 + 12 2^-24 < 4e-6, eleven times the second for the entropy
    for i in range(B * L):
        o = RO.logprobs(want[i], [int(tok[i])], 5)
        assert 0 <= int(tok[i]) < V and top[i].tolist() == o["top_idx"].tolist()
        assert abs(float(logp[i]) - o["logp"][0]) < 4e-6 and abs(float(ent[i]) - o["entropy"]) < 4e-5
        assert np.allclose(top_logp[i].cpu().numpy(), o["top_logp"], atol=4e-6)
    # the same steps captured, replayed with eager work between
    eager = [t.clone() for t in (U, tok, logp, norm, ent, top, top_logp)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (U, logp, norm, ent, top_logp):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (U, tok, logp, norm, ent, top, top_logp)):
            assert torch.equal(a, b)
