"""Measured cases of the operators on both sides of the logit rows: rows in 8
bits with a scale each (``dflash_quant_i8``), the product of two such sets of
rows, as a vocabulary head makes logits (``dflash_linear_i8``), the log
probabilities of given tokens with a row's entropy and its largest
alternatives (``dflash_logprobs``) and their gradient (``dflash_logprobs_grad``).

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through the library's entry points.  Alternatives are ordered by value
descending, then token index ascending; a masked token is -inf.
"""

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# temperatures a serving engine mixes in one batch (a greedy request reports the unscaled distribution)
TEMPERATURES = (1.0, 0.6, 0.0, 1.5, 0.8)


def listed():
    return [
        # one token's hidden vector before the head: the smallest call
        dict(name="quant-one-token", op="quant", R=1, H=2048, dtype="bf16", pad=0),
        # a head's weights when they are loaded, a scale for each token of the vocabulary
        dict(name="quant-head-weights", op="quant", R=151936, H=2048, dtype="bf16", pad=0),
        # the logits of one token: plain decoding of one stream
        dict(name="linear-one-token", op="linear", R=1, H=2048, N=151936, dtype="bf16", pad=0),
        # the drafted positions of 32 streams
        dict(name="linear-concurrent-32", op="linear", R=256, H=2048, N=151936, dtype="bf16", pad=0),
        # the target rows of 128 streams over a large vocabulary
        dict(name="linear-large-vocab-128", op="linear", R=1152, H=4096, N=262144, dtype="bf16", pad=0),
        # odd sizes throughout, fp32 logits in padded rows
        dict(name="linear-odd-f32", op="linear", R=67, H=1003, N=50021, dtype="f32", pad=3),
        # the emitted token of one stream with the 20 alternatives a client may ask for
        dict(name="logprobs-single-stream", op="logprobs", R=1, V=151936, dtype="bf16", pad=0, M=1, N=20, T="none", entropy=False, masked=0.0),
        # every verified position of 32 streams
        dict(name="logprobs-concurrent-32", op="logprobs", R=288, V=151936, dtype="bf16", pad=0, M=1, N=20, T="mixed", entropy=True, masked=0.0),
        # a policy's forward pass over 256 blocks of 8 positions: the tokens taken and the entropy
        dict(name="logprobs-blocks", op="logprobs", R=2048, V=151936, dtype="bf16", pad=0, M=1, N=0, T="none", entropy=True, masked=0.0),
        # one stream's block: the latency of a small gradient
        dict(name="grad-one-block", op="grad", R=8, V=151936, dtype="bf16", pad=0, M=1, T="none", entropy=True, masked=0.0),
        # several given tokens a row, an odd vocabulary, padded fp32 rows, half of it masked by a grammar
        dict(name="grad-odd-f32", op="grad", R=67, V=50021, dtype="f32", pad=3, M=5, T="mixed", entropy=True, masked=0.5),
        # the same policy's backward pass
        dict(name="grad-blocks", op="grad", R=2048, V=151936, dtype="bf16", pad=0, M=1, T="none", entropy=True, masked=0.0),
    ]


# elements (quant, logprobs, grad) or products (linear) of the largest listed case of each operator: no drawn case has more
MOST = {"quant": 151936 * 2048, "linear": 1152 * 4096 * 262144, "logprobs": 2048 * 151936, "grad": 2048 * 151936}


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quant", "linear", "logprobs", "grad"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    half = 2 if dtype == "f32" else 1
    case = dict(op=op, dtype=dtype, pad=rng.choice((0, 0, 1, 5, 8)))
    if op == "quant":
        H = _spread(rng, 16, 16384)
        case.update(R=_spread(rng, 1, min(262144, MOST[op] // H // half)), H=H)
    elif op == "linear":
        H = _spread(rng, 16, 8192)
        N = _spread(rng, 16, min(262144, 262144 * 4096 // H))
        case.update(R=_spread(rng, 1, min(2048, MOST[op] // (H * N), 1152 * 262144 // N // half)), H=H, N=N)
    else:
        V = _spread(rng, 61, 262144)
        case.update(R=_spread(rng, 1, min(2048, MOST[op] // V // half)), V=V, M=_spread(rng, 1, 16),
                    T=rng.choice(("none", "none", "mixed")), entropy=rng.random() < 0.6, masked=rng.choice((0.0, 0.0, 0.5, 0.9)))
        if op == "logprobs":
            case["N"] = rng.choice((0, 0, 1, 5, 20, 32))
    return case


def _logits(gen, R, V, dtype, pad):
    """[R, V] logits: a bulk of N(0, 2) with, in three rows of four, 24 tokens
    raised by 4 to 14 as a model that knows a few continuations has them; the
    fourth row stays flat.  ``pad`` elements lie between rows."""
    z = torch.empty(R, V + pad, dtype=torch.float32, device=DEVICE).normal_(0.0, 2.0, generator=gen)
    at = torch.randint(0, V, (R, 24), device=DEVICE, generator=gen)
    up = 4.0 + 10.0 * torch.rand(R, 24, device=DEVICE, generator=gen)
    up[3::4] = 0.0
    z.scatter_add_(1, at, up)
    return z.to(TYPES[dtype])[:, :V], at


def _activations(gen, R, H, pad=0):
    """[R, H] hidden vectors: N(0, 1), one column in a hundred ten times as large."""
    x = torch.empty(R, H + pad, dtype=torch.float32, device=DEVICE).normal_(generator=gen)
    x.mul_(1.0 + 9.0 * (torch.rand(H + pad, device=DEVICE, generator=gen) < 0.01))
    return x


def _i8(gen, n, x):
    """Rows in 8 bits, 16 bytes' multiple apart, and their scales."""
    H = x.shape[1]
    scale = x.abs().amax(1) / 127.0
    q = torch.zeros(n, -(-H // 16) * 16, dtype=torch.int8, device=DEVICE)
    q[:, :H] = x.mul_(1.0 / scale[:, None]).round_().clamp_(-127, 127).to(torch.int8)
    return q[:, :H], scale


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 2 + 1)
    op, R, dtype, pad = case["op"], case["R"], case["dtype"], case["pad"]
    if op == "quant":
        H = case["H"]
        x = _activations(gen, R, H, pad).to(TYPES[dtype])[:, :H]
        if R > 4:
            x[R // 2] = 0.0  # a padded position
        return dict(op=op, x=x, q=torch.empty(R, -(-H // 16) * 16, dtype=torch.int8, device=DEVICE)[:, :H],
                    scale=torch.empty(R, dtype=torch.float32, device=DEVICE))
    if op == "linear":
        H, N = case["H"], case["N"]
        xq, xs = _i8(gen, R, _activations(gen, R, H))
        w = torch.empty(N, H, dtype=torch.float32, device=DEVICE).normal_(0.0, 0.02, generator=gen)
        w.mul_(0.5 + torch.rand(N, 1, device=DEVICE, generator=gen))
        wq, ws = _i8(gen, N, w)
        del w
        return dict(op=op, xq=xq, xs=xs, wq=wq, ws=ws, y=torch.empty(R, N + pad, dtype=TYPES[dtype], device=DEVICE)[:, :N])
    V, M = case["V"], case["M"]
    z, at = _logits(gen, R, V, dtype, pad)
    if case["masked"]:
        gone = torch.rand(R, V, device=DEVICE, generator=gen) < case["masked"]
        gone[R // 2] |= case["masked"] > 0.85  # a grammar with no way on: an empty row
        z.masked_fill_(gone, -math.inf)
        del gone
    # the first given token is a likely one, the others are any; one in fifty is padding
    tok = torch.randint(0, V, (R, M), device=DEVICE, generator=gen)
    tok[:, 0] = at[:, 0]
    tok[torch.rand(R, M, device=DEVICE, generator=gen) < 0.02] = -1
    state = dict(op=op, z=z, tok=tok.to(torch.int32), T=None, entropy=None)
    if case["T"] == "mixed":
        state["T"] = torch.tensor([TEMPERATURES[(i + int(seed)) % len(TEMPERATURES)] for i in range(R)], dtype=torch.float32, device=DEVICE)
    if op == "logprobs":
        state.update(logp=torch.empty(R, M, dtype=torch.float32, device=DEVICE), norm=torch.empty(R, 2, dtype=torch.float32, device=DEVICE),
                     top_idx=None, top_logp=None)
        if case["entropy"]:
            state["entropy"] = torch.empty(R, dtype=torch.float32, device=DEVICE)
        if case["N"]:
            state["top_idx"] = torch.empty(R, case["N"], dtype=torch.int32, device=DEVICE)
            state["top_logp"] = torch.empty(R, case["N"], dtype=torch.float32, device=DEVICE)
        return state
    # what the forward pass left for the backward, and the gradients that come in: rows of padding have none
    _, state["norm"], h = _distribution(state)
    state["g_logp"] = torch.empty(R, M, dtype=torch.float32, device=DEVICE).normal_(generator=gen)
    state["g_logp"][5::7] = 0.0
    state["g_entropy"] = None
    if case["entropy"]:
        state["entropy"] = h
        state["g_entropy"] = 0.01 + 0.1 * torch.rand(R, dtype=torch.float32, device=DEVICE, generator=gen)
        state["g_entropy"][5::7] = 0.0
    state["dz"] = torch.empty(R, V + pad, dtype=z.dtype, device=DEVICE)[:, :V]
    return state


# ---------------------------------------------------------------- plain forms

def _plain_quant(s):
    x = s["x"].float()
    scale = (x.abs().amax(1).double() / 127.0).float()
    # 64 bits: quotients next to the border between two integers
    q = torch.where(scale[:, None] > 0, x.double() / scale.double()[:, None], 0.0).round().clamp(-127.0, 127.0)
    return q.to(torch.int8), scale


def _plain_linear(s):
    acc = s["xq"].float() @ s["wq"].float().t()
    return acc.mul_(s["xs"][:, None]).mul_(s["ws"]).to(s["y"].dtype)


def _distribution(s):
    """log softmax of the rows (z - m) / T less the log of their sum, (m, that log), and the entropy."""
    z = s["z"].float()
    m = z.amax(1)
    x = z - torch.where(m > -math.inf, m, 0.0)[:, None]
    if s["T"] is not None:
        x = x / torch.where(s["T"] > 0, s["T"], 1.0)[:, None]
    e = x.exp()
    total = e.sum(1, dtype=torch.float64)  # long sums
    dot = torch.where(e > 0, e * x, 0.0).sum(1, dtype=torch.float64)
    some = total > 0
    log_sum = torch.where(some, total.log(), 0.0)
    entropy = torch.where(some, log_sum - dot / torch.where(some, total, 1.0), 0.0)
    norm = torch.stack((m, log_sum.float()), 1)
    return x.sub_(log_sum.float()[:, None]), norm, entropy.float()


def _given(logp, tok):
    inside = (tok >= 0) & (tok < logp.shape[1])
    return torch.where(inside, logp.gather(1, torch.where(inside, tok, 0).long()), 0.0), inside


def _plain_logprobs(s):
    logp, norm, entropy = _distribution(s)
    given, _ = _given(logp, s["tok"])
    out = [given, norm, entropy if s["entropy"] is not None else None, None, None]
    if s["top_idx"] is not None:
        N, V = s["top_idx"].shape[1], logp.shape[1]
        z = s["z"].float() + 0.0  # -0 as +0
        # whole numbers in the order of (value, then lower index)
        bits = z.view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (V - 1 - torch.arange(V, device=z.device))
        at = key.topk(min(N, V), dim=1).indices
        live = z.gather(1, at) > -math.inf
        out[3] = torch.full_like(s["top_idx"], -1)
        out[4] = torch.full_like(s["top_logp"], -math.inf)
        out[3][:, :min(N, V)] = torch.where(live, at, -1).int()
        out[4][:, :min(N, V)] = torch.where(live, logp.gather(1, at), -math.inf)
    return out


def _plain_grad(s):
    z = s["z"].float()
    m, log_sum = s["norm"][:, :1], s["norm"][:, 1:]
    x = z - torch.where(m > -math.inf, m, 0.0)
    scale = torch.ones_like(log_sum)
    if s["T"] is not None:
        scale = torch.where(s["T"] > 0, s["T"], 1.0)[:, None]
        x = x / scale
    logp = x - log_sum
    p = logp.exp()
    _, inside = _given(logp, s["tok"])
    inside = inside & (m > -math.inf)
    g = torch.where(inside, s["g_logp"], 0.0)
    factor = g.sum(1, keepdim=True).neg()
    if s["g_entropy"] is not None:
        factor = factor - s["g_entropy"][:, None] * (torch.where(p > 0, logp, 0.0) + s["entropy"][:, None])
    d = (p * factor).scatter_add_(1, torch.where(inside, s["tok"], 0).long(), g)
    return (d / scale).to(s["z"].dtype)


# ---------------------------------------------------------------- the library's entry points

def _own(s):
    import block_draft_select_amd as dfl
    if s["op"] == "quant":
        if "rows" not in s:
            s["rows"] = dfl.rows(s["x"])
        dfl.dflash_quant_i8(s["rows"], s["x"], s["q"], s["scale"])
        return s["q"], s["scale"]
    if s["op"] == "linear":
        if "linear" not in s:  # a program describes a product once
            s["linear"] = dfl.linear_i8(s["xq"], s["wq"], s["y"])
        dfl.dflash_linear_i8(s["linear"], s["xq"], s["xs"], s["wq"], s["ws"], s["y"])
        return s["y"]
    z = s["z"]
    if "rows" not in s:  # a program describes its rows and takes a workspace once
        s["rows"] = dfl.rows(z)
        s["work"] = dfl.rows_workspace(s["rows"], z.device)
    if s["op"] == "logprobs":
        dfl.dflash_logprobs(s["rows"], z, s["tok"], s["logp"], s["norm"], s["work"], T=s["T"], entropy=s["entropy"],
                            top_idx=s["top_idx"], top_logp=s["top_logp"])
        return [s["logp"], s["norm"], s["entropy"], s["top_idx"], s["top_logp"]]
    dfl.dflash_logprobs_grad(s["rows"], z, s["tok"], s["g_logp"], s["norm"], s["dz"], T=s["T"], entropy=s["entropy"],
                             grad_entropy=s["g_entropy"])
    return s["dz"]


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "linear": _plain_linear, "logprobs": _plain_logprobs, "grad": _plain_grad}[state["op"]](state)


def work(case):
    R, es = case["R"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quant":
        n = R * case["H"]
        return {"bytes": n * (es + 1) + 4 * R, "flops": 4 * n}
    if case["op"] == "linear":
        H, N = case["H"], case["N"]
        return {"bytes": (R + N) * (H + 4) + R * N * es, "flops": 2 * R * N * H}
    n, M = R * case["V"], case["M"]
    if case["op"] == "logprobs":
        return {"bytes": n * es + R * (8 * M + 8 * case["N"] + 12), "flops": 6 * n}
    return {"bytes": 2 * n * es + R * (8 * M + 16), "flops": 8 * n}


# ---------------------------------------------------------------- the definition in 64 bits, some rows at a time

def _exact_rows(s, lo, hi):
    """Logits over T less their largest, as float64 probabilities and their logarithms; empty rows are all -inf."""
    z = s["z"][lo:hi].double()
    if s["T"] is not None:
        t = s["T"][lo:hi].double()
        z = z / torch.where(t > 0, t, torch.ones_like(t))[:, None]
    big = z.max(1, keepdim=True).values
    empty = torch.isinf(big)
    total = torch.exp(z - big.masked_fill(empty, 0.0)).sum(1, keepdim=True)
    log_p = z - (big + torch.log(total)).masked_fill(empty, 0.0)
    return log_p, torch.exp(log_p), torch.log(total).masked_fill(empty, 0.0), empty


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        top = s["x"].double().abs().max(1).values
        return None, top / 127.0
    if case["op"] == "linear":
        x = s["xq"].double() * s["xs"].double()[:, None]
        y = torch.empty(case["R"], case["N"], dtype=torch.float64, device=x.device)
        for lo in range(0, case["N"], 32768):
            w = s["wq"][lo:lo + 32768].double() * s["ws"][lo:lo + 32768].double()[:, None]
            y[:, lo:lo + 32768] = torch.mm(x, w.t())
        return y
    z = s["z"]
    R, V = z.shape
    M = case["M"]
    rows = max(1, (1 << 26) // V)
    if case["op"] == "logprobs":
        given = torch.zeros(R, M, dtype=torch.float64, device=z.device)
        norm = torch.zeros(R, 2, dtype=torch.float64, device=z.device)
        entropy = torch.zeros(R, dtype=torch.float64, device=z.device)
        tops = torch.full((R, max(case["N"], 1)), -math.inf, dtype=torch.float64, device=z.device)
        for lo in range(0, R, rows):
            hi = min(R, lo + rows)
            log_p, p, log_total, empty = _exact_rows(s, lo, hi)
            for k in range(M):
                t = s["tok"][lo:hi, k].long()
                on = (t >= 0) & (t < V)
                v = log_p.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
                given[lo:hi, k] = torch.where(on, v, torch.zeros_like(v))
            norm[lo:hi, 0] = z[lo:hi].double().max(1).values
            norm[lo:hi, 1] = log_total[:, 0]
            entropy[lo:hi] = -torch.special.xlogy(p, p).sum(1)
            n = min(case["N"], V)
            if n:
                tops[lo:hi, :n] = torch.sort(log_p, 1, descending=True).values[:, :n]
        return [given, norm, entropy if case["entropy"] else None, None, tops if case["N"] else None]
    out = torch.zeros(R, V, dtype=torch.float64, device=z.device)
    for lo in range(0, R, rows):
        hi = min(R, lo + rows)
        log_p, p, _, empty = _exact_rows(s, lo, hi)
        d = out[lo:hi]
        for k in range(M):
            t = s["tok"][lo:hi, k].long()
            g = s["g_logp"][lo:hi, k].double() * ((t >= 0) & (t < V))
            d -= g[:, None] * p
            d.scatter_add_(1, t.clamp(0, V - 1)[:, None], g[:, None])
        if s["g_entropy"] is not None:
            neg_h = torch.special.xlogy(p, p).sum(1, keepdim=True)
            d -= s["g_entropy"][lo:hi].double()[:, None] * (torch.special.xlogy(p, p) - p * neg_h)
        if s["T"] is not None:
            t = s["T"][lo:hi].double()
            d /= torch.where(t > 0, t, torch.ones_like(t))[:, None]
        d.masked_fill_(empty, 0.0)
    return out
