"""Measured cases of the operators on rows of vocabulary logits: sampling
under filters (``dflash_sample``), filtered rows (``dflash_filter``),
distillation from a teacher's top logits (``dflash_distill``) and its gradient
(``dflash_distill_grad``).

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through the library's entry points.  The sampling order is by value
descending, then token index ascending; a masked token is -inf.
"""

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
FILL = -16384.0  # written in place of a removed logit: e^FILL is 0 next to any kept one

# request settings a serving engine mixes in one batch: (T, top_k, top_p, min_p);
# 0 and 1 turn a filter off, T = 0 is greedy
REQUESTS = {
    "mixed": ((1.0, 50, 0.95, 0.0), (0.6, 20, 0.9, 0.05), (0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.8, 0, 1.0, 0.1)),
    "top-k": ((1.0, 50, 1.0, 0.0), (0.6, 20, 1.0, 0.0), (1.0, 1000, 1.0, 0.0)),
    "top-p": ((1.0, 0, 0.9, 0.0), (0.6, 0, 0.95, 0.0)),
    "min-p": ((1.0, 0, 1.0, 0.1), (1.5, 0, 1.0, 0.02)),
    "temperature": ((1.0, 0, 1.0, 0.0), (0.6, 0, 1.0, 0.0)),
}


def listed():
    return [
        # the smallest call: one row of the tiny workload, all filters on
        dict(name="sample-tiny", op="sample", R=1, V=1024, dtype="f32", pad=0, requests="mixed", masked=0.0),
        # the first token of one stream after its prompt
        dict(name="sample-single-stream", op="sample", R=1, V=151936, dtype="bf16", pad=0, requests="top-p", masked=0.0),
        # the first tokens of 32 streams with different settings
        dict(name="sample-concurrent-32", op="sample", R=32, V=151936, dtype="bf16", pad=0, requests="mixed", masked=0.0),
        # an odd vocabulary with padded rows in fp32, nine tenths of it masked by a grammar (one row wholly)
        dict(name="sample-odd-f32", op="sample", R=67, V=50021, dtype="f32", pad=3, requests="top-k", masked=0.9),
        # many candidates a stream, or a batch of rollouts: plain temperature sampling
        dict(name="sample-rollouts", op="sample", R=512, V=262144, dtype="bf16", pad=0, requests="temperature", masked=0.0),
        # the target rows of one stream's block before its verify
        dict(name="filter-single-stream", op="filter", R=9, V=151936, dtype="bf16", pad=0, requests="top-p", masked=0.0),
        # the target rows of 128 streams
        dict(name="filter-large-vocab-128", op="filter", R=1152, V=262144, dtype="bf16", pad=0, requests="mixed", masked=0.0),
        # a small fp32 head with an odd vocabulary
        dict(name="distill-odd-f32", op="distill", R=61, V=50021, dtype="f32", pad=3, K=64, rest=False, tau=2.0),
        # a drafter's training step over 256 blocks of 8 positions, the teacher's 16 best tokens and the rest as one class
        dict(name="distill-blocks", op="distill", R=2048, V=151936, dtype="bf16", pad=0, K=16, rest=True, tau=1.0),
        # one stream's block: the latency of a small gradient
        dict(name="grad-one-block", op="grad", R=8, V=151936, dtype="bf16", pad=0, K=16, rest=True, tau=1.0),
        dict(name="grad-odd-f32", op="grad", R=61, V=50021, dtype="f32", pad=3, K=64, rest=False, tau=2.0),
        dict(name="grad-blocks", op="grad", R=2048, V=151936, dtype="bf16", pad=0, K=16, rest=True, tau=1.0),
    ]


# logits of the largest listed case of each operator: no drawn case has more
MOST = {"sample": 512 * 262144, "filter": 1152 * 262144, "distill": 2048 * 151936, "grad": 2048 * 151936}


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("sample", "filter", "distill", "grad"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    V = _spread(rng, 61, 262144)
    R = _spread(rng, 1, min(2048, MOST[op] // V // (2 if dtype == "f32" else 1)))
    case = dict(op=op, R=R, V=V, dtype=dtype, pad=rng.choice((0, 0, 1, 5, 8)))
    if op in ("sample", "filter"):
        case.update(requests=rng.choice(sorted(REQUESTS)), masked=rng.choice((0.0, 0.0, 0.5, 0.9)))
    else:
        case.update(K=_spread(rng, 1, min(256, V // 2)), rest=rng.random() < 0.5, tau=rng.choice((1.0, 1.0, 2.0, 0.7)))
    return case


def _rows(gen, R, V, dtype, pad):
    """[R, V] logits: a bulk of N(0, 2) with, in three rows of four, 24 tokens
    raised by 4 to 14 as a model that knows a few continuations has them; the
    fourth row stays flat.  ``pad`` elements lie between rows."""
    z = torch.empty(R, V + pad, dtype=torch.float32, device=DEVICE).normal_(0.0, 2.0, generator=gen)
    at = torch.randint(0, V, (R, 24), device=DEVICE, generator=gen)
    up = 4.0 + 10.0 * torch.rand(R, 24, device=DEVICE, generator=gen)
    up[3::4] = 0.0
    z.scatter_add_(1, at, up)
    return z.to(TYPES[dtype])[:, :V]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 2 + 1)
    R, V, dtype = case["R"], case["V"], case["dtype"]
    z = _rows(gen, R, V, dtype, case["pad"])
    state = dict(op=case["op"], z=z)
    if case["op"] in ("sample", "filter"):
        if case["masked"]:
            gone = torch.rand(R, V, device=DEVICE, generator=gen) < case["masked"]
            gone[R // 2] |= case["masked"] > 0.85  # a grammar with no way on: an empty row
            z.masked_fill_(gone, -math.inf)
        asked = REQUESTS[case["requests"]]
        pick = [asked[(i + int(seed)) % len(asked)] for i in range(R)]
        state.update(
            T=torch.tensor([p[0] for p in pick], dtype=torch.float32, device=DEVICE),
            top_k=torch.tensor([p[1] for p in pick], dtype=torch.int32, device=DEVICE),
            top_p=torch.tensor([p[2] for p in pick], dtype=torch.float32, device=DEVICE),
            min_p=torch.tensor([p[3] for p in pick], dtype=torch.float32, device=DEVICE),
            u=torch.rand(R, dtype=torch.float64, device=DEVICE, generator=gen))
        if case["op"] == "sample":
            state.update(token=torch.empty(R, dtype=torch.int32, device=DEVICE),
                         prob=torch.empty(R, dtype=torch.float32, device=DEVICE))
        else:
            state["out"] = torch.empty(R, V + case["pad"], dtype=z.dtype, device=DEVICE)[:, :V]
        state["kept"] = torch.empty(R, dtype=torch.int32, device=DEVICE)
        return state
    # the teacher: other rows of the same kind, half of each the student's own; its K best tokens and its log-sum-exp
    K, tau = case["K"], case["tau"]
    t = z.float() * 0.5 + _rows(gen, R, V, "f32", 0) * 0.75
    best, at = torch.topk(t, K, dim=1)
    weight = torch.ones(R, dtype=torch.float32, device=DEVICE)
    weight[5::7] = 0.0  # padded positions
    weight[1::3] *= 0.5
    state.update(tau=tau, t_idx=at.to(torch.int32).contiguous(), t_logit=best.contiguous(), weight=weight, t_lse=None,
                 rest=None)
    if case["rest"]:
        state["t_lse"] = torch.logsumexp(t.double() / tau, 1)
    del t
    if case["op"] == "distill":
        state.update(loss=torch.empty(R, dtype=torch.float32, device=DEVICE),
                     lse=torch.empty(R, dtype=torch.float64, device=DEVICE))
        if case["rest"]:
            state["rest"] = torch.empty(R, dtype=torch.float64, device=DEVICE)
        return state
    # what the forward pass left for the backward
    s = z.double() / tau
    state["lse"] = torch.logsumexp(s, 1) * (weight != 0)
    if case["rest"]:
        state["rest"] = torch.logsumexp(s.scatter_(1, at, -math.inf), 1) * (weight != 0)
    del s
    state["g"] = 0.5 + torch.rand(R, dtype=torch.float32, device=DEVICE, generator=gen)
    state["dS"] = torch.empty(R, V + case["pad"], dtype=z.dtype, device=DEVICE)[:, :V]
    return state


# ---------------------------------------------------------------- plain forms

def _ranked(s):
    """Sorted values, their tokens, weights and running sums (fp64: a cut or a
    draw is decided by sums over the whole row), and how many tokens each row keeps."""
    z = s["z"].float()
    z = torch.where(torch.isnan(z), -math.inf, z).clamp(max=torch.finfo(s["z"].dtype).max) + 0.0
    val, at = torch.sort(z, dim=1, descending=True, stable=True)
    del z
    live = (val > -math.inf).sum(1)
    greedy = ~(s["T"] > 0)
    T = torch.where(greedy, 1.0, s["T"]).double()
    w = val.double().sub_(val[:, :1].double()).div_(T[:, None]).exp_().masked_fill_(val == -math.inf, 0.0)
    run_sum = torch.cumsum(w, 1)

    def upto(n):
        return run_sum.gather(1, (n - 1).clamp(min=0)[:, None])[:, 0]

    k = torch.where(s["top_k"] > 0, torch.minimum(s["top_k"].long(), live), live)
    k = torch.where(greedy, torch.minimum(torch.ones_like(live), live), k)
    p = s["top_p"].double()
    n_p = torch.where(p < 1, (run_sum < (p * upto(k))[:, None]).sum(1) + 1, live)
    m = s["min_p"].double()
    n_m = torch.where(m > 0, (w >= m.clamp(max=1.0)[:, None]).sum(1), live)
    kept = torch.minimum(torch.minimum(k, n_p), n_m)
    return val, at, w, run_sum, kept, upto(kept)


def _plain_sample(s):
    _, at, w, run_sum, kept, mass = _ranked(s)
    pos = (run_sum <= (s["u"] * mass)[:, None]).sum(1)
    pos = torch.minimum(pos, kept - 1).clamp(min=0)[:, None]
    some = kept > 0
    token = torch.where(some, at.gather(1, pos)[:, 0], -1).to(torch.int32)
    prob = torch.where(some, w.gather(1, pos)[:, 0] / mass, 0.0).float()
    return token, prob, kept.to(torch.int32)


def _plain_filter(s):
    z = s["z"]
    val, at, _, _, kept, _ = _ranked(s)
    inside = torch.arange(z.shape[1], device=z.device) < kept[:, None]
    return torch.where(inside, val, FILL).to(z.dtype).gather(1, torch.argsort(at, 1)), kept.to(torch.int32)


def _teacher(s):
    t = s["t_logit"].double() / s["tau"]
    c = torch.logsumexp(t, 1) if s["t_lse"] is None else s["t_lse"]
    logp = t - c[:, None]
    p = logp.exp()
    p_rest = (1.0 - p.sum(1)).clamp(min=0.0) if s["t_lse"] is not None else torch.zeros_like(c)
    return logp, p, p_rest


def _plain_distill(s):
    x = s["z"].double() / s["tau"]  # 64 bits: sums over the whole vocabulary
    at = s["t_idx"].long()
    on = s["weight"] != 0
    lse = torch.where(on, torch.logsumexp(x, 1), 0.0)
    logp, p, p_rest = _teacher(s)
    loss = (p * (logp - x.gather(1, at) + lse[:, None])).sum(1)
    rest = None
    if s["rest"] is not None:
        rest = torch.where(on, torch.logsumexp(x.scatter(1, at, -math.inf), 1), 0.0)
        loss = loss + torch.where(p_rest > 0, p_rest * (p_rest.log() - rest + lse), 0.0)
    return torch.where(on, s["weight"].double() * loss, 0.0).float(), lse, rest


def _plain_grad(s):
    x = s["z"].float() / s["tau"]
    at = s["t_idx"].long()
    _, p, p_rest = _teacher(s)
    total = (p.sum(1) + p_rest).float()[:, None]
    f = (s["weight"] * s["g"] / s["tau"])[:, None]
    d = total * (x.double() - s["lse"][:, None]).float().exp()
    if s["rest"] is not None:
        off = (x.double() - s["rest"][:, None]).float().exp() * p_rest.float()[:, None]
        d = d - off.scatter(1, at, 0.0)
    d = d.scatter_add(1, at, -p.float())
    return torch.where(f != 0, d * f, 0.0).to(s["z"].dtype)


# ---------------------------------------------------------------- the library's entry points

def _own(s):
    import block_draft_select_amd as dfl
    z = s["z"]
    if "rows" not in s:  # a program describes its rows and takes a workspace once
        s["rows"] = dfl.rows(z)
        s["ws"] = dfl.rows_workspace(s["rows"], z.device)
    r, ws = s["rows"], s["ws"]
    if s["op"] == "sample":
        dfl.dflash_sample(r, z, s["u"], s["token"], ws, T=s["T"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                          prob=s["prob"], kept=s["kept"])
        return s["token"], s["prob"], s["kept"]
    if s["op"] == "filter":
        dfl.dflash_filter(r, z, s["out"], ws, fill=FILL, T=s["T"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                          kept=s["kept"])
        return s["out"], s["kept"]
    if s["op"] == "distill":
        dfl.dflash_distill(r, z, s["t_idx"], s["t_logit"], s["loss"], s["lse"], ws, tau=s["tau"], t_lse=s["t_lse"],
                           weight=s["weight"], lse_rest=s["rest"])
        return s["loss"], s["lse"], s["rest"]
    dfl.dflash_distill_grad(r, z, s["t_idx"], s["t_logit"], s["lse"], s["dS"], tau=s["tau"], t_lse=s["t_lse"],
                            weight=s["weight"], grad_loss=s["g"], lse_rest=s["rest"])
    return s["dS"]


def run(state):
    if own:
        return _own(state)
    return {"sample": _plain_sample, "filter": _plain_filter, "distill": _plain_distill, "grad": _plain_grad}[state["op"]](state)


def work(case):
    n = case["R"] * case["V"] * (2 if case["dtype"] == "bf16" else 4)
    if case["op"] == "sample":
        return {"bytes": n + 36 * case["R"], "flops": 4 * case["R"] * case["V"]}
    if case["op"] == "filter":
        return {"bytes": 2 * n + 20 * case["R"], "flops": 4 * case["R"] * case["V"]}
    small = case["R"] * (8 * case["K"] + 32)
    if case["op"] == "distill":
        return {"bytes": n + small, "flops": 4 * case["R"] * case["V"]}
    return {"bytes": 2 * n + small, "flops": 4 * case["R"] * case["V"]}


# ---------------------------------------------------------------- the definition in 64 bits, row by row

def _exact_row(z, T, top_k, top_p, min_p, u):
    """(kept tokens, token, probability) of one fp64 row: softmax, then each filter in turn on what the one before left."""
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    toks = torch.nonzero(z > -math.inf)[:, 0]
    if not len(toks):
        return toks, -1, 0.0
    toks = toks[torch.argsort(-z[toks], stable=True)]
    if not T > 0:
        return toks[:1], int(toks[0]), 1.0
    v = z[toks]
    prob = torch.exp((v - v[0]) / T)
    prob = prob / prob.sum()
    n = len(toks)
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        share = torch.cumsum(prob[:n], 0)
        n = min(n, 1 + int((share < top_p * share[-1]).sum()))
    if min_p > 0:
        n = max(1, min(n, int((torch.exp((v - v[0]) / T) >= min_p).sum())))
    share = torch.cumsum(prob[:n], 0)
    i = min(n - 1, int((share <= u * share[-1]).sum()))
    return toks[:n], int(toks[i]), float(prob[i] / share[-1])


def exact(case, seed):
    s = prepare(case, seed)
    z = s["z"]
    R, V = z.shape
    if case["op"] in ("sample", "filter"):
        asked = list(zip(*(s[n].double().tolist() for n in ("T", "top_k", "top_p", "min_p", "u"))))
        token, prob, kept = [], [], []
        out = torch.full((R, V), FILL, dtype=torch.float64, device=z.device) if case["op"] == "filter" else None
        for r in range(R):
            row = z[r].double()
            T, top_k, top_p, min_p, u = asked[r]
            toks, tok, p = _exact_row(row, T, int(top_k), top_p, min_p, u)
            token.append(tok)
            prob.append(p)
            kept.append(len(toks))
            if out is not None:
                out[r, toks] = row[toks]
        kept = torch.tensor(kept, dtype=torch.int32)
        if out is not None:
            return out, kept
        return torch.tensor(token, dtype=torch.int32), torch.tensor(prob, dtype=torch.float64), kept
    K, tau = case["K"], case["tau"]
    loss, lse, rest = [], [], []
    grad = torch.zeros(R, V, dtype=torch.float64, device=z.device) if case["op"] == "grad" else None
    for r in range(R):
        w = s["weight"][r].double()
        if w == 0:
            loss.append(w)
            lse.append(w)
            rest.append(w)
            continue
        x, at = z[r].double() / tau, s["t_idx"][r].long()
        t = s["t_logit"][r].double() / tau
        top = x.max()
        q = torch.exp(x - top)
        total = q.sum()
        listed_q = q[at]
        q[at] = 0.0
        unlisted = q.sum()
        whole = torch.exp(t - t.max()).sum().log() + t.max() if s["t_lse"] is None else s["t_lse"][r]
        p = torch.exp(t - whole)
        d = (p * (t - whole - torch.log(listed_q / total))).sum()
        p_rest = 1.0 - p.sum()
        if case["rest"] and p_rest > 0:
            d = d + p_rest * torch.log(p_rest * total / unlisted)
        loss.append(w * d)
        lse.append(top + total.log())
        rest.append(top + unlisted.log())
        if grad is not None:
            mass = p.sum() + (p_rest.clamp(min=0.0) if case["rest"] else 0.0)
            grad[r] = q * (mass / total - (p_rest.clamp(min=0.0) / unlisted if case["rest"] else 0.0))
            grad[r, at] = listed_q * (mass / total) - p
            grad[r] *= w * s["g"][r].double() / tau
    if grad is not None:
        return grad
    return torch.stack(loss), torch.stack(lse), torch.stack(rest) if case["rest"] else None
