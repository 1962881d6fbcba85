"""Workloads of the token log-probability and distillation operators: the log-probabilities of given tokens with entropy,
rank and top alternatives, their gradient, and the divergence of a draft's rows from the target's top tokens with its
gradient.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, through the package's calls;
``exact`` is each operator's definition in 64 bits.

Log-probabilities are asked for as a verify step emits tokens: tokens [B, M], -1 past a sequence's last, row m of sequence
b being row ``row_off[b] + m`` of the logits; or flat, one token a row. The others take flat rows: a token (-1: the row
counts for nothing), or a list of K token ids (-1: unused) with the target's log-probabilities or logits of them.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
DIVERGENCES = ("fkl", "rkl", "jsd", "tvd")
REST_FLOOR = 2.0 ** -20  # least mass outside the target's list whose logarithm the reverse divergence takes


def listed():
    return [
        # -- log-probabilities. One user's step: five emitted tokens with five alternatives each, what a chat server shows.
        {"name": "lp_b1_g4_v32000_fp32_k5", "op": "logprobs", "B": 1, "gmin": 4, "gmax": 4, "V": 32000, "dtype": "fp32",
         "T": 1.0, "k": 5, "rank": False, "hidden": 0},
        # A serving batch on the repository's 128256-token workload, with ranks and the twenty alternatives that servers
        # allow at most.
        {"name": "lp_b64_g8_v128256_k20", "op": "logprobs", "B": 64, "gmin": 2, "gmax": 8, "V": 128256, "dtype": "bf16",
         "T": 1.0, "k": 20, "rank": True, "hidden": 256},
        # The benchmark's batch: log-probability and entropy of what the step emitted, no alternatives.
        {"name": "lp_b256_g10_v152064_k0", "op": "logprobs", "B": 256, "gmin": 1, "gmax": 10, "V": 152064, "dtype": "bf16",
         "T": 0.75, "k": 0, "rank": False, "hidden": 0},
        # A target's pass over training text that keeps its 64 best tokens of every position for distillation.
        {"name": "lp_flat_r2000_v152064_k64", "op": "logprobs", "B": 2000, "gmin": 0, "gmax": 0, "V": 152064,
         "dtype": "bf16", "T": 1.0, "k": 64, "rank": False, "hidden": 0},
        # -- their gradient: a policy-gradient step on a short fp32 batch of an odd vocabulary, with an entropy bonus; and
        # maximum likelihood over a packed training batch, prompts masked.
        {"name": "lpgrad_r37_v50257_fp32_ent", "op": "logprobs_grad", "R": 37, "V": 50257, "dtype": "fp32", "T": 1.0,
         "ent": True, "skipped": 5, "hidden": 0},
        {"name": "lpgrad_r2048_v152064", "op": "logprobs_grad", "R": 2048, "V": 152064, "dtype": "bf16", "T": 1.0,
         "ent": False, "skipped": 256, "hidden": 0},
        # -- the divergence alone, as an evaluation takes it: a few rows, and a held-out batch.
        {"name": "distill_r5_v32000_fp32_k8_tvd", "op": "distill_loss", "R": 5, "V": 32000, "dtype": "fp32", "T": 0.875,
         "K": 8, "kmin": 8, "kind": "tvd", "form": "logprobs", "skipped": 0, "hidden": 0},
        {"name": "distill_r1111_v128256_k64_jsd", "op": "distill_loss", "R": 1111, "V": 128256, "dtype": "bf16", "T": 1.0,
         "K": 64, "kmin": 20, "kind": "jsd", "form": "logprobs", "skipped": 111, "hidden": 256},
        # -- with its gradient: a small odd vocabulary; the training batch of the large bf16 vocabulary from stored
        # log-probabilities; and fp32 rows of the largest vocabulary against long lists.
        {"name": "distillgrad_r48_v1001_fp32_k3", "op": "distill_grad", "R": 48, "V": 1001, "dtype": "fp32", "T": 2.0,
         "K": 3, "kmin": 1, "kind": "fkl", "form": "logits", "skipped": 4, "hidden": 0},
        {"name": "distillgrad_r2048_v152064_k64", "op": "distill_grad", "R": 2048, "V": 152064, "dtype": "bf16", "T": 1.0,
         "K": 64, "kmin": 64, "kind": "fkl", "form": "logprobs", "skipped": 256, "hidden": 0},
        {"name": "distillgrad_r512_v256000_fp32_k128_rkl", "op": "distill_grad", "R": 512, "V": 256000, "dtype": "fp32",
         "T": 1.0, "K": 128, "kmin": 100, "kind": "rkl", "form": "logprobs", "skipped": 12, "hidden": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "distill_loss", "distill_grad", "distill_grad"])
    dtype = rng.choice(["bf16", "fp32"])
    V = _log(rng, 500, 256000)
    most = max(2, min(2048, 500_000_000 // (V * SIZE[dtype])))
    c = {"op": op, "V": V, "dtype": dtype, "T": rng.randint(32, 128) / 64,
         "hidden": rng.choice([0, 0, rng.randint(1, V // 4)])}
    if op == "logprobs":
        gmax = rng.choice([0, rng.randint(1, 10)])
        c |= {"B": _log(rng, 1, max(1, most // (gmax + 1))), "gmin": rng.randint(0, gmax), "gmax": gmax,
              "k": rng.choice([0, 1, _log(rng, 2, 128), _log(rng, 2, 32)]), "rank": rng.random() < 0.5}
        return c
    c["R"] = _log(rng, 1, most)
    c["skipped"] = rng.randint(0, c["R"] // 4)
    if op == "logprobs_grad":
        c["ent"] = rng.random() < 0.5
        return c
    c["K"] = _log(rng, 1, min(256, V // 4))
    c["kmin"] = rng.randint(1, c["K"])
    c["kind"] = rng.choice(DIVERGENCES)
    c["form"] = "logprobs" if c["kind"] == "rkl" else rng.choice(["logprobs", "logprobs", "logits"])
    return c


# ---------------------------------------------------------------------------
# inputs

def _steps(lo, hi, n):
    """n sizes spread evenly from lo to hi (one size: hi)."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _spread(gen, lo, hi, n):
    """The same, in an order of the seed's: every seed has the same work."""
    at = torch.randperm(n, generator=gen, device=DEVICE)
    return torch.tensor(_steps(lo, hi, n), dtype=torch.int32).to(DEVICE)[at]


def _emitted(gamma):
    """Tokens that a verify step of that many drafts emits: seven drafts in ten are accepted."""
    return 1 + 7 * gamma // 10


def _rows(gen, c, rows, like=None):
    """[rows, V] logits in rows of whole 16-byte pieces: a heavy tail (logits fall with the logarithm of the rank), one row
    in ten with a token that has nearly all of the mass, `hidden` last tokens masked out; or noise around `like`."""
    V = c["V"]
    stride = -(-V // 8) * 8
    out = torch.empty(rows, stride, dtype=DTYPES[c["dtype"]] if like is None else torch.float32, device=DEVICE)
    for r in range(0, rows, 256):
        n = min(256, rows - r)
        x = torch.randn(n, V, generator=gen, device=DEVICE).mul_(0.5)
        if like is None:
            x.add_(torch.empty_like(x).exponential_(generator=gen), alpha=1.1)
            peak = torch.randint(0, V - c["hidden"], (n, 1), generator=gen, device=DEVICE)
            sharp = (torch.rand(n, 1, generator=gen, device=DEVICE) < 0.1) * 20.0
            x.scatter_add_(1, peak, sharp)
            if c["hidden"]:
                x[:, V - c["hidden"]:] = -math.inf
        else:
            x += like[r: r + n].float()
        out[r: r + n, :V] = x
    out[:, V:] = 0.0
    return out[:, :V]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = {"case": c}
    V, op = c["V"], c["op"]
    if op == "logprobs":
        B, M = c["B"], c["gmax"] + 1
        gamma = _spread(gen, c["gmin"], c["gmax"], B)
        s["row_off"] = (torch.cumsum(gamma + 1, 0) - (gamma + 1)).to(torch.int64) if M > 1 else None
        s["logits"] = _rows(gen, c, B + sum(_steps(c["gmin"], c["gmax"], B)))
        tokens = torch.randint(0, V - c["hidden"], (B, M), generator=gen, device=DEVICE)
        # half of them likely ones: the best of a few thousand tokens around
        near = (tokens[..., None] + torch.arange(2000, device=DEVICE)) % (V - c["hidden"])
        row = torch.arange(M, device=DEVICE) + (torch.arange(B, device=DEVICE) if M == 1 else s["row_off"])[:, None]
        row = row.clamp(max=s["logits"].shape[0] - 1)
        best = torch.gather(near, 2, s["logits"][row[..., None], near].float().argmax(2, keepdim=True))[..., 0]
        tokens = torch.where(torch.rand(B, M, generator=gen, device=DEVICE) < 0.5, best, tokens)
        live = torch.arange(M, device=DEVICE) < _emitted(gamma)[:, None]
        s["tokens"] = torch.where(live, tokens, -1).to(torch.int32)
    else:
        R = c["R"]
        s["logits"] = _rows(gen, c, R)
        skip = torch.randperm(R, generator=gen, device=DEVICE) < c["skipped"]
        if op == "logprobs_grad":
            tokens = torch.randint(0, V - c["hidden"], (R,), generator=gen, device=DEVICE)
            s["tokens"] = torch.where(skip, -1, tokens).to(torch.int32)
            # advantages of both signs; with no entropy bonus, the weights of a mean over the batch
            s["grad_logprob"] = (torch.randn(R, generator=gen, device=DEVICE) if c["ent"]
                                 else torch.full((R,), -1.0 / max(1, R - c["skipped"]), device=DEVICE))
            s["grad_entropy"] = torch.full((R,), -0.01, device=DEVICE) if c["ent"] else None
        else:
            K = c["K"]
            target = _rows(gen, c, R, like=s["logits"])
            top, ids = [], []
            for r in range(0, R, 256):
                x = target[r: r + 256] / c["T"]
                v, i = x.topk(K, dim=1)
                top.append(v - x.logsumexp(1, keepdim=True) if c["form"] == "logprobs" else v * c["T"])
                ids.append(i)
            del target
            length = _spread(gen, c["kmin"], K, R)[:, None]
            gone = skip[:, None] | (torch.arange(K, device=DEVICE) >= length)
            s["ids"] = torch.where(gone, -1, torch.cat(ids)).to(torch.int32)
            s["target"] = torch.cat(top).contiguous()
            s["weight"] = torch.rand(R, generator=gen, device=DEVICE) + 0.5
    if own:
        _describe(s)
    return s


# ---------------------------------------------------------------------------
# the package's calls

def _describe(s):
    """What a program sets up once: the handle and the buffers of a step's results."""
    import speculative_decoding_token_gb300 as sv
    c = s["case"]
    s["handle"] = sv.SpecVerify(1, 1, c["V"])
    if c["op"] == "logprobs":
        s["got"] = s["handle"].token_logprobs_buffers(*s["tokens"].shape, k=c["k"], rank=c["rank"])
        return
    s["loss"] = torch.empty(c["R"], device=DEVICE)
    if c["op"] != "distill_loss":
        s["grad"] = torch.zeros(c["R"], s["logits"].stride(0), dtype=s["logits"].dtype, device=DEVICE)[:, : c["V"]]
    if c["op"] == "logprobs_grad":
        s["entropy"] = torch.empty(c["R"], device=DEVICE)


def _own_logprobs(s):
    c = s["case"]
    r = s["handle"].token_logprobs(s["logits"], s["tokens"], c["T"], k=c["k"], row_off=s["row_off"], out=s["got"])
    return [x for x in (r.logprob, r.entropy, r.lse, r.rank, r.topk_logprob, r.topk_idx) if x is not None]


def _own_logprobs_grad(s):
    return s["handle"].token_logprobs_grad(s["logits"], s["tokens"], s["grad_logprob"], s["grad_entropy"], s["case"]["T"],
                                           grad=s["grad"], logprob=s["loss"], entropy=s["entropy"])


def _own_distill_loss(s):
    c = s["case"]
    return s["handle"].distill_loss(s["logits"], s["ids"], s["target"], c["T"], c["kind"], form=c["form"], loss=s["loss"])


def _own_distill_grad(s):
    c = s["case"]
    return s["handle"].distill_grad(s["logits"], s["ids"], s["target"], s["weight"], c["T"], c["kind"], form=c["form"],
                                    grad=s["grad"], loss=s["loss"])


# ---------------------------------------------------------------------------
# the plain forms

def _softmax(x, T):
    """Log-probabilities, probabilities and logsumexp of the rows of x / T."""
    top = x.amax(1, keepdim=True)
    d = (x - top).div_(T)
    e = d.exp()
    total = e.sum(1, keepdim=True)
    return d - total.log(), e.div_(total), (top / T + total.log())[:, 0]


def _entropy(lp, p):
    return -torch.where(p > 0, p * lp, 0.0).sum(1)


def _plain_logprobs(s):
    c = s["case"]
    B, M = s["tokens"].shape
    k = min(c["k"], c["V"])
    b, m = (s["tokens"] >= 0).nonzero(as_tuple=True)
    row = (s["row_off"][b] if s["row_off"] is not None else b) + m
    y = s["tokens"][b, m].long()[:, None]
    logprob, entropy, lse = (torch.zeros(B, M, device=DEVICE) for _ in range(3))
    raw = s["logits"][row].float()
    lp, p, z = _softmax(raw, c["T"])
    logprob[b, m] = torch.gather(lp, 1, y)[:, 0]
    entropy[b, m] = _entropy(lp, p)
    lse[b, m] = z
    out = [logprob, entropy, lse]
    del p
    if c["rank"]:
        mine = torch.gather(raw, 1, y)
        before = (raw > mine) | ((raw == mine) & (torch.arange(c["V"], device=DEVICE) < y))
        rank = torch.zeros(B, M, dtype=torch.int32, device=DEVICE)
        rank[b, m] = before.sum(1).to(torch.int32)
        out.append(rank)
    if c["k"]:
        top = torch.full((B, M, c["k"]), -math.inf, device=DEVICE)
        idx = torch.full((B, M, c["k"]), -1, dtype=torch.int32, device=DEVICE)
        order = raw.sort(dim=1, descending=True, stable=True)[1][:, :k]
        top[b, m, :k] = torch.gather(lp, 1, order)
        idx[b, m, :k] = order.to(torch.int32)
        out += [top, idx]
    return out


def _plain_logprobs_grad(s):
    c, live = s["case"], s["tokens"] >= 0
    y = s["tokens"].clamp(min=0).long()[:, None]
    lp, p, _ = _softmax(s["logits"].float(), c["T"])
    g = torch.where(live, s["grad_logprob"], 0.0)[:, None] / c["T"]
    H = _entropy(lp, p)
    logprob = torch.where(live, torch.gather(lp, 1, y)[:, 0], 0.0)
    grad = p * -g
    if s["grad_entropy"] is not None:
        h = torch.where(live, s["grad_entropy"], 0.0)[:, None] / c["T"]
        grad -= h * torch.where(p > 0, p * (lp + H[:, None]), 0.0)
    grad.scatter_add_(1, y, g)
    return grad.to(s["logits"].dtype), logprob, torch.where(live, H, 0.0)


def _plain_distill(s, grad):
    """The divergence over the list's tokens and the rest of the vocabulary taken as one, and its gradient: with h = q dF/dq
    of each of them, dF/dz = (h - q sum h) / T for a listed token, and the rest's is shared out by the draft's softmax over
    the rest. The few logarithms of a list are in 64 bits: a small divergence is a difference of much larger terms."""
    c, T = s["case"], s["case"]["T"]
    used = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    z = s["logits"].float()
    z = z.clone() if z is s["logits"] else z
    mine = torch.gather(z, 1, ids).double() / T
    # the draft: the rest's logsumexp without the listed tokens, nothing subtracted
    at = used.nonzero(as_tuple=True)
    z[at[0], ids[at]] = -math.inf
    top = z.amax(1, keepdim=True)
    e = z.sub_(top).div_(T).exp_()
    total = e.sum(1, keepdim=True)
    rest = top.double() / T + total.double().log()
    lq = torch.cat([torch.where(used, mine, -math.inf), rest], 1)
    lq = _softmax(lq, 1.0)[0]
    q = lq.exp()
    # the target, and what its list leaves of one
    t = torch.where(used, s["target"].double() / (T if c["form"] == "logits" else 1.0), -math.inf)
    if c["form"] == "logits":
        t = t - t.amax(1, keepdim=True).clamp(min=-1e300)
        t = t - t.exp().sum(1, keepdim=True).clamp(min=1e-300).log()
        missing = torch.zeros_like(t[:, :1])
    else:
        missing = (1.0 - t.exp().sum(1, keepdim=True)).clamp(min=0.0)
    p = torch.cat([t.exp(), missing], 1)
    lp = torch.cat([t, missing.clamp(min=REST_FLOOR if c["kind"] == "rkl" else 0.0).log()], 1)
    zero = torch.zeros_like(p)
    if c["kind"] == "fkl":
        f = torch.where(p > 0, p * (lp - lq), zero)
        h = -p
    elif c["kind"] == "rkl":
        f = h = torch.where(q > 0, q * (lq - lp), zero)
    elif c["kind"] == "tvd":
        f = 0.5 * (p - q).abs()
        h = 0.5 * q * torch.sign(q - p)
    else:
        lm = (0.5 * p + 0.5 * q).log()
        h = 0.5 * torch.where(q > 0, q * (lq - lm), zero)
        f = 0.5 * torch.where(p > 0, p * (lp - lm), zero) + h
    live = used.any(1)
    loss = torch.where(live, f.sum(1), 0.0).float()
    if not grad:
        return loss
    w = torch.where(live, s["weight"], 0.0)[:, None] / T
    d = (w * (h - q * h.sum(1, keepdim=True))).float()
    out = e.mul_(d[:, -1:] / total)
    out[at[0], ids[at]] = d[:, :-1][at]
    return out.to(s["logits"].dtype), loss


def _plain_distill_loss(s):
    return _plain_distill(s, False)


def _plain_distill_grad(s):
    return _plain_distill(s, True)


def run(state):
    op = state["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](state)


# ---------------------------------------------------------------------------
# cost

def work(case):
    """Logits once each way, a few operations a logit (maximum, exponential, sums), the small arrays."""
    c = case
    row = c["V"] * SIZE[c["dtype"]]
    if c["op"] == "logprobs":
        n = sum(_emitted(g) for g in _steps(c["gmin"], c["gmax"], c["B"]))
        each = 4 + 12 + (4 if c["rank"] else 0) + 8 * c["k"]
        return {"bytes": n * row + c["B"] * (c["gmax"] + 1) * each, "flops": n * c["V"] * (6 + (2 if c["k"] else 0))}
    n = c["R"] - c["skipped"]
    if c["op"] == "logprobs_grad":
        return {"bytes": (n + c["R"]) * row + 20 * c["R"], "flops": n * c["V"] * (12 if c["ent"] else 7)}
    small = 8 * c["R"] * c["K"] + 8 * c["R"]
    if c["op"] == "distill_loss":
        return {"bytes": n * row + small, "flops": n * c["V"] * 4}
    return {"bytes": (n + c["R"]) * row + small, "flops": n * c["V"] * 7}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits

def _exact_logprobs(s):
    c = s["case"]
    B, M = s["tokens"].shape
    V, k = c["V"], min(c["k"], c["V"])
    logprob, entropy, lse = (torch.zeros(B, M, dtype=torch.float64, device=DEVICE) for _ in range(3))
    rank = torch.zeros(B, M, dtype=torch.int32, device=DEVICE)
    top = torch.full((B, M, c["k"]), -math.inf, dtype=torch.float64, device=DEVICE)
    idx = torch.full((B, M, c["k"]), -1, dtype=torch.int32, device=DEVICE)
    tokens = s["tokens"].tolist()
    off = list(range(B)) if s["row_off"] is None else s["row_off"].tolist()
    for b in range(B):
        for m in range(M):
            y = tokens[b][m]
            if y < 0:
                continue
            raw = s["logits"][off[b] + m].double()
            x = raw / c["T"]
            lse[b, m] = torch.logsumexp(x, 0)
            x = x - lse[b, m]
            logprob[b, m] = x[y]
            seen = x[x > -math.inf]
            entropy[b, m] = -(seen.exp() * seen).sum()
            if c["rank"]:
                rank[b, m] = (raw > raw[y]).sum() + (raw[:y] == raw[y]).sum()
            if k:
                # everything that ties with the k-th best, the lower index first
                least = raw.topk(k)[0][-1]
                i = (raw >= least).nonzero()[:, 0]
                i = i[raw[i].argsort(descending=True, stable=True)][:k]
                idx[b, m, :k] = i.to(torch.int32)
                top[b, m, :k] = x[i]
    return [logprob, entropy, lse] + ([rank] if c["rank"] else []) + ([top, idx] if c["k"] else [])


def _exact_logprobs_grad(s):
    c = s["case"]
    logprob, entropy = torch.zeros(2, c["R"], dtype=torch.float64, device=DEVICE)
    grad = torch.zeros_like(s["logits"], dtype=torch.float32)
    for r in range(c["R"]):
        y = int(s["tokens"][r])
        if y < 0:
            continue
        z = s["logits"][r].double().clamp(min=-1e5).requires_grad_()  # exp(-1e5) is 0
        x = torch.log_softmax(z / c["T"], 0)
        H = -(x.exp() * x).sum()
        f = s["grad_logprob"][r].double() * x[y]
        if s["grad_entropy"] is not None:
            f = f + s["grad_entropy"][r].double() * H
        grad[r] = torch.autograd.grad(f, z)[0].float()
        logprob[r], entropy[r] = x[y].detach(), H.detach()
    return grad, logprob, entropy


def _exact_distill(s, with_grad):
    c, T = s["case"], s["case"]["T"]
    loss = torch.zeros(c["R"], dtype=torch.float64, device=DEVICE)
    grad = torch.zeros_like(s["logits"], dtype=torch.float32) if with_grad else None
    lengths = (s["ids"] >= 0).sum(1).tolist()
    for r, n in enumerate(lengths):
        if n == 0:
            continue
        ids, t = s["ids"][r, :n].long(), s["target"][r, :n].double()
        z = s["logits"][r].double().clamp(min=-1e5).requires_grad_(with_grad)
        x = torch.log_softmax(z / T, 0)
        other = torch.ones(c["V"], dtype=torch.bool, device=DEVICE)
        other[ids] = False
        lq = torch.cat([x[ids], torch.logsumexp(x[other], 0)[None]])
        if c["form"] == "logits":
            p = torch.cat([torch.softmax(t / T, 0), t.new_zeros(1)])
        else:
            p = torch.cat([t.exp(), (1.0 - t.exp().sum()).clamp(min=0.0)[None]])
        q = lq.exp()
        if c["kind"] == "fkl":
            f = torch.special.xlogy(p, p).sum() - (p * lq).sum()
        elif c["kind"] == "rkl":
            f = (q * (lq - torch.cat([t, p[-1:].clamp(min=REST_FLOOR).log()]))).sum()
        elif c["kind"] == "tvd":
            f = 0.5 * (p - q).abs().sum()
        else:
            m = 0.5 * (p + q)
            f = 0.5 * (torch.special.xlogy(p, p).sum() - torch.special.xlogy(p, m).sum()) + 0.5 * (q * (lq - m.log())).sum()
        loss[r] = f.detach()
        if with_grad:
            grad[r] = (torch.autograd.grad(f, z)[0] * s["weight"][r].double()).float()
    return (grad, loss) if with_grad else loss


def _exact_distill_loss(s):
    return _exact_distill(s, False)


def _exact_distill_grad(s):
    return _exact_distill(s, True)


def exact(case, seed):
    """The operator's definition in 64 bits, one row at a time, on the inputs of prepare(case, seed)."""
    global own
    mine, own = own, False
    try:
        return globals()["_exact_" + case["op"]](prepare(case, seed))
    finally:
        own = mine
