"""The token log-probability and distillation calls restated in 64 bits, a row at a time, with the tolerances of fp32
sums, and the rows the tests run."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # a rounding's largest relative error
# the least step of the type near zero; fp32 exponentials below the least normal number may be taken as zero
FIRST = {torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}
REST_FLOOR = 2.0 ** -20
LOWEST = {torch.bfloat16: torch.finfo(torch.bfloat16).min, torch.float32: torch.finfo(torch.float32).min}


def xlogy(a, b):
    return torch.where(a > 0, a * torch.log(b), torch.zeros_like(a))


class Soft:
    """A row's softmax at temperature T."""

    def __init__(self, z, T):
        self.z = z.double()
        self.T = float(np.float32(T))
        x = self.z / self.T
        m = x.max()
        total = torch.log(torch.exp(x - m).sum())
        self.lse = m + total
        self.lp = (x - m) - total
        self.p = torch.exp(self.lp)
        self.entropy = -torch.where(self.p > 0, self.p * self.lp, torch.zeros_like(self.p)).sum()
        # A sum of V positive terms, thread by thread and then in a tree: each weight is 2^x with x of relative error 2^-23
        # (the scale and the product rounded) and an exponential good to 2^-22; a chain of V / 128 additions at most
        # (128 threads on a row) and twenty more, half a step each. ln 2^x is at most ~ ln V where weight is left.
        # Relative error of the sum, which is the logsumexp's absolute one.
        V = len(z)
        self.sum_err = 2.0 ** -22 + 2 * math.log(V + 1) * 2.0 ** -23 + (V / 128 + 20) * 2.0 ** -24

    def lp_err(self, lp=None):
        """Absolute error of a log-probability, or of each: the sum's, and roundings of what it is taken from."""
        lp = self.lp if lp is None else lp
        fin = torch.where(torch.isfinite(lp), lp.abs(), torch.zeros_like(lp))
        return self.sum_err + 2.0 ** -22 * (fin + math.log(len(self.z) + 1))

    def lse_err(self):
        return float(self.sum_err + 2.0 ** -22 * (self.lse.abs() + math.log(len(self.z) + 1)))

    def entropy_err(self):
        """H = ln S - sum w d / (S T): the logarithm's error, and that of a sum whose terms are each of one sign."""
        mean = (self.p * torch.where(self.p > 0, (self.z - self.z.max()).abs() / self.T, torch.zeros_like(self.p))).sum()
        return float((self.sum_err + 2.0 ** -22 * math.log(len(self.z) + 1)) * (1 + 2 * mean))

    def rank(self, y):
        return int((self.z > self.z[y]).sum() + (self.z[:y] == self.z[y]).sum())

    def top(self, k):
        """Indexes of the first k tokens by (larger logit, lower index)."""
        return torch.sort(self.z, descending=True, stable=True)[1][:k]

    def grad(self, y, g, h):
        """d (g lp_y + h H) / dz, and its error before the last rounding."""
        s = torch.where(self.p > 0, self.lp + self.entropy, torch.zeros_like(self.p))
        d = -g * self.p - h * self.p * s
        d[y] += g
        # p is good to its logarithm's error; where it is multiplied, s also has its own
        e = self.lp_err()
        part = abs(g) * self.p * e + abs(h) * self.p * (s.abs() * e + e + self.entropy_err())
        # and a probability below the least normal number may be taken as zero, ahead of its factor
        err = 2 * part + 2.0 ** -22 * d.abs() + FIRST[torch.float32] * (abs(g) + abs(h) * s.abs())
        err[y] += 2.0 ** -22 * abs(g)
        return d / self.T, err / self.T


class Divergence:
    """The divergence of a draft row from a list (ids, target values), and its gradient."""

    def __init__(self, z, ids, target, T, kind, form="logprobs", beta=0.5):
        used = ids >= 0
        self.soft = s = Soft(z, T)
        self.ids = ids = ids[used].long()
        t = target[used].double()
        T = s.T
        other = torch.ones(len(z), dtype=torch.bool, device=z.device)
        other[ids] = False
        x = s.lp
        rest = torch.logsumexp(x[other], 0)[None] if other.any() else x.new_full((1,), -math.inf)
        lq = torch.cat([x[ids], rest])
        q = torch.exp(lq)
        if form == "logits":
            t = torch.log_softmax(t / T, 0)
            missing = t.new_zeros(1)
        else:
            missing = (1.0 - torch.exp(t).sum()).clamp(min=0.0)[None]
        p = torch.cat([torch.exp(t), missing])
        zero = torch.zeros_like(p)
        lp = torch.cat([t, torch.log(missing.clamp(min=REST_FLOOR if kind == "rkl" else 0.0))])
        if kind == "fkl":
            f = torch.where(p > 0, p * (lp - lq), zero)
            h = -p
        elif kind == "rkl":
            f = h = torch.where(q > 0, q * (lq - lp), zero)
        elif kind == "tvd":
            f, h = 0.5 * (p - q).abs(), 0.5 * q * torch.sign(q - p)
        else:
            lm = torch.log(beta * p + (1 - beta) * q)
            h = (1 - beta) * torch.where(q > 0, q * (lq - lm), zero)
            f = beta * torch.where(p > 0, p * (lp - lm), zero) + h
        self.loss = f.sum()
        C = h.sum()
        # A term's error: the logarithms' (each side's own), its products' roundings, and for p_rest, one less a sum of
        # fp32 values in 64 bits or pairs of floats: 2^-40 of one.
        e = float(s.lp_err(lq).max()) * 2 + 2.0 ** -22
        if form == "logits":
            e += 2.0 ** -22 * (1 + float(t[torch.isfinite(t)].abs().max()))
        self.loss_err = float(e * (1 + h.abs().sum()) + 2.0 ** -22 * torch.where(torch.isfinite(f), f.abs(), zero).sum()
                              + 2.0 ** -40 * (1 + (q[-1] + p[-1]) / max(float(missing), REST_FLOOR)))
        d = h - q * C
        # the draft's softmax over the rest; nothing where the rest has no mass
        share = torch.where(other & torch.isfinite(x), torch.exp(x - rest), torch.zeros_like(x))
        self.grad = d[-1] * share / T
        self.grad[ids] = d[:-1] / T
        # TVD's sign is only as good as q and p: a listed token where they agree to that error may take either sign
        close = ((q - p).abs() <= 2 * e * (q + p)) & (kind == "tvd")
        slack = torch.where(close, q, zero)
        size = h.abs() + q * h.abs().sum() + q
        err = 2 * e * size + slack + q * slack.sum()
        self.grad_err = err[-1] * share + d[-1].abs() * share * 2 * s.lp_err(x)
        self.grad_err[ids] = err[:-1]
        self.grad_err /= T


def close(got, want, err, dtype=torch.float32):
    """Elementwise: within the error, one rounding to the type and its least step; equal where infinite (or past the type's
    largest value, which rounds to infinity), NaN alike."""
    got, want = got.double(), torch.as_tensor(want, device=got.device).double()
    err = torch.as_tensor(err, device=got.device).double()
    lim = err * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + FIRST[dtype]
    same = (got == want.to(dtype).double()) | (got.isnan() & want.isnan())
    return bool((same | ((got - want).abs() <= lim)).all())


def logits(rows, V, dtype, seed=0, kind="plain", pad=0, device="cpu"):
    """[rows, V] in rows of whole 16-byte pieces, `pad` more elements between them; NaN between rows."""
    g = torch.Generator().manual_seed(seed)
    step = 16 // dtype.itemsize
    x = 0.5 * torch.randn(rows, V, generator=g) + 1.1 * torch.empty(rows, V).exponential_(generator=g)
    if kind == "peaked":  # nearly all of the mass on one token
        x[torch.arange(rows), torch.randint(0, V, (rows,), generator=g)] += 40.0
    elif kind == "ties":
        x = torch.randint(0, 6, (rows, V), generator=g).float()
    elif kind == "equal":
        x = torch.full((rows, V), 2.5)
    elif kind == "rising":
        x = torch.sort(x, 1)[0]
    elif kind == "falling":
        x = torch.sort(x, 1, descending=True)[0]
    elif kind == "masked":  # -inf, the type's lowest value, both; nothing else in the last row
        x[:, ::3] = -math.inf
        x[:, 1::5] = LOWEST[dtype]
        if V > 1:
            x[0, : V // 2] = -math.inf
            x[-1] = LOWEST[dtype]
            x[-1, ::2] = -math.inf
        else:
            x[:] = LOWEST[dtype]
    elif kind == "wide":  # weights over many binades
        x = 30.0 * torch.randn(rows, V, generator=g)
    out = torch.full((rows, (-(-V // step)) * step + pad * step), math.nan, dtype=dtype)
    out[:, :V] = x.to(dtype)
    return out.to(device)[:, :V]


def lists(z, K, seed=0, form="logprobs", T=1.0, noise=0.7, dtype=torch.float32, short=True):
    """Ids and values of the K best tokens of rows near z, some lists shorter, one entry unused in the middle."""
    g = torch.Generator().manual_seed(seed + 1000)
    rows, V = z.shape
    x = (z.float().cpu() + noise * torch.randn(rows, V, generator=g)) / T
    x = x.masked_fill(torch.isinf(z.cpu()), -math.inf)
    v, i = x.topk(min(K, V), 1)
    lp = v - torch.logsumexp(x, 1, keepdim=True)
    val = lp if form == "logprobs" else v * T
    i = i.masked_fill(torch.isinf(v), -1)  # a masked token is not listed
    ids = torch.full((rows, K), -1, dtype=torch.int32)
    tgt = torch.zeros(rows, K)
    ids[:, : i.shape[1]], tgt[:, : i.shape[1]] = i.to(torch.int32), torch.where(torch.isinf(val), 0.0, val)
    if short:
        for r in range(rows):
            if r % 3 == 1:
                ids[r, 1 + (r * 7) % K:] = -1
            if r % 3 == 2 and K > 2:
                ids[r, K // 2] = -1
    return ids.to(z.device), tgt.to(dtype).to(z.device)
