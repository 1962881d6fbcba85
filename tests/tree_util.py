"""Token-tree calls restated in 64 bits on the CPU, one sequence and head at a time, and the batches the tests run."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # a rounding's largest relative error
F32 = 2.0 ** -24
FIRST = {torch.float16: 2.0 ** -24, torch.bfloat16: 0.0}  # the least step of the type near zero


def chain(parent, j):
    out = [j]
    while parent[out[-1]] >= 0:
        out.append(int(parent[out[-1]]))
    return out


def random_tree(rng, T, kind="random"):
    if kind == "chain":
        return np.arange(-1, T - 1)
    if kind == "star":
        return np.array([-1] + [0] * (T - 1))[:T]
    return np.array([-1] + [int(rng.integers(0, j)) for j in range(1, T)])[:T]


class Batch:
    """Ragged sequences over a pool of pages; `poison` fills every slot that no sequence uses with NaN."""

    def __init__(self, lens, nodes, heads, kv_heads, d, page, dtype, *, seed=0, kind="random", token_major=False,
                 layers=1, poison=True, extra_rows=3, sharp=2.0, room=0, device="cuda"):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.B, self.lens, self.nodes, self.heads, self.kv_heads = B, list(lens), list(nodes), heads, kv_heads
        self.d, self.page, self.dtype, self.G, self.layers = d, page, dtype, heads // kv_heads, layers
        T = max(1, max(nodes))
        self.T = T
        need = [-(-(lens[b] + nodes[b] + room) // page) for b in range(B)]
        mp = max(1, max(need))
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.table = np.full((B, mp), -7, dtype=np.int32)  # never read past a sequence's pages
        at = 0
        for b in range(B):
            self.table[b, : need[b]] = order[at: at + need[b]]
            at += need[b]
        shape = (layers, pages, page, kv_heads, d) if token_major else (layers, pages, kv_heads, page, d)
        k = torch.randn(shape, generator=gen).to(dtype)
        v = torch.randn(shape, generator=gen).to(dtype)
        if token_major:
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        if poison:
            used = torch.zeros(pages, page, dtype=torch.bool)
            for b in range(B):
                for s in range(lens[b] + nodes[b]):
                    used[self.table[b, s // page], s % page] = True
            for x in (k, v):
                x.masked_fill_(~used[None, :, None, :, None], float("nan"))
        self.row_off, row = [], 1
        for b in rng.permutation(B):  # rows of the sequences in another order than the sequences, a gap before the first
            self.row_off.append((int(b), row))
            row += nodes[b]
        self.row_off = [r for _, r in sorted(self.row_off)]
        self.rows = row + extra_rows
        self.q = (torch.randn(self.rows, heads, d, generator=gen) * sharp).to(dtype)
        self.parent = np.full((B, T), 999, dtype=np.int32)
        for b in range(B):
            self.parent[b, : nodes[b]] = random_tree(rng, nodes[b], kind)
        self.k, self.v, self.rng, self.gen = k, v, rng, gen
        self.device = device

    def dev(self, x, dtype=None):
        t = torch.as_tensor(x)
        if dtype is not None:
            t = t.to(dtype)
        if t.dim() > 3 and not t.is_contiguous():  # keep a token-major pool's strides
            out = t.transpose(-3, -2).contiguous().to(self.device).transpose(-3, -2)
            return out
        return t.to(self.device)

    def one(self, x):
        return x[0] if self.layers == 1 else x

    def upload(self, mass=None, pos=None, tokens=None):
        import speculative_decoding_token_gb300 as sv
        self.dk, self.dv = self.dev(self.one(self.k)), self.dev(self.one(self.v))
        self.dmass = None if mass is None else self.dev(self.one(mass))
        self.dpos = None if pos is None else self.dev(self.one(pos))
        self.dq, self.dlens = self.dev(self.q), self.dev(self.lens, torch.int32)
        self.cache = sv.KVCache(self.dk, self.dv, self.dev(self.table), mass=self.dmass, pos=self.dpos)
        self.tree = sv.TokenTree(self.dev(self.row_off, torch.int64), self.dev(self.nodes, torch.int32),
                                 self.dev(self.parent), None if tokens is None else self.dev(tokens, torch.int32))
        return self

    def slots(self, b, count):
        s = np.arange(count)
        return torch.as_tensor(self.table[b, s // self.page].astype(np.int64)), torch.as_tensor(s % self.page)


def scores(q, k, scale):
    """Scores in 64 bits, and what bounds their error in 32: sum |q||k| per row and slot."""
    q, k = q.double(), k.double()
    return q @ k.T * scale, (q.abs() @ k.abs().T) * scale


def weight_error(d, size, top):
    """The relative error of exp(score - reference) when a score of d exact products is summed in fp32 in any order, with
    each partial sum rounded or cut (2^-23 of sum |q||k| = size each), scaled and exponentiated (arguments of size top)."""
    return (d + 8) * 2.0 ** -23 * size + 8 * 2.0 ** -23 * (1 + top)


def attention(bt, scale):
    """out, lse and their tolerances, rows of no sequence NaN."""
    out = torch.full((bt.rows, bt.heads, bt.d), float("nan"), dtype=torch.float64)
    lse = torch.full((bt.rows, bt.heads), float("nan"), dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = HALF[bt.dtype]
    for b in range(bt.B):
        L, T, o = bt.lens[b], bt.nodes[b], bt.row_off[b]
        pg, at = bt.slots(b, L + T)
        for g in range(bt.kv_heads):
            k, v = bt.k[0][pg, g, at], bt.v[0][pg, g, at].double()
            for j in range(T):
                see = torch.as_tensor(sorted(list(range(L)) + [L + i for i in chain(bt.parent[b], j)]))
                hs = slice(g * bt.G, (g + 1) * bt.G)
                x, size = scores(bt.q[o + j, hs], k[see], scale)
                z = torch.logsumexp(x, 1)
                p = torch.exp(x - z[:, None])
                out[o + j, hs] = p @ v[see]
                lse[o + j, hs] = z
                e = weight_error(bt.d, size.max(1)[0], x.abs().max(1)[0])
                n = len(see)
                # a weight's own rounding and error, the sums over n slots, the final rounding
                both = (2 * e + (u + 4 * n * 2.0 ** -23))[:, None] * (p @ v[see].abs())
                tol[o + j, hs] = both * (1 + u) + u * out[o + j, hs].abs() + FIRST[bt.dtype] + 1e-30
                tol_lse[o + j, hs] = e + 4 * n * F32 + 8 * F32 * (z.abs() + 1)
    return out, lse, tol, tol_lse


def verify(parent, nodes, tokens, row_off, target):
    B, T = tokens.shape
    n, out, path = np.full(B, -1), np.full((B, T), -1), np.full((B, T), -1)
    for b in range(B):
        at, walk, emitted = 0, [0], []
        while nodes[b] > 0:
            row = np.asarray(target[row_off[b] + at].double())
            if np.isnan(row).any():
                walk = None
                break
            best = int(np.argmax(row))
            emitted.append(best)
            below = [j for j in range(1, nodes[b]) if parent[b][j] == at and tokens[b][j] == best]
            if not below:
                break
            at = below[0]
            walk.append(at)
        if nodes[b] > 0 and walk is not None:
            n[b] = len(walk) - 1
            out[b, : len(walk)] = emitted
            path[b, : len(walk)] = walk
    return n, out, path


def accumulate(bt, mass, lse, n, path, scale):
    """mass + the accepted nodes' weights, [pages, heads, page], and the tolerance."""
    total = mass.double().clone()
    tol = torch.zeros_like(total)
    for b in range(bt.B):
        if n[b] < 0:
            continue
        for g in range(bt.kv_heads):
            pg, at = bt.slots(b, bt.lens[b] + n[b] + 1)
            k = bt.k[0][pg, g, at]
            add, err = torch.zeros(len(at), dtype=torch.float64), torch.zeros(len(at), dtype=torch.float64)
            for i in range(n[b] + 1):
                row = bt.row_off[b] + int(path[b][i])
                hs = slice(g * bt.G, (g + 1) * bt.G)
                x, size = scores(bt.q[row, hs], k, scale)
                z = lse[row, hs].double()
                p = torch.exp(x - z[:, None])
                p[:, bt.lens[b] + i + 1:] = 0
                add += p.sum(0)
                err += (p * weight_error(bt.d, size, x.abs() + z.abs()[:, None])).sum(0)
            rows = (n[b] + 1) * bt.G
            total[pg, g, at] += add
            tol[pg, g, at] = err + (2 * rows + 4) * F32 * (add + total[pg, g, at].abs())
    return total, tol


def keep_slots(mass, pos, seen, budget, sink, recent):
    """(source of each of the first min(len, budget) slots)."""
    L = len(mass)
    if L <= budget:
        return np.arange(L)
    safe = (pos < sink) | (pos >= seen - recent)
    key = np.where(np.isnan(mass), -np.inf, mass)
    nan = np.isnan(mass)
    order = sorted(range(L), key=lambda s: (not safe[s], 0 if safe[s] else (nan[s], -key[s]), s))
    stay = sorted(order[:budget])
    free = [s for s in range(budget) if s not in set(stay)]
    src = np.arange(budget)
    src[free] = [s for s in stay if s >= budget]
    return src
