"""Workloads of the token-tree operators: attention of a tree of drafted tokens over a paged cache, the greedy walk that
accepts a path of the tree, the commit of that path into the cache, the accumulation of attention weight per cached token
and the eviction of the tokens that gathered least of it.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, through the package's calls;
``exact`` is each operator's definition in 64 bits.

Layout shared by all of them: caches are [layers, pages, kv heads, page size, head size] (without ``layers`` where one layer
is served), ``table`` [B, pages per sequence] names the pages of sequence b, ``lens`` [B] its committed tokens. Node j of
sequence b's tree has its key and value in slot lens[b] + j and its query and logits in row ``row_off[b] + j``; node 0 is the
token that the last step emitted, and parent[b, j] < j.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # -- tree attention. One user, a small tree, a short dialogue: the call is a few microseconds of latency.
        {"name": "attn_b1_t8_len900", "op": "attention", "B": 1, "tmin": 8, "tmax": 8, "hkv": 8, "G": 4, "d": 128,
         "lmin": 900, "lmax": 900, "page": 16, "dtype": "bf16", "token_major": False},
        # Plain decoding (trees of one node) of a few sequences with 7 query heads a key head and head size 64, odd lengths,
        # from a pool that is laid out token by token.
        {"name": "attn_b5_t1_g7_d64_fp16", "op": "attention", "B": 5, "tmin": 1, "tmax": 1, "hkv": 4, "G": 7, "d": 64,
         "lmin": 1, "lmax": 4099, "page": 32, "dtype": "fp16", "token_major": True},
        # A serving batch: ragged trees up to 26 nodes, ragged contexts.
        {"name": "attn_b16_t1to26_len300to8000", "op": "attention", "B": 16, "tmin": 1, "tmax": 26, "hkv": 8, "G": 4,
         "d": 128, "lmin": 300, "lmax": 8000, "page": 64, "dtype": "bf16", "token_major": False},
        # The largest: 64-node trees, 8 query heads a key head (512 rows share every key), contexts to 16 thousand.
        {"name": "attn_b32_t64_g8_len16k", "op": "attention", "B": 32, "tmin": 64, "tmax": 64, "hkv": 8, "G": 8,
         "d": 128, "lmin": 12000, "lmax": 16200, "page": 128, "dtype": "bf16", "token_major": False},
        # -- greedy tree verify. One sequence and a small vocabulary; and a serving batch on the repository's largest
        # bf16 vocabulary, of which only the rows on the accepted path decide.
        {"name": "verify_b1_t16_v32000", "op": "verify", "B": 1, "tmin": 16, "tmax": 16, "V": 32000, "dtype": "bf16"},
        {"name": "verify_b64_t4to48_v152064", "op": "verify", "B": 64, "tmin": 4, "tmax": 48, "V": 152064,
         "dtype": "bf16"},
        # -- commit of the accepted path: one layer's call for one sequence, and one call for all layers of a batch.
        {"name": "commit_b1_t16", "op": "commit", "B": 1, "tmin": 16, "tmax": 16, "hkv": 8, "d": 128, "layers": 1,
         "lmin": 700, "lmax": 700, "page": 16, "dtype": "bf16", "token_major": False},
        {"name": "commit_b64_t32_layers24", "op": "commit", "B": 64, "tmin": 8, "tmax": 32, "hkv": 8, "d": 128,
         "layers": 24, "lmin": 1, "lmax": 460, "page": 64, "dtype": "bf16", "token_major": False},
        # -- attention weight gathered by the accepted nodes: a single short sequence, and a long-context batch.
        {"name": "mass_b2_t9_g7_d64_fp16", "op": "accumulate", "B": 2, "tmin": 5, "tmax": 9, "hkv": 4, "G": 7, "d": 64,
         "lmin": 100, "lmax": 1500, "page": 16, "dtype": "fp16", "token_major": True},
        {"name": "mass_b24_t32_g4_len16k", "op": "accumulate", "B": 24, "tmin": 8, "tmax": 32, "hkv": 8, "G": 4,
         "d": 128, "lmin": 9000, "lmax": 16200, "page": 128, "dtype": "bf16", "token_major": False},
        # -- eviction: a cache that went a few steps over its budget (every step of a bounded cache), and a long prompt
        # cut down to its budget.
        {"name": "evict_b4_over40_keep2048", "op": "evict", "B": 4, "hkv": 8, "d": 128, "layers": 1, "lmin": 2040,
         "lmax": 2088, "budget": 2048, "sink": 4, "recent": 256, "page": 16, "dtype": "bf16", "token_major": False},
        {"name": "evict_b16_len32k_keep4096", "op": "evict", "B": 16, "hkv": 8, "d": 128, "layers": 1, "lmin": 20000,
         "lmax": 32700, "budget": 4096, "sink": 4, "recent": 512, "page": 128, "dtype": "bf16", "token_major": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "verify", "commit", "accumulate", "evict"])
    tmax = _log(rng, 1, 64)
    c = {"op": op, "B": _log(rng, 1, 32), "tmin": rng.randint(1, tmax), "tmax": tmax}
    if op == "verify":
        c["V"] = _log(rng, 1000, 152064)
        c["dtype"] = rng.choice(["bf16", "fp32"])
        return c
    c |= {"hkv": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128]), "page": rng.choice([8, 16, 24, 32, 64, 128, 256]),
          "dtype": rng.choice(["bf16", "fp16"]), "token_major": rng.random() < 0.3}
    if op in ("attention", "accumulate"):
        c["G"] = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        c["lmax"] = _log(rng, 10, 16200)
        c["lmin"] = rng.randint(1, c["lmax"])
    elif op == "commit":
        c["layers"] = _log(rng, 1, 16)
        c["lmax"] = _log(rng, 1, 460)
        c["lmin"] = rng.randint(0, c["lmax"])
    else:
        del c["tmin"], c["tmax"]
        c["B"] = min(c["B"], 16)
        c["layers"] = 1 if c["B"] > 4 else rng.randint(1, 4)
        c["lmax"] = _log(rng, 60, 30000 // c["layers"])
        c["lmin"] = rng.randint(c["lmax"] // 2, c["lmax"])
        c["budget"] = _log(rng, 20, c["lmax"])
        c["sink"] = rng.randint(0, min(8, c["budget"] // 2))
        c["recent"] = rng.randint(0, c["budget"] // 2)
    return c


# ---------------------------------------------------------------------------
# inputs

def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device=DEVICE, dtype=torch.int32)


def _steps(lo, hi, n):
    """n sizes spread evenly from lo to hi (one size: hi)."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _spread(gen, lo, hi, n):
    """The same, in an order of the seed's: every seed has the same work."""
    at = torch.randperm(n, generator=gen, device=DEVICE)
    return torch.tensor(_steps(lo, hi, n), dtype=torch.int32).to(DEVICE)[at]


def _tree(gen, s, c):
    """Random recursive trees: node j hangs below a uniform earlier node."""
    B, T = c["B"], c["tmax"]
    s["nodes"] = _spread(gen, c["tmin"], T, B)
    s["row_off"] = (torch.cumsum(s["nodes"], 0) - s["nodes"]).to(torch.int64)
    s["rows"] = int(s["nodes"].sum())
    j = torch.arange(T, device=DEVICE)
    u = torch.rand(B, T, generator=gen, device=DEVICE)
    s["parent"] = torch.where(j > 0, (u * j).floor().clamp(max=T), -1.0).clamp(max=(j - 1).clamp(min=-1)).to(torch.int32)


def _caches(gen, s, c, layers, room, value=True):
    """A pool of pages in random order, its table, and lengths; `room` slots beyond the longest sequence."""
    B, page, hkv, d = c["B"], c["page"], c["hkv"], c["d"]
    s["lens"] = _spread(gen, c["lmin"], c["lmax"], B)
    mp = -(-(c["lmax"] + room) // page)
    pages = B * mp + 3
    s["table"] = torch.randperm(pages, generator=gen, device=DEVICE)[: B * mp].view(B, mp).to(torch.int32)
    shape = (layers, pages, page, hkv, d) if c["token_major"] else (layers, pages, hkv, page, d)

    def pool():
        x = torch.randn(shape, generator=gen, device=DEVICE, dtype=DTYPES[c["dtype"]])
        return x.transpose(2, 3) if c["token_major"] else x

    s["k"] = pool()
    s["v"] = pool() if value else s["k"]
    return pages


def _queries(gen, s, c):
    q = torch.randn(s["rows"], c["hkv"] * c["G"], c["d"], generator=gen, device=DEVICE)
    sharp = 0.5 + 2.5 * torch.rand(c["hkv"] * c["G"], 1, generator=gen, device=DEVICE)  # heads differ in how peaked they are
    s["q"] = (q * sharp).to(DTYPES[c["dtype"]])
    s["scale"] = c["d"] ** -0.5


def _first_child(parent):
    same = parent[:, :, None] == parent[:, None, :]
    return ~(same & torch.ones_like(same).tril(-1)).any(2)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "verify":
        _tree(gen, s, c)
        B, T, V = c["B"], c["tmax"], c["V"]
        stride = -(-V // 8) * 8
        s["logits"] = (3.0 * torch.randn(s["rows"], stride, generator=gen, device=DEVICE)).to(DTYPES[c["dtype"]])[:, :V]
        s["tokens"] = torch.randint(0, V, (B, T), generator=gen, device=DEVICE, dtype=torch.int32)
        # the target agrees with three in four of the first children: a run of accepted drafts
        good = (torch.rand(B, T, generator=gen, device=DEVICE) < 0.75) & _first_child(s["parent"])
        j = torch.arange(T, device=DEVICE)
        good &= (j > 0) & (j < s["nodes"][:, None])
        b, j = good.nonzero(as_tuple=True)
        s["logits"][s["row_off"][b] + s["parent"][b, j], s["tokens"][b, j].long()] = 30.0
    elif c["op"] == "attention":
        _tree(gen, s, c)
        _caches(gen, s, c, 1, c["tmax"])
        s["k"], s["v"] = s["k"][0], s["v"][0]
        _queries(gen, s, c)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["rows"], c["hkv"] * c["G"], device=DEVICE)
    elif c["op"] in ("commit", "accumulate"):
        _tree(gen, s, c)
        layers = c.get("layers", 1)
        pages = _caches(gen, s, c, layers, c["tmax"], value=c["op"] == "commit")
        # an accepted path: node 0, then steps of one to three nodes
        B, T = c["B"], c["tmax"]
        step = torch.randint(1, 4, (B, T), generator=gen, device=DEVICE)
        path = torch.cumsum(step, 1) - step[:, :1]
        ok = path < s["nodes"][:, None]
        deep = torch.randint(1, 12, (B, 1), generator=gen, device=DEVICE)
        ok &= torch.arange(T, device=DEVICE) < deep
        s["path"] = torch.where(ok, path, -1).to(torch.int32)
        s["n"] = (ok.sum(1) - 1).to(torch.int32)
        shape = (layers, pages, c["hkv"], c["page"])
        s["mass"] = torch.rand(shape, generator=gen, device=DEVICE)
        if c["op"] == "commit":
            s["pos"] = torch.zeros(shape, device=DEVICE, dtype=torch.int32)
            s["seen"] = s["lens"] + _ints(gen, 0, 1000, B)
            s["new_lens"], s["new_seen"] = torch.empty_like(s["lens"]), torch.empty_like(s["lens"])
        else:
            s["k"], s["v"], s["mass"] = s["k"][0], s["v"][0], s["mass"][0]
            _queries(gen, s, c)
            # the logsumexp of the attention over the same rows; about what such scores give
            s["lse"] = (s["lens"].float().clamp(min=1).log()[_owner(s)][:, None] + 1.5
                        + 0.5 * torch.rand(s["rows"], c["hkv"] * c["G"], generator=gen, device=DEVICE))
    else:
        pages = _caches(gen, s, c, c["layers"], 0)
        shape = (c["layers"], pages, c["hkv"], c["page"])
        # heavy-tailed weights; one token in ten has gathered none
        heavy = (2.0 * torch.randn(shape, generator=gen, device=DEVICE)).exp()
        s["mass"] = torch.where(torch.rand(shape, generator=gen, device=DEVICE) < 0.1, 0.0, heavy)
        # positions: in order, with the gaps that earlier evictions left
        mp = s["table"].shape[1]
        slots = mp * c["page"]
        gaps = torch.randint(1, 3, (c["layers"], c["B"], c["hkv"], slots), generator=gen, device=DEVICE)
        order = torch.cumsum(gaps, 3) - gaps[..., :1]
        last = torch.gather(order, 3, (s["lens"].long() - 1).clamp(min=0)[None, :, None, None]
                            .expand(c["layers"], c["B"], c["hkv"], 1))
        s["seen"] = (last.amax((0, 2, 3)) + 1).to(torch.int32)
        order = order + (s["seen"][None, :, None, None] - 1 - last)
        s["pos"] = torch.zeros(shape, device=DEVICE, dtype=torch.int32)
        s["pos"][:, s["table"].long()] = order.view(c["layers"], c["B"], c["hkv"], mp, c["page"]).transpose(2, 3).to(torch.int32)
        s["mass_out"], s["pos_out"] = torch.zeros_like(s["mass"]), torch.zeros_like(s["pos"])
        s["new_lens"] = torch.empty_like(s["lens"])
        if c["layers"] == 1:
            for name in ("k", "v", "mass", "pos", "mass_out", "pos_out"):
                s[name] = s[name][0]
    if own:
        _describe(s)
    return s


def _owner(s):
    """The sequence of every row."""
    r = torch.arange(s["rows"], device=DEVICE)
    return torch.searchsorted(s["row_off"] + s["nodes"], r, right=True)


# ---------------------------------------------------------------------------
# the package's calls

def _describe(s):
    """What a program sets up once: the handle, and the descriptions of its cache and of the tree's buffers."""
    import speculative_decoding_token_gb300 as sv
    c = s["case"]
    moves = 0
    if c["op"] == "evict":
        room = s["table"].shape[1] * c["page"] - c["budget"]
        moves = c["layers"] * c["B"] * c["hkv"] * max(0, min(c["budget"], room))
    s["handle"] = sv.SpecTree(c["B"], max_moves=moves)
    if "nodes" in s:
        s["tree"] = sv.TokenTree(s["row_off"], s["nodes"], s["parent"], s.get("tokens"))
    if "k" in s:
        s["cache"] = sv.KVCache(s["k"], s["v"], s["table"], mass=s.get("mass"), pos=s.get("pos"))
    if c["op"] == "verify":
        B, T = c["B"], c["tmax"]
        s["got"] = [torch.empty(B, dtype=torch.int32, device=DEVICE), torch.empty(B, T, dtype=torch.int32, device=DEVICE),
                    torch.empty(B, T, dtype=torch.int32, device=DEVICE)]


def _own_attention(s):
    return s["handle"].attention(s["q"], s["cache"], s["tree"], s["lens"], scale=s["scale"], out=s["out"], lse=s["lse"])


def _own_verify(s):
    n, tokens, path = s["got"]
    return s["handle"].verify(s["tree"], s["logits"], n=n, tokens=tokens, path=path)


def _own_commit(s):
    s["handle"].commit(s["cache"], s["lens"], s["n"], s["path"], seen=s["seen"], new_lens=s["new_lens"],
                       new_seen=s["new_seen"])
    return s["k"], s["v"], s["mass"], s["pos"], s["new_lens"], s["new_seen"]


def _own_accumulate(s):
    s["handle"].accumulate(s["q"], s["lse"], s["cache"], s["tree"], s["lens"], s["n"], s["path"], scale=s["scale"])
    return s["mass"]


def _own_evict(s):
    c = s["case"]
    s["handle"].evict(s["cache"], s["lens"], s["seen"], c["budget"], sink=c["sink"], recent=c["recent"],
                      mass_out=s["mass_out"], pos_out=s["pos_out"], new_lens=s["new_lens"])
    return s["k"], s["v"], s["mass_out"], s["pos_out"], s["new_lens"]


# ---------------------------------------------------------------------------
# the plain forms

def _dense(pool, table):
    """[B, kv heads, slots, ...] of a pool [pages, kv heads, page, ...]."""
    x = pool[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])


def _padded(s, x):
    """Rows of x by (sequence, node), the missing ones repeating a row."""
    T = s["parent"].shape[1]
    at = s["row_off"][:, None] + torch.arange(T, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)]


def _ancestors(parent, nodes):
    """[B, T, T]: whether node i is node j or above it. The inverse of (1 - P), P the matrix of parents, sums P's powers."""
    B, T = parent.shape
    eye = torch.eye(T, device=parent.device)
    real = torch.arange(T, device=parent.device) < nodes[:, None]
    hang = (parent[:, :, None] == torch.arange(T, device=parent.device)) & real[:, :, None]
    return torch.linalg.solve_triangular(eye - hang.float(), eye.expand(B, T, T), upper=False, unitriangular=True) > 0.5


def _plain_attention(s):
    c, L = s["case"], s["lens"].long()
    T, hkv, G, d = c["tmax"], c["hkv"], c["G"], c["d"]
    k, v = _dense(s["k"], s["table"]).float(), _dense(s["v"], s["table"]).float()
    B, N = k.shape[0], k.shape[2]
    q = _padded(s, s["q"]).float().view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    i = torch.arange(N, device=k.device) - L[:, None]
    above = _ancestors(s["parent"], s["nodes"])
    node = i.clamp(0, T - 1)[:, None, :].expand(B, T, N)
    see = (i < 0)[:, None, :] | ((i >= 0) & (i < s["nodes"][:, None]))[:, None, :] & torch.gather(above, 2, node)
    see = see[:, None, :, None, :].expand(B, hkv, T, G, N).reshape(B, hkv, T * G, N)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~see, -math.inf)
    top = x.amax(3, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(3, keepdim=True)
    used = (torch.arange(N, device=k.device) < (L + s["nodes"])[:, None])[:, None, :, None]
    out = torch.matmul(x, v.masked_fill_(~used, 0.0)) / total
    lse = (top + total.log()).view(B, hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, hkv * G)
    out = out.view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, hkv * G, d)
    b = _owner(s)
    j = torch.arange(s["rows"], device=k.device) - s["row_off"][b]
    return out[b, j].to(s["q"].dtype), lse[b, j]


def _plain_verify(s):
    parent, nodes, tokens = s["parent"].long(), s["nodes"], s["tokens"]
    B, T = parent.shape
    best = _padded(s, torch.argmax(s["logits"], 1))
    j = torch.arange(T, device=parent.device)
    real = j < nodes[:, None]
    want = torch.gather(best, 1, parent.clamp(min=0))
    good = (tokens == want) & real
    twin = (parent[:, :, None] == parent[:, None, :]) & (tokens[:, :, None] == tokens[:, None, :])
    good &= ~(twin & torch.ones(T, T, dtype=torch.bool, device=parent.device).tril(-1)).any(2)
    good |= j == 0
    above = _ancestors(s["parent"], nodes)
    taken = ~(above & ~good[:, None, :]).any(2) & real
    order = torch.sort(torch.where(taken, j, T), 1)[0]
    n = taken.sum(1) - 1
    path = torch.where(order < T, order, -1)
    last = torch.gather(order, 1, n[:, None])
    final = torch.gather(best, 1, last)
    after = torch.cat([order[:, 1:], torch.full_like(order[:, :1], T)], 1)
    out = torch.where(j < n[:, None], torch.gather(tokens.long(), 1, after.clamp(max=T - 1)), -1)
    out = torch.where(j == n[:, None], final, out)
    return n.int(), out.int(), path.int()


def _place(table, slot, page):
    return torch.gather(table.long(), 1, slot // page), slot % page


def _plain_commit(s):
    L, n, page = s["lens"].long(), s["n"].long(), s["case"]["page"]
    T = s["path"].shape[1]
    i = torch.arange(T, device=L.device).expand(len(L), T)
    i = torch.where(i <= n[:, None], i, 0)  # what lies past the path repeats its first entry
    src = torch.gather(s["path"].long(), 1, i) + L[:, None]
    dst = i + L[:, None]
    sp, so = _place(s["table"], src, page)
    dp, do = _place(s["table"], dst, page)
    for pool in (s["k"], s["v"]):
        pool[:, dp, :, do] = pool[:, sp, :, so]
    s["mass"][:, dp, :, do] = torch.zeros((), device=L.device)
    at = (s["seen"][:, None] + i).to(torch.int32)[:, :, None, None]
    s["pos"][:, dp, :, do] = at.expand(len(L), T, s["pos"].shape[0], s["pos"].shape[2])
    torch.add(s["lens"], s["n"] + 1, out=s["new_lens"])
    torch.add(s["seen"], s["n"] + 1, out=s["new_seen"])
    return s["k"], s["v"], s["mass"], s["pos"], s["new_lens"], s["new_seen"]


def _plain_accumulate(s):
    c, L = s["case"], s["lens"].long()
    hkv, G, d, T = c["hkv"], c["G"], c["d"], s["path"].shape[1]
    k = _dense(s["k"], s["table"]).float()
    B, N = k.shape[0], k.shape[2]
    rows = s["row_off"][:, None] + s["path"].long().clamp(min=0)
    q = s["q"][rows].float().view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    lse = s["lse"][rows].view(B, T, hkv, G).permute(0, 2, 1, 3).reshape(B, hkv, T * G, 1)
    i = torch.arange(T, device=k.device)
    see = (torch.arange(N, device=k.device) <= (L[:, None] + i)[:, :, None]) & (i <= s["n"][:, None])[:, :, None]
    see = see[:, None, :, None, :].expand(B, hkv, T, G, N).reshape(B, hkv, T * G, N)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).sub_(lse).masked_fill_(~see, -math.inf).exp_().sum(2)
    x = x.view(B, hkv, -1, c["page"]).transpose(1, 2)
    t = s["table"].long()
    s["mass"][t] = s["mass"][t] + x
    return s["mass"]


def _plain_evict(s):
    c, L = s["case"], s["lens"].long()
    keep, page = c["budget"], c["page"]
    one = s["k"].dim() == 4
    k, v, mass, pos, mass_out, pos_out = ((s[x][None] if one else s[x]) for x in ("k", "v", "mass", "pos", "mass_out", "pos_out"))
    t = s["table"].long()

    def dense(x):
        y = x[:, t].transpose(2, 3)
        return y.reshape(*y.shape[:3], -1)

    m, p = dense(mass), dense(pos)
    N = m.shape[3]
    slot = torch.arange(N, device=m.device)
    real = (slot < L[:, None])[None, :, None]
    safe = (p < c["sink"]) | (p >= s["seen"][None, :, None, None] - c["recent"])
    key = torch.where(real, torch.where(safe, math.inf, m), -math.inf)
    rank = torch.sort(key, dim=3, descending=True, stable=True)[1]
    kept = torch.zeros_like(real.expand_as(key)).scatter_(3, rank[..., :keep], True) & real
    low = slot < keep
    # the free slots and the movers, each in ascending order; a list's tail names slots that stay
    free = torch.sort((kept | ~low).to(torch.int8), dim=3, stable=True)[1][..., :keep]
    move = torch.sort((~kept | low).to(torch.int8), dim=3, stable=True)[1][..., :keep]
    count = (kept & ~low).sum(3, keepdim=True)
    pad = torch.arange(free.shape[3], device=m.device) < count
    src = torch.where(pad, move, free)
    lay = torch.arange(k.shape[0], device=m.device)[:, None, None, None]
    head = torch.arange(k.shape[2], device=m.device)[None, None, :, None]
    b = torch.arange(len(L), device=m.device)[None, :, None, None]
    at = lambda x: (lay, t[b, x // page], head, x % page)  # noqa: E731
    for pool in (k, v):
        pool[at(free)] = pool[at(src)]
    new = L.clamp(max=keep)
    line = slot[: min(keep, N)].expand(*m.shape[:3], -1)
    come = torch.arange(N, device=m.device).expand_as(p).scatter(3, free, src)[..., : line.shape[3]]
    held = (line < new[None, :, None, None])
    for out, x in ((mass_out, m), (pos_out, p)):
        out[at(line)] = torch.where(held, torch.gather(x, 3, come), out[at(line)])
    torch.clamp(s["lens"], max=keep, out=s["new_lens"])
    return s["k"], s["v"], s["mass_out"], s["pos_out"], s["new_lens"]


def run(state):
    op = state["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](state)


# ---------------------------------------------------------------------------
# cost

def _totals(c):
    """Tokens and nodes of a case's sequences together, and the mean length of an accepted path."""
    tokens = sum(_steps(c["lmin"], c["lmax"], c["B"])) if "lmax" in c else 0
    nodes = sum(_steps(c["tmin"], c["tmax"], c["B"])) if "tmax" in c else 0
    return tokens, nodes, min(6.0, 1 + 0.5 * nodes / c["B"])


def work(case):
    c = case
    B, size = c["B"], SIZE[c["dtype"]]
    tokens, nodes, path = _totals(c)
    if c["op"] == "verify":  # the rows on the accepted path: about two
        rows = 2 * B if c["tmax"] > 1 else B
        return {"bytes": rows * c["V"] * size + 12 * nodes + 12 * B, "flops": rows * c["V"]}
    row = c["hkv"] * c["d"] * size
    if c["op"] == "attention":
        q = nodes * c["G"] * row
        per = (nodes / B) * c["G"] * c["hkv"] * c["d"]
        return {"bytes": 2 * (tokens + nodes) * row + 2 * q + 4 * nodes * c["G"] * c["hkv"], "flops": 4 * per * tokens}
    if c["op"] == "commit":  # half of the path is in place already
        return {"bytes": 2 * c["layers"] * B * path * row + 8 * c["layers"] * B * path * c["hkv"] + 16 * B,
                "flops": 2 * B}
    if c["op"] == "accumulate":
        q = B * path * c["G"] * row
        return {"bytes": tokens * (row + 8 * c["hkv"]) + q + 4 * B * path * c["G"] * c["hkv"],
                "flops": (2 * c["d"] + 3) * c["hkv"] * c["G"] * path * tokens}
    mean = tokens / B
    over = max(0.0, mean - c["budget"]) / mean  # that share of the kept tokens lies past the budget
    items = c["layers"] * B * c["hkv"]
    moves = items * min(c["budget"], mean) * over
    return {"bytes": 8 * items * mean + 4 * moves * c["d"] * size + 8 * items * min(c["budget"], mean),
            "flops": items * mean}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits

def _seq_slots(table, b, count, page):
    i = torch.arange(count, device=table.device)
    return table[b, i // page].long(), i % page


def _up(parent, j):
    chain = [j]
    while parent[chain[-1]] >= 0:
        chain.append(int(parent[chain[-1]]))
    return chain


def _exact_attention(s):
    c = s["case"]
    G, page = c["G"], c["page"]
    parent, nodes, lens, off = (s[x].cpu().numpy() for x in ("parent", "nodes", "lens", "row_off"))
    out = torch.empty(s["rows"], c["hkv"] * G, c["d"], dtype=torch.float64, device=DEVICE)
    lse = torch.empty(s["rows"], c["hkv"] * G, dtype=torch.float64, device=DEVICE)
    for b in range(c["B"]):
        L, T, o = int(lens[b]), int(nodes[b]), int(off[b])
        pg, at = _seq_slots(s["table"], b, L + T, page)
        see = np.zeros((T, L + T), dtype=bool)
        see[:, :L] = True
        for j in range(T):
            see[j, [L + i for i in _up(parent[b], j)]] = True
        see = torch.from_numpy(see).to(DEVICE)
        for h in range(c["hkv"]):
            k, v = s["k"][pg, h, at].double(), s["v"][pg, h, at].double()
            q = s["q"][o: o + T, h * G: (h + 1) * G].double()
            x = torch.einsum("tgd,nd->tgn", q, k) * s["scale"]
            x = torch.where(see[:, None], x, -torch.inf)
            z = torch.logsumexp(x, 2)
            lse[o: o + T, h * G: (h + 1) * G] = z
            out[o: o + T, h * G: (h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.exp(x - z[..., None]), v)
    return out, lse


def _exact_verify(s):
    parent, nodes, off, tokens = (s[x].cpu().numpy() for x in ("parent", "nodes", "row_off", "tokens"))
    B, T = parent.shape
    n, out, path = np.zeros(B, np.int32), np.full((B, T), -1, np.int32), np.full((B, T), -1, np.int32)
    for b in range(B):
        at, walk = 0, [0]
        while True:
            row = s["logits"][off[b] + at].double()
            best = int((row == row.max()).nonzero()[0, 0])
            below = [j for j in range(1, nodes[b]) if parent[b, j] == at and tokens[b, j] == best]
            out[b, len(walk) - 1] = best
            if not below:
                break
            at = below[0]
            walk.append(at)
        n[b] = len(walk) - 1
        path[b, : len(walk)] = walk
    return n, out, path


def _exact_commit(s):
    c = s["case"]
    lens, n, path, seen, table = (s[x].cpu().numpy() for x in ("lens", "n", "path", "seen", "table"))
    page = c["page"]
    k, v, mass, pos = (s[x].clone() for x in ("k", "v", "mass", "pos"))
    for b in range(c["B"]):
        for i in range(int(n[b]) + 1):
            src, dst = int(lens[b] + path[b, i]), int(lens[b]) + i
            for old, new in ((s["k"], k), (s["v"], v)):
                new[:, table[b, dst // page], :, dst % page] = old[:, table[b, src // page], :, src % page]
            mass[:, table[b, dst // page], :, dst % page] = 0.0
            pos[:, table[b, dst // page], :, dst % page] = int(seen[b]) + i
    return k, v, mass, pos, s["lens"] + s["n"] + 1, s["seen"] + s["n"] + 1


def _exact_accumulate(s):
    c = s["case"]
    G = c["G"]
    lens, n, path, off = (s[x].cpu().numpy() for x in ("lens", "n", "path", "row_off"))
    mass = s["mass"].double()
    for b in range(c["B"]):
        L, m = int(lens[b]), int(n[b])
        pg, at = _seq_slots(s["table"], b, L + m + 1, c["page"])
        rows = [int(off[b]) + int(path[b, i]) for i in range(m + 1)]
        x = torch.einsum("ihgd,nhd->ihgn", s["q"][rows].double().view(m + 1, c["hkv"], G, c["d"]), s["k"][pg, :, at].double())
        x = torch.exp(x * s["scale"] - s["lse"][rows].double().view(m + 1, c["hkv"], G, 1))
        late = torch.arange(L + m + 1, device=DEVICE) > L + torch.arange(m + 1, device=DEVICE)[:, None]
        x = x.masked_fill(late[:, None, None], 0.0)
        mass[pg, :, at] += x.sum((0, 2)).T
    return mass


def _exact_evict(s):
    c = s["case"]
    page, keep = c["page"], c["budget"]
    one = s["k"].dim() == 4
    k, v, mass_out, pos_out = (s[x].clone() for x in ("k", "v", "mass_out", "pos_out"))
    lift = lambda x: x[None] if one else x  # noqa: E731
    k_new, v_new, mass_new, pos_new = lift(k), lift(v), lift(mass_out), lift(pos_out)
    mass, pos = lift(s["mass"]).cpu().numpy(), lift(s["pos"]).cpu().numpy()
    lens, seen, table = (s[x].cpu().numpy() for x in ("lens", "seen", "table"))
    for b in range(c["B"]):
        L = int(lens[b])
        slots = np.arange(L)
        pg, at = table[b, slots // page], slots % page
        for a in range(c["layers"]):
            for h in range(c["hkv"]):
                m, p = mass[a, pg, h, at].astype(np.float64), pos[a, pg, h, at]
                stay = slots
                if L > keep:
                    safe = (p < c["sink"]) | (p >= seen[b] - c["recent"])
                    best = np.lexsort((slots, -m, ~safe))[:keep]
                    # two protected tokens tie, whatever they gathered
                    first = slots[safe]
                    best = first[:keep] if len(first) >= keep else best
                    stay = np.sort(best)
                free = np.setdiff1d(np.arange(min(keep, L)), stay)
                move = stay[stay >= keep]
                where = np.arange(min(keep, L))
                where[free] = move
                f, w = torch.from_numpy(free).to(DEVICE), torch.from_numpy(move).to(DEVICE)
                t = s["table"][b].long()
                for new in (k_new, v_new):
                    new[a, t[f // page], h, f % page] = new[a, t[w // page], h, w % page]
                d = torch.arange(len(where), device=DEVICE)
                mass_new[a, t[d // page], h, d % page] = torch.from_numpy(m[where]).to(DEVICE, torch.float32)
                pos_new[a, t[d // page], h, d % page] = torch.from_numpy(p[where]).to(DEVICE)
    return k, v, mass_out, pos_out, s["lens"].clamp(max=keep)


def exact(case, seed):
    """The operator's definition in 64 bits, one sequence (and head) at a time, on the inputs of prepare(case, seed)."""
    global own
    mine, own = own, False
    try:
        return globals()["_exact_" + case["op"]](prepare(case, seed))
    finally:
        own = mine
