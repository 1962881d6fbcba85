"""Token-tree calls on the GPU against their restatement in 64 bits."""
import itertools

import numpy as np
import pytest
import torch

import tree_util as tu

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def st():
    import speculative_decoding_token_gb300 as sv
    h = sv.SpecTree(64, max_moves=1 << 20)
    yield h
    assert h.device_status() == 0
    h.close()


def near(got, want, tol):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    bad = ((got - want).abs() > tol) & ~torch.isnan(want)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, at most " \
                          f"{float(((got - want).abs() / tol.clamp(min=1e-300)).nan_to_num().max()):.3g} tolerances"


def run_attention(st, bt, scale=None, **kw):
    scale = bt.d ** -0.5 if scale is None else scale
    bt.upload()
    out = torch.full_like(bt.dq, float("nan"))
    lse = torch.full((bt.rows, bt.heads), float("nan"), device=bt.device)
    st.attention(bt.dq, bt.cache, bt.tree, bt.dlens, scale=scale, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check_attention(st, bt, scale=None):
    out, lse = run_attention(st, bt, scale)
    want = tu.attention(bt, bt.d ** -0.5 if scale is None else scale)
    near(out, want[0], want[2])
    near(lse, want[1], want[3])


ATTENTION = {
    # lens, nodes, heads, kv heads, head size, page, dtype, options
    "one token": ([0], [1], 1, 1, 128, 8, BF16, {}),
    "first step": ([0, 0, 5], [3, 8, 0], 4, 2, 64, 8, FP16, {}),
    "single row long": ([1000], [1], 8, 8, 128, 16, BF16, {}),
    "tile edges": ([126, 127, 128, 129, 255, 256, 257], [1, 2, 3, 1, 2, 1, 4], 8, 2, 128, 16, BF16, {}),
    "odd group": ([37, 300, 511], [9, 4, 13], 14, 2, 64, 24, FP16, {"token_major": True}),
    "five a head": ([200, 64], [26, 7], 5, 1, 128, 48, FP16, {}),
    "128 rows": ([333], [16], 16, 2, 128, 64, BF16, {}),
    "129 rows": ([333, 77], [43, 1], 3, 1, 128, 40, BF16, {"token_major": True}),
    "256 rows": ([640], [32], 8, 1, 64, 128, BF16, {}),
    "many rows": ([190, 0], [128, 128], 16, 2, 128, 256, BF16, {"kind": "random"}),
    "deep chain": ([100, 1], [128, 100], 2, 2, 64, 8, BF16, {"kind": "chain"}),
    "star": ([100], [64], 4, 1, 128, 32, FP16, {"kind": "star"}),
    "some idle": ([50, 0, 700, 3], [0, 0, 5, 1], 8, 4, 128, 32, BF16, {}),
    "sharp": ([900, 400], [6, 20], 4, 2, 128, 16, BF16, {"sharp": 12.0}),
    "flat": ([900, 400], [6, 20], 4, 2, 64, 16, FP16, {"sharp": 0.0}),
    "many short": ([i * 7 % 90 for i in range(60)], [1 + i % 5 for i in range(60)], 4, 2, 64, 16, BF16, {}),
    "page above tile": ([500, 1030], [3, 9], 4, 4, 64, 1040, BF16, {}),
    "one head for all": ([260, 9], [5, 3], 64, 1, 128, 16, BF16, {}),
    "more heads than a tile's rows": ([150], [2], 300, 1, 64, 16, BF16, {}),
    "blocks of rows": ([400, 20, 300, 0, 700], [64, 3, 33, 0, 128], 16, 2, 64, 16, FP16, {}),
}


@pytest.mark.parametrize("name", ATTENTION)
def test_attention(st, name):
    *args, kw = ATTENTION[name]
    check_attention(st, tu.Batch(*args, seed=len(name), **kw))


@pytest.mark.parametrize("d,page,G,dtype", [(d, p, G, t) for (d, p), G, t in itertools.product(
    [(64, 8), (128, 56), (128, 128)], [1, 2, 3, 7, 8, 16], [BF16, FP16])])
def test_attention_layouts(st, d, page, G, dtype):
    rng = np.random.default_rng(d + page + G)
    lens, nodes = rng.integers(0, 700, 3).tolist(), rng.integers(1, 30, 3).tolist()
    check_attention(st, tu.Batch(lens, nodes, 2 * G, 2, d, page, dtype, seed=G, token_major=G % 2 == 1))


def test_attention_long_context_split(st):
    """Keys of one row split over every SM; scores whose maximum keeps rising."""
    bt = tu.Batch([30011], [2], 2, 1, 128, 64, BF16, seed=3)
    ramp = torch.linspace(0.01, 3.0, bt.k.shape[1] * bt.page).view(1, bt.k.shape[1], 1, bt.page, 1)
    ordered = torch.empty_like(ramp)
    for i, pg in enumerate(bt.table[0]):
        ordered[0, pg] = ramp[0, i]
    bt.k = (bt.k.float() * ordered).to(BF16)
    check_attention(st, bt)


def test_attention_of_many_sequences():
    """More sequences than threads of a CTA."""
    import speculative_decoding_token_gb300 as sv
    h = sv.SpecTree(700)
    check_attention(h, tu.Batch([i % 23 for i in range(700)], [i % 3 for i in range(700)], 2, 1, 64, 8, BF16, seed=4))
    assert h.device_status() == 0
    h.close()


def test_attention_shared_pages_and_layer_views(st):
    """Two sequences whose tables share a prefix's pages, one layer of a pool that holds k and v of several layers side by
    side, and a page table with columns to spare."""
    import speculative_decoding_token_gb300 as sv
    bt = tu.Batch([100, 90], [3, 6], 4, 2, 64, 16, BF16, seed=21, poison=False)
    bt.table[1, :4] = bt.table[0, :4]
    bt.upload()
    pool = torch.full((3, 2, *bt.dk.shape), float("nan"), dtype=BF16, device="cuda")  # layers, k and v
    pool[1, 0], pool[1, 1] = bt.dk, bt.dv
    wide = torch.full((2, 40), -9, dtype=torch.int32, device="cuda")
    wide[:, : bt.table.shape[1]] = bt.dev(bt.table)
    cache = sv.KVCache(pool[1, 0], pool[1, 1], wide)
    out, lse = st.attention(bt.dq, cache, bt.tree, bt.dlens)
    want = tu.attention(bt, 0.125)
    real = ~torch.isnan(want[1][:, 0])
    near(out[real.cuda()], want[0][real], want[2][real])
    near(lse[real.cuda()], want[1][real], want[3][real])


def test_attention_repeats_bit_for_bit(st):
    """Whatever ran before on the SMs: the Q tile's rows past a tree's hold what the last call left there."""
    bt = tu.Batch([20000, 9000, 3], [26, 16, 9], 8, 2, 128, 16, FP16, seed=13)
    other = tu.Batch([700, 300], [32, 30], 8, 2, 128, 16, FP16, seed=14, sharp=40.0).upload()
    first = run_attention(st, bt)
    for i in range(8):
        if i % 2:
            st.attention(other.dq, other.cache, other.tree, other.dlens)
        again = run_attention(st, bt)
        assert torch.equal(first[0].nan_to_num(9.0), again[0].nan_to_num(9.0))
        assert torch.equal(first[1].nan_to_num(9.0), again[1].nan_to_num(9.0))


def test_calls_of_one_handle_back_to_back():
    """Attention and eviction of several batches through one handle's workspace, with nothing between the calls."""
    import speculative_decoding_token_gb300 as sv
    h = sv.SpecTree(8, max_moves=1 << 16)
    bts = [tu.Batch([3000 + 900 * i, 77], [5 + 9 * i, 20], 8, 2, 128, 16, BF16, seed=40 + i, poison=False) for i in range(3)]
    rng, budget = np.random.default_rng(3), 600
    for bt in bts:
        shape = bt.k.shape[:-1]
        mass = torch.rand(shape, generator=bt.gen)
        pos, seen = make_positions(rng, bt, shape)
        bt.upload(mass=mass, pos=pos)
        bt.att = (torch.zeros_like(bt.dq), torch.zeros(bt.rows, bt.heads, device="cuda"))
        bt.ev = (torch.zeros_like(bt.dmass), torch.zeros_like(bt.dpos), torch.zeros(2, dtype=torch.int32, device="cuda"))
        bt.dseen = bt.dev(seen, torch.int32)

    def attend(bt):
        h.attention(bt.dq, bt.cache, bt.tree, bt.dlens, out=bt.att[0], lse=bt.att[1])

    def evict(bt):
        h.evict(bt.cache, bt.dlens, bt.dseen, budget, sink=4, recent=50, mass_out=bt.ev[0], pos_out=bt.ev[1],
                new_lens=bt.ev[2])

    want = []
    for bt in bts:
        keep = bt.dk.clone(), bt.dv.clone()
        attend(bt)
        evict(bt)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (*bt.att, *bt.ev, bt.dk, bt.dv)])
        bt.dk.copy_(keep[0]), bt.dv.copy_(keep[1])
        bt.keep = keep
    for _ in range(20):
        for bt in bts:
            for t in (*bt.att, *bt.ev):
                t.zero_()
            bt.dk.copy_(bt.keep[0]), bt.dv.copy_(bt.keep[1])
        for bt in bts * 2:
            attend(bt)
        for bt in bts:
            evict(bt)
        for bt, w in zip(bts, want):
            for t, x in zip((*bt.att, *bt.ev, bt.dk, bt.dv), w):
                assert torch.equal(t, x)
    assert h.device_status() == 0
    h.close()


def test_attention_scale(st):
    check_attention(st, tu.Batch([300], [9], 4, 2, 64, 16, BF16, seed=8), scale=0.7)


def test_attention_strided_rows(st):
    """q and out as slices of wider buffers."""
    bt = tu.Batch([140, 33], [5, 12], 6, 2, 64, 16, BF16, seed=5)
    bt.upload()
    wide = torch.zeros(bt.rows, 10, 3 * 64, dtype=BF16, device="cuda")
    wide[:, 2:8, 64:128] = bt.dq
    sink = torch.full((bt.rows, 2, 6, 64), 7.0, dtype=BF16, device="cuda")
    out, lse = st.attention(wide[:, 2:8, 64:128], bt.cache, bt.tree, bt.dlens, out=sink[:, 1])
    want = tu.attention(bt, 0.125)
    real = ~torch.isnan(want[1][:, 0])
    near(out[real.cuda()], want[0][real], want[2][real])
    assert bool((sink[:, 0] == 7.0).all()) and bool((sink[:, 1][~real.cuda()] == 7.0).all())


def test_attention_infinite_values_stay_with_their_nodes(st):
    """A node whose value overflowed: its descendants see it, no other row does."""
    bt = tu.Batch([120], [40], 4, 1, 128, 16, BF16, seed=11, kind="random")
    j = 7
    pg, at = bt.slots(0, 160)
    bt.v[0, pg[120 + j], 0, at[120 + j], 3] = float("inf")
    bt.v[0, pg[120 + j], 0, at[120 + j], 60] = float("nan")
    bt.v[0, pg[120 + 9], 0, at[120 + 9], 60] = float("-inf")
    bt.k[0, pg[120 + 11], 0, at[120 + 11], 5] = float("nan")
    out, lse = run_attention(st, bt)
    want = tu.attention(bt, bt.d ** -0.5)
    near(lse, want[1], want[3])
    fin = torch.isfinite(want[0])
    got = out.double().cpu()
    assert torch.equal(torch.isfinite(got), fin)
    assert torch.equal(got[~fin & ~torch.isnan(want[0])], want[0][~fin & ~torch.isnan(want[0])])
    assert bool(((got - want[0]).abs() <= want[2])[fin].all())
    hit = [r for r in range(40) if j in tu.chain(bt.parent[0], r)]
    assert 0 < len(hit) < 40


def test_attention_bad_input_marks_its_sequence(st):
    import speculative_decoding_token_gb300 as sv
    good = tu.Batch([60, 70, 80, 90, 100, 30], [4, 5, 6, 7, 8, 2], 4, 2, 64, 16, BF16, seed=2)
    bits = sv.STATUS_BITS
    for b, change, bit in [
        (0, lambda t: t.nodes.__setitem__(0, 999), "bad_tree"),
        (0, lambda t: t.nodes.__setitem__(0, -1), "bad_tree"),
        (1, lambda t: t.parent.__setitem__((1, 3), 3), "bad_tree"),
        (1, lambda t: t.parent.__setitem__((1, 0), 0), "bad_tree"),
        (2, lambda t: t.row_off.__setitem__(2, t.rows - 1), "bad_row"),
        (2, lambda t: t.row_off.__setitem__(2, -1), "bad_row"),
        (3, lambda t: t.lens.__setitem__(3, 10 ** 6), "bad_cache"),
        (3, lambda t: t.lens.__setitem__(3, -5), "bad_cache"),
        (4, lambda t: t.table.__setitem__((4, 2), t.k.shape[1]), "bad_cache"),
        (4, lambda t: t.table.__setitem__((4, 0), -1), "bad_cache"),
    ]:
        bt = tu.Batch([60, 70, 80, 90, 100, 30], [4, 5, 6, 7, 8, 2], 4, 2, 64, 16, BF16, seed=2)
        change(bt)
        out, lse = run_attention(st, bt)
        assert st.device_status() == bits[bit]
        want = tu.attention(good, 0.125)
        o, n = good.row_off[b], good.nodes[b]
        for w in want[:2]:
            w[o: o + n] = float("nan")
        near(out, want[0], want[2])
        near(lse, want[1], want[3])


def test_attention_bad_pages_under_the_tree(st):
    """Pages of nodes that lie outside the pool, in tiles whose shared memory still holds other sequences' NaN (slots past
    their trees): nothing is read there, the rows are NaN, the sequences between them are right."""
    import speculative_decoding_token_gb300 as sv
    B = 400
    lens, nodes = [192 if b % 2 == 0 else 200 for b in range(B)], [1 if b % 2 == 0 else 8 for b in range(B)]
    bt = tu.Batch(lens, nodes, 4, 2, 128, 16, BF16, seed=71)
    want = tu.attention(bt, bt.d ** -0.5)
    for b in range(1, B, 2):
        bt.table[b, 12] = (-1, -(2 ** 31), bt.k.shape[1], 2 ** 31 - 1)[b // 2 % 4]
        for w in want[:2]:
            w[bt.row_off[b]: bt.row_off[b] + nodes[b]] = float("nan")
    h = sv.SpecTree(B)
    out, lse = run_attention(h, bt)
    assert h.device_status() == sv.STATUS_BITS["bad_cache"]
    near(out, want[0], want[2])
    near(lse, want[1], want[3])


# ---------------------------------------------------------------------------
# verify

def make_verify(rng, B, T, V, dtype, agree=0.75, levels=None):
    nodes = rng.integers(1, T + 1, B)
    nodes[0] = T
    row_off = np.concatenate([[2], 2 + np.cumsum(nodes)[:-1]])
    rows = 2 + int(nodes.sum()) + 1
    parent = np.full((B, T), -1)
    tokens = rng.integers(0, V, (B, T))
    stride = -(-V // 8) * 8
    x = torch.from_numpy(rng.standard_normal((rows, stride)).astype(np.float32) if levels is None
                         else rng.integers(0, levels, (rows, stride)).astype(np.float32))
    target = x.to(dtype)[:, :V]
    for b in range(B):
        parent[b, : nodes[b]] = tu.random_tree(rng, nodes[b])
        for j in range(1, nodes[b]):
            if rng.random() < agree:
                tokens[b, j] = int(torch.argmax(target[row_off[b] + parent[b, j]].double()))
    return nodes, row_off, parent, tokens, target


def run_verify(st, nodes, row_off, parent, tokens, target):
    import speculative_decoding_token_gb300 as sv
    dev = lambda x, t: torch.as_tensor(np.asarray(x)).to("cuda", t)  # noqa: E731
    tree = sv.TokenTree(dev(row_off, torch.int64), dev(nodes, torch.int32), dev(parent, torch.int32),
                        dev(tokens, torch.int32))
    wide = torch.zeros(target.shape[0], -(-target.shape[1] // 8) * 8, dtype=target.dtype, device="cuda")
    wide[:, : target.shape[1]] = target.cuda()
    wide[:, target.shape[1]:] = float("inf")  # past V: never read as a logit
    return [x.cpu().numpy() for x in st.verify(tree, wide[:, : target.shape[1]])]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("B,T,V,levels", [(1, 1, 1, None), (3, 5, 7, 2), (1, 16, 32000, None), (9, 128, 1001, None),
                                          (40, 33, 999, 3), (4, 20, 50257, None), (2, 8, 8, 1), (5, 64, 64, 4)])
def test_verify(st, B, T, V, levels, dtype):
    case = make_verify(np.random.default_rng(B + T + V), B, T, V, dtype, levels=levels)
    got = run_verify(st, *case)
    want = tu.verify(case[2], case[0], case[3], case[1], case[4])
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_verify_special_logits(st):
    """-inf rows, +inf, and NaN off the path are answered; NaN on the path marks the sequence; idle sequences."""
    import speculative_decoding_token_gb300 as sv
    rng = np.random.default_rng(4)
    nodes, row_off, parent, tokens, target = make_verify(rng, 6, 12, 500, torch.float32, agree=0.0)
    nodes[:] = [12, 12, 12, 12, 0, 12]
    row_off = np.array([0, 12, 24, 36, 47, 47])
    target = torch.randn(59, 500)
    parent[:] = tu.random_tree(rng, 12, "star")
    tokens[:, 1:] = np.arange(11) + 3
    target[0] = float("-inf")                    # argmax 0: no child
    target[12, 7] = float("inf")                 # token 7: child 5
    target[12 + 5] = float("-inf")
    target[24, 4], target[24 + 1] = 50.0, float("nan")   # token 4: child 2; NaN in a sibling's row
    target[36, 499] = float("nan")
    target[47, 6], target[47 + 4, 0] = 50.0, float("nan")  # token 6: child 4, whose row is bad
    got = run_verify(st, nodes, row_off, parent, tokens, target)
    assert st.device_status() == sv.STATUS_BITS["bad_logit"]
    want = tu.verify(parent, nodes, tokens, row_off, target)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert got[0].tolist() == [0, 1, 1, -1, -1, -1]


def test_verify_bad_input(st):
    import speculative_decoding_token_gb300 as sv
    bits = sv.STATUS_BITS
    case = make_verify(np.random.default_rng(5), 5, 9, 300, BF16)
    want = tu.verify(case[2], case[0], case[3], case[1], case[4])
    for arg, at, value, bit in [(0, 0, 10, "bad_tree"), (0, 0, -3, "bad_tree"), (1, 0, -1, "bad_row"), (1, 0, 10 ** 9, "bad_row"),
                                (2, (0, 4), 4, "bad_tree"), (2, (0, 0), 1, "bad_tree"), (3, (0, 2), 300, "bad_token"),
                                (3, (0, 2), -1, "bad_token")]:
        bad = [x.copy() if isinstance(x, np.ndarray) else x for x in case]
        bad[arg][at] = value
        got = run_verify(st, *bad)
        assert st.device_status() == bits[bit]
        assert got[0][0] == -1 and (got[1][0] == -1).all() and (got[2][0] == -1).all()
        for g, w in zip(got, want):
            assert np.array_equal(g[1:], w[1:])


def test_verify_agrees_with_the_chain_verify(st):
    """A tree that is a chain gives what the greedy verify of that chain gives."""
    import speculative_decoding_token_gb300 as sv
    from speculative_decoding_token_gb300 import workload
    batch = workload.make_batch(1, device="cuda")
    h = sv.SpecVerify(batch.B, batch.gamma_max, batch.V)
    n, toks = h.verify_batch(batch, greedy=True)
    T = batch.gamma_max + 1
    parent = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(batch.B, 1)
    tokens = torch.cat([torch.zeros(batch.B, 1, dtype=torch.int32, device="cuda"), batch.draft_tokens], 1).contiguous()
    tree = sv.TokenTree(batch.p_row_off, batch.gamma + 1, parent, tokens)
    n2, toks2, _ = st.verify(tree, batch.target)
    assert torch.equal(n, n2) and torch.equal(toks, toks2)
    h.close()


# ---------------------------------------------------------------------------
# commit

def make_paths(rng, nodes, T):
    n, path = [], np.full((len(nodes), T), -1)
    for b, t in enumerate(nodes):
        walk = [0]
        while t and walk[-1] + 1 < t and rng.random() < 0.8:
            walk.append(min(t - 1, walk[-1] + int(rng.integers(1, 4))))
        n.append(len(walk) - 1 if t else -1)
        if t:
            path[b, : len(walk)] = walk
    return n, path


@pytest.mark.parametrize("layers,d,page,dtype,token_major", [(1, 64, 8, BF16, False), (3, 128, 16, FP16, True),
                                                             (2, 128, 24, BF16, False), (5, 64, 40, FP16, True)])
def test_commit(st, layers, d, page, dtype, token_major):
    rng = np.random.default_rng(layers + d)
    lens, nodes = rng.integers(0, 90, 7).tolist(), [1, 0, 128, 40, 9, 3, 17]
    bt = tu.Batch(lens, nodes, 3, 3, d, page, dtype, seed=page, layers=layers, token_major=token_major, poison=False)
    n, path = make_paths(rng, nodes, bt.T)
    mass = torch.rand(bt.k.shape[:-1], generator=bt.gen)
    pos = torch.randint(0, 99, bt.k.shape[:-1], generator=bt.gen, dtype=torch.int32)
    seen = rng.integers(0, 10 ** 6, 7)
    bt.upload(mass=mass, pos=pos)
    k, v, m, p = bt.k.clone(), bt.v.clone(), mass.clone(), pos.clone()
    for b in range(7):
        for i in range(n[b] + 1):
            (s_pg, s), (d_pg, at) = ((int(bt.table[b, x // page]), x % page) for x in (lens[b] + path[b, i], lens[b] + i))
            for old, new in ((bt.k, k), (bt.v, v)):
                new[:, d_pg, :, at] = old[:, s_pg, :, s]
            m[:, d_pg, :, at], p[:, d_pg, :, at] = 0.0, int(seen[b]) + i
    dn = bt.dev(n, torch.int32)
    new_lens, new_seen = st.commit(bt.cache, bt.dlens, dn, bt.dev(path, torch.int32), seen=bt.dev(seen, torch.int32))
    for got, want in ((bt.dk, k), (bt.dv, v), (bt.dmass, m), (bt.dpos, p)):
        assert torch.equal(got.cpu(), bt.one(want))
    assert new_lens.tolist() == [x + y + 1 for x, y in zip(lens, n)]
    assert new_seen.tolist() == [x + y + 1 for x, y in zip(seen.tolist(), n)]


def test_commit_without_positions(st):
    bt = tu.Batch([5, 9], [4, 6], 2, 2, 64, 8, BF16, poison=False).upload()
    path = bt.dev([[0, 2, 3, -1, -1, -1], [0, -1, -1, -1, -1, -1]], torch.int32)
    new_lens, new_seen = st.commit(bt.cache, bt.dlens, bt.dev([2, 0], torch.int32), path)
    assert new_lens.tolist() == [8, 10] and new_seen is None
    pg, at = bt.slots(0, 9)
    assert torch.equal(bt.dk.cpu()[pg[6:8], :, at[6:8]], bt.k[0][pg[7:9], :, at[7:9]])


def test_commit_bad_input(st):
    import speculative_decoding_token_gb300 as sv
    bits = sv.STATUS_BITS
    good = [[0, 2, 3, 4], [0, 1, 3, -1], [0, -1, -1, -1]]
    for b, i, value, bit in [(0, 1, 0, "bad_tree"), (0, 2, 1, "bad_tree"), (0, 3, 4, "bad_tree"), (0, 0, 1, "bad_tree"),
                             (1, 1, -1, "bad_tree"), ("n", 0, 4, "bad_tree"), ("len", 0, 1000, "bad_cache"),
                             ("len", 0, -1, "bad_cache"), ("table", 0, 10 ** 6, "bad_cache")]:
        bt = tu.Batch([5, 9, 20], [5, 5, 5], 2, 2, 64, 8, BF16, poison=False, seed=1)
        n, path = [3, 2, 0], [r[:] + [-1] for r in good]
        lens = bt.lens[:]
        path[0][3] = 4
        if b == "n":
            n[0] = 99
        elif b == "len":
            bt.lens[0] = lens[0] = value
        elif b == "table":
            bt.table[0, 0] = value
        else:
            path[b][i] = value
            if (b, i, value) == (0, 3, 4):
                path[0][3] = 5  # a node past the rows of the path
        bt.upload()
        new_lens, _ = st.commit(bt.cache, bt.dlens, bt.dev(n, torch.int32), bt.dev(path, torch.int32),
                                seen=bt.dev([7, 8, 9], torch.int32))
        assert st.device_status() == bits[bit], (b, i, value)
        bad = b if isinstance(b, int) else 0
        assert new_lens[bad] == lens[bad]
        pg, at = bt.slots(bad, 10) if bad else (None, None)
        others = [x for x in range(3) if x != bad]
        assert [int(new_lens[x]) for x in others] == [lens[x] + n[x] + 1 for x in others]
        if b != "table" and bad == 0 and lens[0] == 5:
            pg, at = bt.slots(0, 10)
            assert torch.equal(bt.dk.cpu()[pg, :, at], bt.k[0][pg, :, at])


# ---------------------------------------------------------------------------
# accumulated weight

@pytest.mark.parametrize("d,G,page,dtype,lens,nodes", [
    (64, 1, 8, BF16, [0, 1, 77], [1, 4, 9]),
    (128, 4, 16, BF16, [127, 128, 129, 1000], [8, 1, 0, 26]),
    (64, 7, 24, FP16, [300, 2], [30, 11]),
    (128, 8, 128, BF16, [700], [64]),
    (128, 5, 56, FP16, [255, 256, 257], [128, 3, 40]),
    (64, 16, 1040, BF16, [1100, 12], [20, 128]),
])
def test_accumulate(st, d, G, page, dtype, lens, nodes):
    rng = np.random.default_rng(d + G)
    bt = tu.Batch(lens, nodes, 2 * G, 2, d, page, dtype, seed=G, token_major=G % 2 == 1)
    n, path = make_paths(rng, nodes, bt.T)
    if 128 in nodes:  # the whole tree accepted
        b = nodes.index(128)
        n[b], path[b] = 127, np.arange(128)
    mass = torch.rand(bt.k.shape[:-1], generator=bt.gen)
    bt.upload(mass=mass)
    z = torch.rand(bt.rows, bt.heads, generator=bt.gen) * 3 + 4
    scale = d ** -0.5
    st.accumulate(bt.dq, z.cuda(), bt.cache, bt.tree, bt.dlens, bt.dev(n, torch.int32), bt.dev(path, torch.int32))
    want, tol = tu.accumulate(bt, mass[0], z, n, path, scale)
    near(bt.dmass, want, tol)


def test_accumulate_of_attention_sums_to_its_rows(st):
    """With the attention's own lse every accepted row hands out a weight of one."""
    bt = tu.Batch([500, 90], [8, 8], 8, 2, 128, 16, BF16, seed=6, kind="chain")
    bt.upload(mass=torch.zeros(bt.k.shape[:-1]))
    _, lse = st.attention(bt.dq, bt.cache, bt.tree, bt.dlens)
    n = torch.tensor([7, 3], dtype=torch.int32, device="cuda")
    path = torch.arange(8, dtype=torch.int32, device="cuda").repeat(2, 1)
    st.accumulate(bt.dq, lse, bt.cache, bt.tree, bt.dlens, n, path)
    total = [float(bt.dmass[torch.as_tensor(bt.table[b, : -(-(bt.lens[b] + 8) // 16)]).long().cuda()].double().sum())
             for b in range(2)]
    # 8 heads, n + 1 rows each; lse and every weight are good to 1e-5
    assert abs(total[0] - 64) < 64e-5 and abs(total[1] - 32) < 32e-5


def test_accumulate_bad_input(st):
    import speculative_decoding_token_gb300 as sv
    bits = sv.STATUS_BITS
    for what, bit in [("n", "bad_tree"), ("path", "bad_tree"), ("row", "bad_row"), ("len", "bad_cache"), ("page", "bad_cache"),
                      ("nodes", "bad_tree")]:
        bt = tu.Batch([50, 70], [5, 5], 2, 1, 64, 8, BF16, seed=1)
        good = tu.Batch([50, 70], [5, 5], 2, 1, 64, 8, BF16, seed=1)
        n, path = [2, 3], np.array([[0, 1, 4, -1, -1], [0, 2, 3, 4, -1]])
        want, tol = tu.accumulate(good, torch.zeros(bt.k.shape[1:-1]), torch.full((bt.rows, 2), 5.0), [-1, 3], path, 0.125)
        if what == "n":
            n[0] = 5
        elif what == "path":
            path[0, 2] = 1
        elif what == "row":
            bt.row_off[0] = bt.rows
        elif what == "len":
            bt.lens[0] = 10 ** 7
        elif what == "page":
            bt.table[0, 3] = -2
        else:
            bt.nodes[0] = 2
        bt.upload(mass=torch.zeros(bt.k.shape[:-1]))
        st.accumulate(bt.dq, torch.full((bt.rows, 2), 5.0, device="cuda"), bt.cache, bt.tree, bt.dlens,
                      bt.dev(n, torch.int32), bt.dev(path, torch.int32))
        assert st.device_status() == bits[bit], what
        near(bt.dmass, want, tol)


# ---------------------------------------------------------------------------
# eviction

def make_positions(rng, bt, shape):
    """Rising positions with gaps in every sequence, and what comes next."""
    pos, seen = torch.zeros(shape, dtype=torch.int32), []
    for b in range(bt.B):
        L = bt.lens[b]
        seen.append(2 * L + 5)
        for a in range(bt.layers):
            for g in range(bt.kv_heads):
                p = np.sort(rng.choice(2 * L + 5, L, replace=False))
                p = rng.permutation(p) if b % 2 else p
                pg, at = bt.slots(b, L)
                pos[a, pg, g, at] = torch.as_tensor(p.astype(np.int32))
    return pos, seen


def expected_evict(bt, mass, pos, seen, budget, sink, recent, mass_out, pos_out):
    k, v, m, p = bt.k.clone(), bt.v.clone(), mass_out.clone(), pos_out.clone()
    for b in range(bt.B):
        pg, at = bt.slots(b, bt.lens[b])
        for a in range(bt.layers):
            for g in range(bt.kv_heads):
                src = tu.keep_slots(mass[a, pg, g, at].numpy().astype(np.float64), pos[a, pg, g, at].numpy(), seen[b],
                                    budget, sink, recent)
                to = np.arange(len(src))
                sp, sa, dp, da = pg[src], at[src], pg[to], at[to]
                for old, new in ((bt.k, k), (bt.v, v), (mass, m), (pos, p)):
                    new[a, dp, g, da] = old[a, sp, g, sa]
    return k, v, m, p


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layers,d,page,dtype,lens,budget,sink,recent,kind", [
    (1, 64, 8, BF16, [0, 1, 15, 16, 17, 100], 16, 2, 4, "normal"),
    (3, 128, 16, FP16, [300, 40, 90], 64, 4, 16, "zeros"),
    (1, 128, 24, BF16, [1500, 2047, 1], 1000, 0, 0, "normal"),
    (2, 64, 40, BF16, [500, 400], 1, 0, 1, "normal"),
    (1, 64, 16, FP16, [700, 650], 512, 256, 256, "zeros"),
    (1, 128, 16, BF16, [300, 301], 299, 1, 1, "special"),
    (1, 64, 32, BF16, [5000, 33], 4096, 4, 100, "narrow"),
    (1, 64, 8, BF16, [90, 60], 200, 4, 100, "normal"),
])
def test_evict(st, layers, d, page, dtype, lens, budget, sink, recent, kind, in_place):
    rng = np.random.default_rng(budget + layers)
    bt = tu.Batch(lens, [0] * len(lens), 2, 2, d, page, dtype, seed=d, layers=layers, poison=False, token_major=layers == 2)
    shape = bt.k.shape[:-1]
    mass = torch.randn(shape, generator=bt.gen).exp()
    if kind == "zeros":
        mass[torch.rand(shape, generator=bt.gen) < 0.7] = 0.0
        mass[torch.rand(shape, generator=bt.gen) < 0.1] = -0.0
    elif kind == "narrow":
        mass = 1.0 + torch.randint(0, 5, shape, generator=bt.gen) * 2.0 ** -23
    elif kind == "special":
        pick = torch.rand(shape, generator=bt.gen)
        mass[pick < 0.2], mass[pick > 0.9], mass[(pick > 0.4) & (pick < 0.5)] = float("nan"), float("inf"), -1.0
    pos, seen = make_positions(rng, bt, shape)
    bt.upload(mass=mass, pos=pos)
    m0, p0 = (mass, pos) if in_place else (torch.full(shape, 3.0), torch.full(shape, -9, dtype=torch.int32))
    dm, dp = (bt.dmass, bt.dpos) if in_place else (bt.dev(bt.one(m0)), bt.dev(bt.one(p0)))
    _, _, new_lens = st.evict(bt.cache, bt.dlens, bt.dev(seen, torch.int32), budget, sink=sink, recent=recent,
                              mass_out=dm, pos_out=dp)
    k, v, m, p = expected_evict(bt, mass, pos, seen, budget, sink, recent, m0, p0)
    assert new_lens.tolist() == [min(x, budget) for x in lens]
    for got, want in ((bt.dk, k), (bt.dv, v), (dp, p)):
        assert torch.equal(got.cpu(), bt.one(want))
    assert torch.equal(dm.cpu().nan_to_num(77.0), bt.one(m).nan_to_num(77.0))


def test_evict_more_slots_than_shared_memory_holds():
    import speculative_decoding_token_gb300 as sv
    rng = np.random.default_rng(2)
    lens, budget = [50011, 49153, 7], 30000
    bt = tu.Batch(lens, [0, 0, 0], 1, 1, 64, 256, BF16, seed=2, poison=False)
    shape = bt.k.shape[:-1]
    mass = torch.randint(0, 4000, shape, generator=bt.gen).float()  # many ties
    pos, seen = make_positions(rng, bt, shape)
    bt.upload(mass=mass, pos=pos)
    h = sv.SpecTree(3, max_moves=3 * 30000)
    out = torch.zeros_like(bt.dmass)
    _, p, new_lens = h.evict(bt.cache, bt.dlens, bt.dev(seen, torch.int32), budget, sink=4, recent=100, mass_out=out)
    want = expected_evict(bt, mass, pos, seen, budget, 4, 100, torch.zeros(shape), pos)
    assert new_lens.tolist() == [30000, 30000, 7] and h.device_status() == 0
    for got, w in ((bt.dk, want[0]), (bt.dv, want[1]), (out, want[2]), (p, want[3])):
        assert torch.equal(got.cpu(), w[0])
    h.close()


def test_evict_bad_input(st):
    import speculative_decoding_token_gb300 as sv
    for change in (lambda t: t.lens.__setitem__(0, -4), lambda t: t.lens.__setitem__(0, 10 ** 8),
                   lambda t: t.table.__setitem__((0, 2), t.k.shape[1])):
        bt = tu.Batch([60, 50], [0, 0], 1, 1, 64, 8, BF16, poison=False)
        shape = bt.k.shape[:-1]
        mass = torch.rand(shape, generator=bt.gen)
        pos, seen = make_positions(np.random.default_rng(1), bt, shape)
        want = expected_evict(bt, mass, pos, seen, 20, 2, 5, mass, pos)
        change(bt)
        bt.upload(mass=mass, pos=pos)
        _, _, new_lens = st.evict(bt.cache, bt.dlens, bt.dev(seen, torch.int32), 20, sink=2, recent=5)
        assert st.device_status() == sv.STATUS_BITS["bad_cache"]
        assert new_lens.tolist() == [bt.lens[0], 20]
        pg, at = bt.slots(1, 50)
        assert torch.equal(bt.dk.cpu()[pg, :, at], want[0][0][pg, :, at])
        rest = torch.ones(bt.k.shape[1], dtype=torch.bool)
        rest[pg] = False
        assert torch.equal(bt.dk.cpu()[rest], bt.k[0][rest]) and torch.equal(bt.dmass.cpu()[rest], mass[0][rest])


# ---------------------------------------------------------------------------
# refusals, streams, graphs

def test_refusals(st):
    import speculative_decoding_token_gb300 as sv
    bt = tu.Batch([20], [4], 4, 2, 64, 8, BF16, poison=False)
    shape = bt.k.shape[:-1]
    bt.upload(mass=torch.zeros(shape), pos=torch.zeros(shape, dtype=torch.int32))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, n, path = bt.dlens, i32(0), torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    att = lambda q=bt.dq, cache=bt.cache, tree=bt.tree, ln=lens, **kw: st.attention(q, cache, tree, ln, **kw)  # noqa: E731
    for bad in (lambda: att(q=bt.dq.float()), lambda: att(q=bt.dq[:, :3]), lambda: att(q=bt.dq[:, :, :32]),
                lambda: att(ln=lens.long()), lambda: att(ln=i32(1, 2)), lambda: att(ln=lens.cpu()),
                lambda: att(out=torch.empty_like(bt.dq)[:, :2]), lambda: att(lse=torch.empty(1, 4, device="cuda")),
                lambda: st.verify(bt.tree, bt.dq[0].float()),  # the tree has no tokens
                lambda: st.commit(bt.cache, lens, n, path),  # positions without `seen`
                lambda: st.evict(bt.cache, lens, lens, 4, mass_out=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(bt.rows, 4, 65, dtype=BF16, device="cuda")[:, :, :64]
    for bad, rc in ((lambda: att(scale=0.0), -1), (lambda: att(scale=-1.0), -1), (lambda: att(scale=float("nan")), -1),
                    (lambda: att(scale=float("inf")), -1), (lambda: att(q=odd), -1),
                    (lambda: st.commit(bt.cache, lens, n, path, seen=i32(3), new_lens=lens), -1),
                    (lambda: st.commit(bt.cache, lens, n, path, seen=i32(3), new_lens=n), -1),
                    (lambda: st.evict(bt.cache, lens, i32(3), 4, sink=3, recent=2), -1),
                    (lambda: st.evict(bt.cache, lens, i32(3), 0), -1),
                    (lambda: st.evict(bt.cache, lens, i32(3), 4, new_lens=lens), -1),
                    (lambda: sv.SpecTree(1).evict(bt.cache, lens, i32(3), 4), -6),
                    (lambda: sv.SpecTree(0), -1), (lambda: sv.SpecTree(1, max_moves=-1), -1)):
        with pytest.raises(sv.SpecVerifyError) as e:
            bad()
        assert e.value.rc == rc
    with pytest.raises(sv.SpecVerifyError):
        big = tu.Batch([1, 1], [1, 1], 1, 1, 64, 8, BF16).upload()
        sv.SpecTree(1).attention(big.dq, big.cache, big.tree, big.dlens)
    k = bt.dk
    for bad in (lambda: sv.KVCache(k.float(), k.float(), bt.cache.page_table), lambda: sv.KVCache(k, k[:1], bt.cache.page_table),
                lambda: sv.KVCache(k[..., :32], k[..., :32], bt.cache.page_table),
                lambda: sv.KVCache(k[:, :, :4], k[:, :, :4], bt.cache.page_table),
                lambda: sv.KVCache(k, k, bt.cache.page_table.long()), lambda: sv.KVCache(k, k, bt.cache.page_table[0]),
                lambda: sv.KVCache(k, k, bt.cache.page_table, mass=torch.zeros(shape[1:], dtype=torch.float64, device="cuda")),
                lambda: sv.KVCache(k.cpu(), k.cpu(), bt.cache.page_table.cpu()),
                lambda: sv.TokenTree(bt.tree.row_off, bt.tree.nodes, bt.tree.parent[:, :0]),
                lambda: sv.TokenTree(bt.tree.row_off.int(), bt.tree.nodes, bt.tree.parent),
                lambda: sv.TokenTree(bt.tree.row_off, bt.tree.nodes, bt.tree.parent.repeat(1, 40)),
                lambda: sv.TokenTree(bt.tree.row_off, bt.tree.nodes, bt.tree.parent, bt.tree.parent.long())):
        with pytest.raises(ValueError):
            bad()
    assert st.device_status() == 0


def test_attention_refuses_an_expanded_output_and_takes_an_expanded_query(st):
    import speculative_decoding_token_gb300 as sv
    bt = tu.Batch([40, 7], [5, 3], 4, 2, 64, 8, BF16, seed=6)
    bt.q = bt.q[:1, :1].expand(bt.rows, 4, 64).contiguous()
    want = tu.attention(bt, 0.125)
    bt.upload()
    one = bt.dq[:1, :1]
    for out in (torch.zeros_like(bt.dq[:1]).expand(bt.rows, -1, -1), torch.zeros_like(bt.dq[:, :1]).expand(-1, 4, -1)):
        with pytest.raises(sv.SpecVerifyError) as e:
            st.attention(bt.dq, bt.cache, bt.tree, bt.dlens, out=out)
        assert e.value.rc == -1 and not bool(out.any())
    out, lse = torch.full_like(bt.dq, float("nan")), torch.full((bt.rows, 4), float("nan"), device="cuda")
    st.attention(one.expand(bt.rows, 4, 64), bt.cache, bt.tree, bt.dlens, out=out, lse=lse)
    near(out, want[0], want[2])
    near(lse, want[1], want[3])


def test_a_handle_too_large_leaves_no_error_behind(st):
    import speculative_decoding_token_gb300 as sv
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.SpecTree(1, max_moves=1 << 36)  # three lists of 256 GiB
    assert e.value.rc == sv.ERR_OOM
    assert float(torch.ones(8, device="cuda").sum()) == 8.0  # a launch that checks for errors before it


def test_empty_batch(st):
    import speculative_decoding_token_gb300 as sv
    bt = tu.Batch([3], [2], 2, 1, 64, 8, BF16, poison=False)
    shape = bt.k.shape[:-1]
    bt.upload(mass=torch.zeros(shape), pos=torch.zeros(shape, dtype=torch.int32))
    none = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = sv.KVCache(bt.dk, bt.dv, none(0, 4), mass=bt.dmass, pos=bt.dpos)
    tree = sv.TokenTree(none(0).long(), none(0), none(0, 4), none(0, 4))
    out, lse = st.attention(bt.dq, cache, tree, none(0))
    n, toks, path = st.verify(tree, torch.zeros(0, 8, device="cuda"))
    a, b = st.commit(cache, none(0), none(0), none(0, 4), seen=none(0))
    st.accumulate(bt.dq, lse, cache, tree, none(0), none(0), none(0, 4))
    _, _, c = st.evict(cache, none(0), none(0), 4)
    assert [x.numel() for x in (n, toks, path, a, b, c)] == [0] * 6
    assert st.device_status() == 0


def test_attention_on_another_stream_and_in_graphs(st):
    """Two handles' captured calls replayed side by side, and an eager call on a side stream, agree bit for bit."""
    import speculative_decoding_token_gb300 as sv
    bts = [tu.Batch([3000 + i, 900], [8, 20], 8, 2, 128, 16, BF16, seed=i).upload() for i in range(2)]
    want = [st.attention(b.dq, b.cache, b.tree, b.dlens) for b in bts]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = st.attention(bts[0].dq, bts[0].cache, bts[0].tree, bts[0].dlens, stream=side)
    side.synchronize()
    real = ~torch.isnan(tu.attention(bts[0], bts[0].d ** -0.5)[1][:, 0]).cuda()
    assert torch.equal(got[0][real], want[0][0][real]) and torch.equal(got[1][real], want[0][1][real])
    handles, graphs, outs = [], [], []
    for b in bts:
        h = sv.SpecTree(4)
        out, lse = torch.zeros_like(b.dq), torch.zeros(b.rows, b.heads, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h.attention(b.dq, b.cache, b.tree, b.dlens, out=out, lse=lse)
        handles.append(h), graphs.append(g), outs.append((out, lse))
    streams = [torch.cuda.Stream() for _ in bts]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0][real], want[i][0][real]) and torch.equal(outs[i][1][real], want[i][1][real])
    # the graph reads what its buffers hold now
    bts[0].dlens.copy_(torch.tensor([1500, 10], dtype=torch.int32))
    graphs[0].replay()
    now = st.attention(bts[0].dq, bts[0].cache, bts[0].tree, bts[0].dlens)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0][real], now[0][real])
    for h in handles:
        assert h.device_status() == 0
        h.close()


def test_cache_calls_in_a_graph_and_on_a_stream():
    """Commit, accumulation and eviction captured together and replayed on a side stream give what eager calls give."""
    import speculative_decoding_token_gb300 as sv
    rng = np.random.default_rng(31)
    lens, nodes, budget = [200, 90, 64], [12, 9, 1], 60
    base = tu.Batch(lens, nodes, 4, 2, 64, 16, BF16, seed=31, poison=False)
    n, path = make_paths(rng, nodes, base.T)
    shape = base.k.shape[:-1]
    mass0 = torch.rand(shape, generator=base.gen)
    pos0, seen0 = make_positions(rng, base, shape)
    lse = torch.rand(base.rows, 4, generator=base.gen) + 4

    def state():
        bt = tu.Batch(lens, nodes, 4, 2, 64, 16, BF16, seed=31, poison=False).upload(mass=mass0, pos=pos0)
        bufs = [torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(3)]
        moves = 3 * 2 * budget
        return bt, sv.SpecTree(3, max_moves=moves), bufs, [x.cuda() for x in (
            torch.tensor(n, dtype=torch.int32), torch.tensor(path, dtype=torch.int32), torch.tensor(seen0, dtype=torch.int32),
            lse)]

    def step(bt, h, bufs, args):
        dn, dpath, dseen, dlse = args
        h.commit(bt.cache, bt.dlens, dn, dpath, seen=dseen, new_lens=bufs[0], new_seen=bufs[1])
        h.accumulate(bt.dq, dlse, bt.cache, bt.tree, bt.dlens, dn, dpath)
        h.evict(bt.cache, bufs[0], bufs[1], budget, sink=2, recent=10, new_lens=bufs[2])

    eager, graphed = state(), state()
    step(*eager)
    keep = [t.clone() for t in (graphed[0].dk, graphed[0].dv, graphed[0].dmass, graphed[0].dpos)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*graphed)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            for t, k in zip((graphed[0].dk, graphed[0].dv, graphed[0].dmass, graphed[0].dpos), keep):
                t.copy_(k)
            g.replay()
    side.synchronize()
    torch.cuda.synchronize()
    a, b = eager[0], graphed[0]
    for x, y in ((a.dk, b.dk), (a.dv, b.dv), (a.dmass, b.dmass), (a.dpos, b.dpos), *zip(eager[2], graphed[2])):
        assert torch.equal(x, y)
    assert eager[2][2].tolist() == [min(x + y + 1, budget) for x, y in zip(lens, n)]
    for x in (eager, graphed):
        assert x[1].device_status() == 0
        x[1].close()


def test_steps_of_a_bounded_cache(st):
    """A dialogue of tree steps over one layer, every call in its place, against a cache kept in Python."""
    import speculative_decoding_token_gb300 as sv
    rng, gen = np.random.default_rng(9), torch.Generator().manual_seed(9)
    B, T, heads, kv, d, page, V, budget, sink, recent = 3, 12, 6, 2, 64, 8, 40, 20, 2, 6
    mp = -(-(budget + 2 * T) // page)
    pages = B * mp
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32)).view(B, mp)
    k = torch.randn(pages, kv, page, d, generator=gen).to(BF16).cuda()
    v = torch.randn(pages, kv, page, d, generator=gen).to(BF16).cuda()
    mass = torch.zeros(pages, kv, page, device="cuda")
    pos = torch.zeros(pages, kv, page, dtype=torch.int32, device="cuda")
    cache = sv.KVCache(k, v, table.cuda(), mass=mass, pos=pos)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    seen = torch.zeros(B, dtype=torch.int32, device="cuda")
    scale = d ** -0.5
    # the model: per (sequence, head) a list of [key, value, mass, position]
    held = [[[] for _ in range(kv)] for _ in range(B)]
    evictions = 0
    for step in range(14):
        nodes = rng.integers(1, T + 1, B)
        row_off = np.concatenate([[0], np.cumsum(nodes)[:-1]])
        rows = int(nodes.sum())
        parent, tokens = np.full((B, T), -1, np.int32), rng.integers(0, V, (B, T)).astype(np.int32)
        logits = torch.randn(rows, V, generator=gen)
        q = torch.randn(rows, heads, d, generator=gen).to(BF16)
        nk, nv = torch.randn(rows, kv, d, generator=gen).to(BF16), torch.randn(rows, kv, d, generator=gen).to(BF16)
        for b in range(B):
            parent[b, : nodes[b]] = tu.random_tree(rng, nodes[b])
            for j in range(1, nodes[b]):
                if rng.random() < 0.8:
                    tokens[b, j] = int(torch.argmax(logits[row_off[b] + parent[b, j]]))
        # the program stores the nodes' keys and values behind the committed tokens
        for b in range(B):
            L = len(held[b][0])
            assert L == int(lens[b])
            for j in range(nodes[b]):
                pg, at = int(table[b, (L + j) // page]), (L + j) % page
                k[pg, :, at], v[pg, :, at] = nk[row_off[b] + j].cuda(), nv[row_off[b] + j].cuda()
        dev = lambda x, t: torch.as_tensor(x).to("cuda", t)  # noqa: E731
        tree = sv.TokenTree(dev(row_off, torch.int64), dev(nodes, torch.int32), dev(parent, torch.int32),
                            dev(tokens, torch.int32))
        dq = q.cuda()
        out, lse = st.attention(dq, cache, tree, lens)
        n, emitted, path = st.verify(tree, logits.cuda())
        new_lens, new_seen = st.commit(cache, lens, n, path, seen=seen)
        st.accumulate(dq, lse, cache, tree, lens, n, path)
        _, _, kept = st.evict(cache, new_lens, new_seen, budget, sink=sink, recent=recent)
        assert st.device_status() == 0
        out, lse = out.double().cpu(), lse.double().cpu()
        want_n, want_tok, want_path = tu.verify(parent, nodes, tokens, row_off, logits)
        assert n.tolist() == want_n.tolist() and emitted.tolist() == want_tok.tolist() and path.tolist() == want_path.tolist()
        for b in range(B):
            at0 = int(seen[b])
            for g in range(kv):
                old = held[b][g]
                ks = torch.stack([e[0] for e in old] + [nk[row_off[b] + j, g] for j in range(nodes[b])]).double()
                vs = torch.stack([e[1] for e in old] + [nv[row_off[b] + j, g] for j in range(nodes[b])]).double()
                L = len(old)
                hs = slice(g * heads // kv, (g + 1) * heads // kv)
                for j in range(nodes[b]):
                    see = torch.as_tensor(list(range(L)) + sorted(L + i for i in tu.chain(parent[b], j)))
                    x, size = tu.scores(q[row_off[b] + j, hs], ks[see], scale)
                    p = torch.softmax(x, 1)
                    e = tu.weight_error(d, size.max(), x.abs().max())
                    tol = (2 * e + 2.0 ** -8 + 4e-5) * (p @ vs[see].abs()) * 1.01 + 2.0 ** -8 * (p @ vs[see]).abs()
                    assert bool(((out[row_off[b] + j, hs] - p @ vs[see]).abs() <= tol).all())
                    assert torch.allclose(lse[row_off[b] + j, hs], torch.logsumexp(x, 1), rtol=1e-6, atol=float(e) + 1e-5)
                walk = [int(j) for j in want_path[b] if j >= 0]
                now = [list(e) for e in old] + [[nk[row_off[b] + j, g], nv[row_off[b] + j, g], 0.0, at0 + i]
                                                for i, j in enumerate(walk)]
                kk = torch.stack([e[0] for e in now]).double()
                for i, j in enumerate(walk):
                    w = torch.exp(q[row_off[b] + j, hs].double() @ kk[: L + i + 1].T * scale
                                  - lse[row_off[b] + j, hs][:, None]).sum(0)
                    for s in range(L + i + 1):
                        now[s][2] += float(w[s])
                # the cache decides by its own masses: equal within 1e-4 here, and taken over from it
                sl = np.arange(len(now))
                size = int(kept[b])
                pg, at = table[b, sl // page].long(), torch.as_tensor(sl % page)
                got_pos = pos[pg.cuda(), g, at.cuda()].tolist()[:size]
                got_mass = mass[pg.cuda(), g, at.cuda()].tolist()[:size]
                by_pos = {e[3]: e for e in now}
                assert len(set(got_pos)) == size == min(len(now), budget)
                total = at0 + len(walk)
                for p_, m_ in zip(got_pos, got_mass):
                    assert abs(by_pos[p_][2] - m_) <= 1e-4 * (1 + abs(m_))
                gone = [e for e in now if e[3] not in set(got_pos)]
                if gone:
                    evictions += 1
                    least = min(by_pos[p_][2] for p_ in got_pos if sink <= p_ < total - recent)
                    assert all(sink <= e[3] < total - recent and e[2] <= least + 1e-4 * (1 + least) for e in gone)
                held[b][g] = [[k[int(table[b, s // page]), g, s % page].cpu(), v[int(table[b, s // page]), g, s % page].cpu(),
                               got_mass[s], got_pos[s]] for s in range(size)]
                for e in held[b][g]:
                    assert torch.equal(e[0], by_pos[e[3]][0]) and torch.equal(e[1], by_pos[e[3]][1])
        lens, seen = kept, new_seen
    assert evictions > 10


def long_paths(bt, nodes):
    """Every node of every tree accepted."""
    n = [t - 1 for t in nodes]
    path = np.full((bt.B, bt.T), -1)
    for b, t in enumerate(nodes):
        path[b, :t] = np.arange(t)
    return bt.dev(n, torch.int32), bt.dev(path, torch.int32)


def test_accumulate_adds_the_chunks_of_a_slot_in_order(st):
    """Three and four chunks of 128 rows over one to three tiles. Every score is 0, so a row weighs exactly 1 (logsumexp 0)
    or nothing (200, under fp32's least number), and sums next to 2^24 show the order in which the chunks were added."""
    B, G = 48, 8
    lens, nodes = [(60, 200, 300, 0)[b % 4] for b in range(B)], [40 + 3 * (b % 5) for b in range(B)]
    bt = tu.Batch(lens, nodes, 8 * G, 8, 64, 16, BF16, seed=51, kind="chain", poison=False)
    bt.q.zero_()
    start = 2.0 ** 24 - 2
    bt.upload(mass=torch.full(bt.k.shape[:-1], start))
    weigh = torch.zeros(bt.rows, bt.heads)
    want = torch.full(bt.k.shape[1:-1], start)
    for b in range(B):
        own = torch.zeros(nodes[b], bt.kv_heads, G)  # a node's rows of a key head
        for i, count in ((0, 3), (17, 1), (34, 1)):  # in chunks 0, 1 and 2
            own[i, :, :count] = 1
        weigh[bt.row_off[b]: bt.row_off[b] + nodes[b]] = own.view(nodes[b], -1)
        pg, at = bt.slots(b, lens[b] + nodes[b])
        for s in range(lens[b] + nodes[b]):
            rows = own[max(0, s - lens[b]):, 0].reshape(-1)  # of the nodes that see the slot
            first = max(0, s - lens[b]) * G
            total = np.float32(start)
            for c in range(0, nodes[b] * G, 128):
                total = np.float32(total + np.float32(float(rows[max(0, c - first): max(0, c + 128 - first)].sum())))
            want[pg[s], :, at[s]] = float(total)
    lse = torch.where(weigh > 0, 0.0, 200.0).cuda()
    n, path = long_paths(bt, nodes)
    for _ in range(10):
        bt.dmass.fill_(start)
        st.accumulate(bt.dq, lse, bt.cache, bt.tree, bt.dlens, n, path)
        assert torch.equal(bt.dmass.cpu(), want)


@pytest.mark.parametrize("lens,nodes,G,d", [([60, 20], [40, 64], 8, 64), ([300, 310, 5], [48, 70, 50], 8, 128),
                                            ([1000, 333, 90], [128, 100, 33], 4, 64)])
def test_accumulate_of_many_rows_repeats_bit_for_bit(st, lens, nodes, G, d):
    bt = tu.Batch(lens, nodes, 4 * G, 4, d, 16, BF16, seed=G + d)
    mass = torch.rand(bt.k.shape[:-1], generator=bt.gen)
    bt.upload(mass=mass)
    lse = (torch.rand(bt.rows, bt.heads, generator=bt.gen) * 3 + 4).cuda()
    n, path = long_paths(bt, nodes)
    first = None
    for _ in range(20):
        bt.dmass.copy_(mass[0])
        st.accumulate(bt.dq, lse, bt.cache, bt.tree, bt.dlens, n, path)
        first = bt.dmass.clone() if first is None else first
        assert torch.equal(bt.dmass, first)
    want, tol = tu.accumulate(bt, mass[0], lse.cpu(), n.tolist(), path.cpu().numpy(), d ** -0.5)
    near(first, want, tol)


# ---------------------------------------------------------------------------
# waits that run out

def with_short_waits(h, call, check):
    """Calls whose every wait gives up after a microsecond, until one has timed out: each returns and says so, and the next
    call with the default limit is right. Whether one timed out."""
    import speculative_decoding_token_gb300 as sv
    cold = torch.zeros(1 << 26, device="cuda")  # more than L2 holds
    for i in range(100):
        cold.add_(1)
        h.set_wait_limit(1)
        call()
        status = h.device_status()
        assert status in (0, sv.STATUS_BITS["timeout"])
        h.set_wait_limit(0)
        if status or i % 20 == 0:
            check()
            assert h.device_status() == 0
        if status:
            return True
    return False


def test_attention_whose_waits_run_out():
    import speculative_decoding_token_gb300 as sv
    h, late = sv.SpecTree(4), 0
    for lens, nodes, heads, d in (([20000, 700, 90], [3, 30, 1], 4, 128), ([4000, 9000], [64, 40], 16, 64)):
        bt = tu.Batch(lens, nodes, heads, 2, d, 16, BF16, seed=d, poison=False)
        late += with_short_waits(h, lambda: run_attention(h, bt), lambda: check_attention(h, bt))
    assert late
    h.close()


def test_accumulate_whose_waits_run_out():
    import speculative_decoding_token_gb300 as sv
    h, late = sv.SpecTree(4), 0
    for lens, nodes, G, d in (([9000, 700, 90], [30, 3, 1], 4, 128), ([400, 3000], [64, 40], 8, 64)):
        bt = tu.Batch(lens, nodes, 2 * G, 2, d, 16, BF16, seed=d, poison=False)
        n, path = long_paths(bt, nodes)
        mass = torch.rand(bt.k.shape[:-1], generator=bt.gen)
        bt.upload(mass=mass)
        lse = torch.rand(bt.rows, bt.heads, generator=bt.gen) * 3 + 4
        want, tol = tu.accumulate(bt, mass[0], lse, n.tolist(), path.cpu().numpy(), d ** -0.5)
        dlse = lse.cuda()

        def call():
            h.accumulate(bt.dq, dlse, bt.cache, bt.tree, bt.dlens, n, path)

        def check():
            bt.dmass.copy_(mass[0])
            call()
            near(bt.dmass, want, tol)

        late += with_short_waits(h, call, check)
    assert late
    h.close()


def test_verify_whose_waits_run_out():
    """A sequence whose waits ran out has no answer; one that was done in time has the right one."""
    import speculative_decoding_token_gb300 as sv
    case = make_verify(np.random.default_rng(8), 40, 48, 50257, BF16)
    want = tu.verify(case[2], case[0], case[3], case[1], case[4])
    h, late = sv.SpecTree(40), 0

    def call():
        n, tokens, path = run_verify(h, *case)
        gone = n == -1
        assert (tokens[gone] == -1).all() and (path[gone] == -1).all()
        for g, w in zip((n, tokens, path), want):
            assert np.array_equal(g[~gone], w[~gone])

    def check():
        for g, w in zip(run_verify(h, *case), want):
            assert np.array_equal(g, w)

    for _ in range(5):
        late += with_short_waits(h, call, check)
    assert late
    h.close()


def test_evict_into_buffers_whose_strides_differ_where_nothing_lies(st):
    """The stride of a cache's only key head says nothing."""
    rng = np.random.default_rng(6)
    bt = tu.Batch([90, 40], [0, 0], 1, 1, 64, 16, BF16, seed=6, poison=False)
    shape = bt.k.shape[:-1]
    mass = torch.rand(shape, generator=bt.gen)
    pos, seen = make_positions(rng, bt, shape)
    bt.upload(mass=mass, pos=pos)
    wide = torch.zeros(shape[1], 3, shape[3], device="cuda")  # pages of three heads
    out = torch.zeros(shape[1], 1, shape[3], device="cuda").as_strided(bt.dmass.shape, (shape[3], 7, 1))
    assert out.stride() != bt.dmass.stride()
    _, p, new_lens = st.evict(bt.cache, bt.dlens, bt.dev(seen, torch.int32), 32, sink=1, recent=4, mass_out=out)
    want = expected_evict(bt, mass, pos, seen, 32, 1, 4, torch.zeros(shape), pos)
    assert new_lens.tolist() == [32, 32]
    for got, w in ((bt.dk, want[0]), (bt.dv, want[1]), (out, want[2]), (p, want[3])):
        assert torch.equal(got.cpu(), w[0])
    with pytest.raises(ValueError):  # a stride that is used
        st.evict(bt.cache, bt.dlens, bt.dev(seen, torch.int32), 32, mass_out=wide[:, 1:2])


@pytest.mark.parametrize("B,high", [(1, 260), (150, 260), (1, 250), (150, 250)])
def test_attention_of_large_values_whose_weight_vanishes(B, high):
    """Values of 1e36 with scores 300 under the others': pieces and groups of tiles that hold nothing else count for nothing
    (one sequence: joined across CTAs; many: within them)."""
    import speculative_decoding_token_gb300 as sv
    bt = tu.Batch([400 + b % 3 for b in range(B)], [2] * B, 2, 1, 64, 16, BF16, seed=B)
    for b in range(B):
        pg, at = bt.slots(b, 402)
        bt.k[0, pg, 0, at] = 0.0
        bt.k[0, pg[130:high], 0, at[130:high], 0] = 150.0
        bt.v[0, pg[:130], 0, at[:130]] = 1e36
        bt.v[0, pg[high:400], 0, at[high:400]] = -1e36
    bt.q.zero_()
    bt.q[:, :, 0] = 16.0
    h = sv.SpecTree(B)
    check_attention(h, bt)
    assert h.device_status() == 0
    h.close()


def test_benchmark_step_does_the_same_work_every_time():
    """The benchmark's step accepts drafts, moves tokens, and commits and evicts the same slots however often it has run."""
    import os
    import sys
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    import bench
    from speculative_decoding_token_gb300 import workload
    batch = workload.make_batch(1, device="cuda", B=24)
    step = bench.tree_step({**workload.CONFIGS[1], "B": 24}, batch)
    first = None
    for _ in range(4):
        for call in step.calls:
            call()
        now = [t.clone() for t in (step.n, step.path, step.emitted, step.new_lens, step.kept, step.mass_out, step.pos_out)]
        first = now if first is None else first
        for a, b in zip(now, first):
            assert torch.equal(a, b)
    assert int((step.n > 0).sum()) > 4 and int((step.kept < step.new_lens).sum()) > 0
    assert float(step.mass.max()) > 0 and step.handle.device_status() == 0
    step.handle.close()


def test_numbers_that_do_not_fit_are_refused(st):
    """Not cut to their lowest bits: a budget of 2^32 + 4 is not one of 4."""
    import speculative_decoding_token_gb300 as sv
    bt = tu.Batch([20], [0], 2, 2, 64, 8, BF16, poison=False)
    shape = bt.k.shape[:-1]
    pos = torch.arange(bt.k.shape[1] * 8, dtype=torch.int32).view(1, -1, 1, 8).expand(shape).contiguous()
    bt.upload(mass=torch.rand(shape, generator=bt.gen), pos=pos)
    big = 1 << 32
    k, m = bt.dk.clone(), bt.dmass.clone()
    for bad in (lambda: st.evict(bt.cache, bt.dlens, bt.dlens, big + 4), lambda: st.evict(bt.cache, bt.dlens, bt.dlens, 4, sink=big),
                lambda: st.evict(bt.cache, bt.dlens, bt.dlens, 4, recent=big + 1), lambda: st.evict(bt.cache, bt.dlens, bt.dlens, -big),
                lambda: sv.SpecTree(big + 1), lambda: sv.SpecTree(1, max_moves=1 << 64), lambda: sv.SpecTree(1, device=big),
                lambda: st.set_wait_limit(-1), lambda: st.set_wait_limit(1 << 64)):
        with pytest.raises(ValueError):
            bad()
    assert torch.equal(bt.dk, k) and torch.equal(bt.dmass, m)
    assert st.device_status() == 0
