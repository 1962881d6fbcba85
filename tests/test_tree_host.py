"""Host-side checks of the token-tree calls (no GPU needed): refusals before any CUDA call, and the restatement in 64 bits
that the GPU tests compare against, pinned by cases worked by hand."""
import ctypes

import numpy as np
import pytest
import torch

import tree_util as tu


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_token_gb300 as sv
    sv.build()
    return sv.load()


def test_refusals_without_a_handle(lib):
    from speculative_decoding_token_gb300 import tree
    h, cache, t = ctypes.c_void_p(), tree.SpecverifyCache(), tree.SpecverifyTree(B=1, max_nodes=4)
    for args in ((None, 0, 1, 0), (ctypes.byref(h), 0, 0, 0), (ctypes.byref(h), 0, 70000, 0), (ctypes.byref(h), 0, 1, -1),
                 (ctypes.byref(h), -1, 1, 0), (ctypes.byref(h), 0, 1, 1 << 40)):
        assert lib.specverify_tree_create(*args) == -1
    c, tr = ctypes.byref(cache), ctypes.byref(t)
    assert lib.specverify_tree_attention(None, c, tr, None, None, 1, 1, 8, 8, 1.0, None, 8, 8, None, None) == -1
    assert lib.specverify_verify_tree(None, tr, None, 0, 8, 8, 1, None, None, None, None) == -1
    assert lib.specverify_tree_commit(None, c, 1, 4, None, None, None, None, None, None, None) == -1
    assert lib.specverify_cache_accumulate(None, c, tr, None, None, None, None, 1, 1, 8, 8, None, 1.0, None) == -1
    assert lib.specverify_cache_evict(None, c, 1, None, None, 4, 0, 0, None, None, None, None) == -1
    assert lib.specverify_tree_status(None, None, None) == -1
    assert lib.specverify_tree_workspace_bytes(None, None) == -1
    assert lib.specverify_tree_destroy(None) == 0


def test_structs_match_the_header(lib):
    from speculative_decoding_token_gb300 import tree
    # 5 ints and an int64 between them, 2 pointers, 4 strides, 2 pointers, 4 strides, pointer, int64, int
    assert ctypes.sizeof(tree.SpecverifyCache) == 8 + 8 + 16 + 2 * 8 + 4 * 8 + 2 * 8 + 4 * 8 + 8 + 8 + 8
    assert ctypes.sizeof(tree.SpecverifyTree) == 8 + 4 * 8


def test_descriptions_refuse_host_tensors_and_bad_shapes():
    import speculative_decoding_token_gb300 as sv
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    for bad in (lambda: sv.KVCache(k, k, table), lambda: sv.KVCache(k[0], k[0], table),
                lambda: sv.KVCache(k, k.half(), table), lambda: sv.KVCache(k.float(), k.float(), table),
                lambda: sv.TokenTree(None, None, torch.zeros(2, 3, dtype=torch.int32)),
                lambda: sv.TokenTree(None, None, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(AttributeError):
        sv.NoSuchName


def test_attention_restated_on_worked_cases():
    """Equal scores give the mean of the seen values; a score far above the others gives its value."""
    bt = tu.Batch([3], [3], 1, 1, 64, 8, torch.bfloat16, seed=0, poison=True, device="cpu")
    bt.parent[0, :3] = [-1, 0, 0]
    bt.q.zero_()
    out, lse, _, _ = tu.attention(bt, 1.0)
    o = bt.row_off[0]
    pg, at = bt.slots(0, 6)
    v = bt.v[0][pg, 0, at].double()
    for j, seen in ((0, [0, 1, 2, 3]), (1, [0, 1, 2, 3, 4]), (2, [0, 1, 2, 3, 5])):
        assert torch.allclose(out[o + j, 0], v[seen].mean(0), atol=1e-12)
        assert abs(float(lse[o + j, 0]) - np.log(len(seen))) < 1e-12
    assert bool(torch.isnan(out[0]).all())  # a row of no sequence
    bt.k.zero_()
    bt.k[0, pg[1], 0, at[1], 0] = 100.0
    bt.q[o, 0, 0] = 1.0
    out, lse, _, _ = tu.attention(bt, 1.0)
    assert torch.allclose(out[o, 0], v[1], atol=1e-12) and abs(float(lse[o, 0]) - 100.0) < 1e-9


def test_verify_restated_on_worked_cases():
    target = torch.zeros(4, 5)
    target[0, 3] = target[1, 1] = target[2, 4] = 1.0
    parent, tokens = [[-1, 0, 0, 2]], np.array([[0, 2, 3, 4]])
    n, out, path = tu.verify(parent, [4], tokens, [0], target)
    # row 0 says 3 (node 2), row 2 says 4 (node 3), row 3 is flat: token 0
    assert n.tolist() == [2] and out.tolist() == [[3, 4, 0, -1]] and path.tolist() == [[0, 2, 3, -1]]
    target[2, 0] = float("nan")
    assert tu.verify(parent, [4], tokens, [0], target)[0].tolist() == [-1]
    assert tu.verify(parent, [0], tokens, [0], target)[0].tolist() == [-1]


def test_kept_slots_on_worked_cases():
    mass, pos = np.array([5.0, 1.0, 4.0, 4.0, 0.0, 2.0]), np.arange(6)
    assert tu.keep_slots(mass, pos, 6, 9, 0, 0).tolist() == [0, 1, 2, 3, 4, 5]
    assert tu.keep_slots(mass, pos, 6, 3, 0, 0).tolist() == [0, 3, 2]  # 5, 4, 4: slot 3 moves to the free slot 1
    assert tu.keep_slots(mass, pos, 6, 3, 1, 1).tolist() == [0, 5, 2]  # first and last position stay, then the lower tie
    mass[0] = np.nan
    assert set(tu.keep_slots(mass, pos, 6, 2, 0, 0).tolist()) == {2, 3}


# ---------------------------------------------------------------------------
# checks ahead of the device: a handle whose device does not exist, so that a call that passes them ends there

NO_DEVICE, TOO_LARGE, INVALID = -2, -6, -1


class FakeHandle(ctypes.Structure):
    """The first members of the handle, as the library lays them out."""
    _fields_ = [("device", ctypes.c_int), ("num_sms", ctypes.c_int), ("max_batch", ctypes.c_int32),
                ("max_moves", ctypes.c_int64), ("rest", ctypes.c_char * 256)]


class HostCalls:
    """The calls with addresses that are never read: buffers far apart, of a cache of `layers` layers, B = 1."""

    def __init__(self, lib, *, layers=1, pages=4, kv_heads=2, page=16, d=64, max_pages=4, nodes=4):
        from speculative_decoding_token_gb300 import tree
        self.lib, self.handle = lib, FakeHandle(device=10 ** 6, num_sms=152, max_batch=4, max_moves=1 << 30)
        self.h = ctypes.byref(self.handle)
        token, head = d, page * d
        self.cache = tree.SpecverifyCache(
            dtype=1, layers=layers, num_pages=pages, page_size=page, kv_heads=kv_heads, head_dim=d, k=1 << 44, v=1 << 45,
            layer_stride=pages * kv_heads * head if layers > 1 else 0, page_stride=kv_heads * head, head_stride=head, token_stride=token,
            mass=1 << 42, pos=1 << 43, mass_layer_stride=pages * kv_heads * page, mass_page_stride=kv_heads * page,
            mass_head_stride=page, mass_token_stride=1, page_table=4096, table_stride=max_pages, max_pages=max_pages)
        self.tree = tree.SpecverifyTree(B=1, max_nodes=nodes, row_off=4096, nodes=4096, parent=4096, tokens=4096)

    def attention(self, heads, rows=4, q_strides=None, out_strides=None, q=1 << 40, out=1 << 41, lse=1 << 39):
        d = self.cache.head_dim
        q_strides, out_strides = q_strides or (heads * d, d), out_strides or (heads * d, d)
        return self.lib.specverify_tree_attention(self.h, ctypes.byref(self.cache), ctypes.byref(self.tree), 4096, q, rows,
                                                  heads, *q_strides, 0.125, out, *out_strides, lse, None)

    def accumulate(self, heads, rows=4):
        d = self.cache.head_dim
        return self.lib.specverify_cache_accumulate(self.h, ctypes.byref(self.cache), ctypes.byref(self.tree), 4096, 4096,
                                                    4096, 1 << 40, rows, heads, heads * d, d, 1 << 41, 0.125, None)

    def commit(self):
        return self.lib.specverify_tree_commit(self.h, ctypes.byref(self.cache), 1, 4, 4096, 8192, 12288, 16384, 20480,
                                               24576, None)

    def evict(self, mass_out=None, pos_out=None):
        return self.lib.specverify_cache_evict(self.h, ctypes.byref(self.cache), 1, 4096, 8192, 8, 0, 0,
                                               mass_out or self.cache.mass, pos_out or self.cache.pos, 12288, None)


def test_plain_calls_pass_the_host_checks(lib):
    c = HostCalls(lib, layers=1)
    assert [c.attention(4), c.accumulate(4), c.commit(), c.evict()] == [NO_DEVICE] * 4
    c = HostCalls(lib, layers=3)
    assert [c.commit(), c.evict()] == [NO_DEVICE] * 2


def test_work_that_does_not_fit_31_bits_is_refused(lib):
    """The kernels count a sequence's tiles, and what the start of each key head weighs beside them, in 31 bits: six units
    for the attention, one for the accumulation."""
    most = 2 ** 31 - 1
    for head, call in ((6, "attention"), (1, "accumulate")):
        for slots, tiles in ((128, 1), (136, 2), (8, 1), (128 * 40, 40)):
            fit = most // (tiles + head)
            if fit * 8 * 64 > 2 ** 38:  # more heads than a page stride can span
                continue
            for kv_heads, want in ((fit, NO_DEVICE), (fit + 1, TOO_LARGE)):
                c = HostCalls(lib, kv_heads=kv_heads, page=8, max_pages=slots // 8, pages=slots // 8)
                assert getattr(c, call)(kv_heads) == want, (call, slots, kv_heads)


def test_rows_of_a_key_head_that_do_not_fit_31_bits_are_refused(lib):
    for call in ("attention", "accumulate"):
        c = HostCalls(lib, kv_heads=1, nodes=128)
        most = (2 ** 31 - 1 - 256) // 128
        assert getattr(c, call)(most) == NO_DEVICE
        assert getattr(c, call)(most + 1) == TOO_LARGE


def test_attention_refuses_an_output_that_shares_memory(lib):
    c = HostCalls(lib)
    d, out = 64, 1 << 41
    for rows, heads, strides in ((4, 4, (4 * d, 8)), (4, 4, (8, 4 * d)), (4, 4, (2 * d, d)), (4, 4, (0, d)), (4, 4, (4 * d, 0)),
                                 (4, 4, (4 * d - 8, d)), (5, 4, (d, 4 * d)), (2, 4, (d - 8, 4 * d))):
        assert c.attention(heads, rows, out_strides=strides) == INVALID, (rows, heads, strides)
    for rows, heads, strides in ((4, 4, (4 * d, d)), (4, 4, (d, 4 * d)), (4, 4, (12 * d, 3 * d)), (4, 4, (2 * d, 8 * d)),
                                 (1, 4, (0, d)), (4, 2, (2 * d + 8, d + 8))):
        assert c.attention(heads, rows, out_strides=strides) == NO_DEVICE, (rows, heads, strides)
    # queries and outputs: one buffer, buffers that overlap, halves of one row
    assert c.attention(4, q=out, out=out) == INVALID
    assert c.attention(4, q=out, out=out, q_strides=(0, 0)) == INVALID
    assert c.attention(4, q=out + 2 * d, out=out) == INVALID
    assert c.attention(4, q=out + 2 * 4 * d, out=out) == INVALID
    assert c.attention(4, q=out + 2 * 16 * d, out=out) == NO_DEVICE
    wide = (8 * d, d)
    assert c.attention(4, q=out + 2 * 4 * d, out=out, q_strides=wide, out_strides=wide) == NO_DEVICE


def test_caches_that_share_memory_are_read_and_not_written(lib):
    def calls(**changes):
        c = HostCalls(lib, layers=2)
        for name, value in changes.items():
            setattr(c.cache, name, value)
        one = HostCalls(lib)
        for name, value in changes.items():
            if not name.endswith("layer_stride"):
                setattr(one.cache, name, value)
        return one.attention(4), one.accumulate(4), c.commit(), c.evict()

    ok, no = NO_DEVICE, INVALID
    assert calls() == (ok, ok, ok, ok)
    # keys and values: overlapping tokens, heads or pages, the same buffer twice, buffers that overlap
    for change in (dict(token_stride=8), dict(head_stride=8 * 64), dict(page_stride=8), dict(v=1 << 44),
                   dict(v=(1 << 44) + 64), dict(v=(1 << 44) + 2 * 64)):
        assert calls(**change) == (ok, ok, no, no), change
    assert calls(layer_stride=64) == (ok, ok, no, no)
    # token-major, and keys beside values in one pool: by page, by head, by token
    assert calls(token_stride=2 * 64, head_stride=64) == (ok, ok, ok, ok)
    assert calls(page_stride=2 * 2048, layer_stride=4 * 4096, v=(1 << 44) + 2 * 2048) == (ok, ok, ok, ok)
    assert calls(head_stride=2048, page_stride=4096, layer_stride=4 * 4096, v=(1 << 44) + 2 * 1024) == (ok, ok, ok, ok)
    assert calls(token_stride=128, head_stride=2048, page_stride=4096, layer_stride=4 * 4096,
                 v=(1 << 44) + 2 * 64) == (ok, ok, ok, ok)
    # masses and positions
    for change in (dict(mass_token_stride=0), dict(mass_token_stride=-1), dict(mass_head_stride=8), dict(mass_page_stride=16),
                   dict(mass_head_stride=-16)):
        assert calls(**change) == (ok, no, no, no), change
    for change in (dict(pos=1 << 42), dict(pos=(1 << 42) + 4), dict(mass_layer_stride=3)):
        assert calls(**change) == (ok, ok, no, no), change
    assert calls(mass_token_stride=2, mass_head_stride=2, mass_page_stride=64, mass_layer_stride=256) == (ok, no, no, no)
    assert calls(mass_token_stride=2, mass_head_stride=32, mass_page_stride=64, mass_layer_stride=256,
                 pos=(1 << 42) + 4) == (ok, ok, ok, ok)
    # what the eviction writes: the cache's own, or buffers apart from them
    c = HostCalls(lib)
    m, p, far = c.cache.mass, c.cache.pos, 1 << 38
    assert [c.evict(m, p), c.evict(far, p), c.evict(m, far), c.evict(far, far + (1 << 20))] == [ok] * 4
    for a, b in ((m + 4, p), (m, p + 4), (far, far), (far, far + 4), (p, m), (p, far), (far, m), (m + 4 * 100, p)):
        assert c.evict(a, b) == no, (a, b)
    c.cache.mass = None
    assert c.commit() == ok
    c.cache.pos = None
    assert c.commit() == ok


@pytest.mark.parametrize("config,kw", [(1, {}), (3, dict(B=24, V=1001)), (3, dict(B=30, V=5))])
def test_drafted_trees_take_steps(config, kw):
    from speculative_decoding_token_gb300 import workload
    batch = workload.make_batch(config, **kw)
    nodes, rows = (batch.gamma + 1).tolist(), batch.p_row_off.tolist()
    for chain in (False, True):
        parent, tokens = workload.draft_tree(batch, chain=chain, seed=3)
        assert parent.dtype == tokens.dtype == torch.int32 and parent.shape == tokens.shape == (batch.B, batch.gamma_max + 1)
        for b in range(batch.B):
            up = parent[b, : nodes[b]].tolist()
            assert up[0] == -1 and all(0 <= p < j for j, p in enumerate(up) if j)
            assert not chain or up == list(range(-1, nodes[b] - 1))
        assert bool(((tokens >= 0) & (tokens < batch.V)).all())
        n = tu.verify(parent.numpy(), nodes, tokens.numpy(), rows, batch.target)[0]
        assert (n > 0).sum() > batch.B // 3
        # every first child agrees: the walk ends in a leaf; no child does but by chance
        parent, tokens = workload.draft_tree(batch, agree=1.0, chain=chain, seed=4)
        n, _, path = tu.verify(parent.numpy(), nodes, tokens.numpy(), rows, batch.target)
        for b in range(batch.B):
            assert int(path[b, n[b]]) not in parent[b, : nodes[b]].tolist()
        assert not chain or n.tolist() == batch.gamma.tolist()
    assert torch.equal(workload.draft_tree(batch, agree=0.0)[1][:, 1:], batch.draft_tokens)
