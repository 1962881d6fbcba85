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
