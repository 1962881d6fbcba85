"""Token log-probabilities, their gradient and the distillation calls against their restatement in 64 bits."""
import math

import pytest
import torch

import token_util as tu
from speculative_decoding_token_gb300 import workload

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
KINDS = ["plain", "peaked", "ties", "equal", "rising", "falling", "masked", "wide"]


@pytest.fixture(scope="module")
def svm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_token_gb300 as sv
    sv.build()
    sv.load()
    return sv


@pytest.fixture(scope="module")
def h(svm):
    h = svm.SpecVerify(1, 1, 1000)  # the calls take any sizes, whatever the handle's workspace is for
    yield h
    h.close()


def clean(h):
    torch.cuda.synchronize()
    assert h.device_status() == 0


def check_entry(z, T, y, r, at, k):
    """One entry's outputs; z is its row."""
    s = tu.Soft(z, T)
    assert tu.close(r.logprob[at], s.lp[y], s.lp_err(s.lp[y])), (at, float(r.logprob[at]), float(s.lp[y]))
    assert tu.close(r.entropy[at], s.entropy, s.entropy_err()), (at, float(r.entropy[at]), float(s.entropy))
    assert tu.close(r.lse[at], s.lse, s.lse_err())
    if r.rank is not None:
        assert int(r.rank[at]) == s.rank(y)
    if k:
        n = min(k, len(z))
        i = s.top(n)
        assert torch.equal(r.topk_idx[at][:n].long(), i)
        assert (r.topk_idx[at][n:] == -1).all() and (r.topk_logprob[at][n:] == -math.inf).all()
        assert tu.close(r.topk_logprob[at][:n], s.lp[i], s.lp_err(s.lp[i]))


# ---------------------------------------------------------------------------
# log-probabilities

@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,rows,k,pad", [(1, 3, 0, 0), (1, 2, 3, 1), (5, 4, 7, 0), (8, 9, 8, 2), (31, 5, 1, 0),
                                          (257, 40, 128, 0), (1000, 7, 20, 1), (1001, 65, 5, 0), (8193, 33, 64, 0),
                                          (32000, 5, 5, 0), (50257, 12, 32, 0), (152064, 3, 100, 0), (128256, 700, 20, 0)])
def test_logprobs_sizes(h, dtype, V, rows, k, pad):
    z = tu.logits(min(rows, 40), V, dtype, V + rows, pad=pad, device="cuda")
    if rows > 40:  # many rows: the same ones over and over, in a larger buffer
        n = -(-rows // 40)
        z = torch.as_strided(z, (z.shape[0], z.stride(0)), (z.stride(0), 1)).repeat(n, 1)[:, :V]
        rows = z.shape[0]
    y = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
    r = h.token_logprobs(z, y, 0.75, k=k, rank=True)
    clean(h)
    for i in list(range(min(rows, 40))) + [rows - 1]:
        check_entry(z[i], 0.75, int(y[i]), r, i, k)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,k,T", [(700, 10, 1.0), (20000, 64, 0.5), (40001, 1, 2.0)])
def test_logprobs_values(h, kind, dtype, V, k, T):
    z = tu.logits(6, V, dtype, V, kind, device="cuda")
    y = torch.tensor([0, V - 1, V // 2, 1, int(z[4].float().argmax()), 5], device="cuda", dtype=torch.int32)
    r = h.token_logprobs(z, y, T, k=k, rank=True)
    clean(h)
    for i in range(6):
        check_entry(z[i], T, int(y[i]), r, i, k)


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "rising", "masked"])
@pytest.mark.parametrize("dtype,V,k", [(BF, 152064, 5), (BF, 150001, 16), (FP, 256000, 8), (FP, 131077, 3), (BF, 131072, 32)])
def test_alternatives_of_few_long_rows(svm, h, kind, dtype, V, k):
    """Rows that clusters share, each CTA's own top tokens put in order once more; one that asks for nothing, one that is bad."""
    z = tu.logits(5, V, dtype, V + k, kind, device="cuda")
    y = torch.tensor([0, V - 1, -1, V // 2, 1], device="cuda", dtype=torch.int32)
    z[3, V - 2] = math.nan
    r = h.token_logprobs(z, y, 0.5, k=k, rank=True)
    assert h.device_status() == svm.STATUS_BITS["bad_logit"]
    for i in (0, 1, 4):
        check_entry(z[i], 0.5, int(y[i]), r, i, k)
    assert (r.topk_idx[2:4] == -1).all() and (r.topk_logprob[2] == -math.inf).all() and r.topk_logprob[3].isnan().all()
    assert float(r.logprob[2]) == 0 and r.logprob[3].isnan() and r.rank.tolist()[2:4] == [0, -1]
    one = h.token_logprobs(z[4:], y[4:], 0.5, k=k, rank=True)
    clean(h)
    check_entry(z[4], 0.5, 1, one, 0, k)


@pytest.mark.parametrize("k,entropy,lse,rank", [(0, True, True, False), (0, False, False, False), (0, False, False, True),
                                                (5, False, True, False), (5, True, False, True)])
def test_logprobs_outputs_not_asked_for(h, k, entropy, lse, rank):
    z = tu.logits(9, 5003, BF, 4, "masked", device="cuda")
    y = torch.arange(9, device="cuda", dtype=torch.int32)
    full = h.token_logprobs(z, y, k=5, rank=True)
    r = h.token_logprobs(z, y, k=k, entropy=entropy, lse=lse, rank=rank)
    clean(h)
    assert (r.entropy is None, r.lse is None, r.rank is None, r.topk_idx is None) == (not entropy, not lse, not rank, k == 0)
    # a call that computes less may sum in another order
    for i in range(9):
        s = tu.Soft(z[i], 1.0)
        assert tu.close(r.logprob[i], s.lp[i], s.lp_err(s.lp[i]))
    for a, b in ((r.rank, full.rank), (r.topk_idx, full.topk_idx)):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,M,V", [(1, 5, 32000), (7, 4, 999), (40, 11, 2000)])
def test_logprobs_of_sequences(h, dtype, B, M, V):
    """Ragged sequences in an order of their own, a gap between them, -1 past each, a path through a tree."""
    g = torch.Generator().manual_seed(B)
    n = torch.randint(0, M + 1, (B,), generator=g)
    off = torch.empty(B, dtype=torch.int64)
    row = 2
    for b in torch.randperm(B, generator=g).tolist():
        off[b], row = row, row + M
    z = tu.logits(row, V, dtype, B, device="cuda")
    y = torch.randint(0, V, (B, M), generator=g).to(torch.int32)
    y[torch.arange(M) >= n[:, None]] = -1
    path = torch.stack([torch.randperm(M, generator=g) for _ in range(B)]).to(torch.int32)
    path[y < 0] = -1
    for p in (None, path):
        r = h.token_logprobs(z, y.cuda(), 1.5, k=3, row_off=off.cuda(), rank=True, path=None if p is None else p.cuda())
        clean(h)
        for b in range(B):
            for m in range(M):
                if y[b, m] < 0:
                    assert float(r.logprob[b, m]) == float(r.entropy[b, m]) == float(r.lse[b, m]) == int(r.rank[b, m]) == 0
                    assert (r.topk_idx[b, m] == -1).all() and (r.topk_logprob[b, m] == -math.inf).all()
                elif (b + m) % 3 == 0 or B < 10:
                    check_entry(z[int(off[b]) + (m if p is None else int(p[b, m]))], 1.5, int(y[b, m]), r, (b, m), 3)


def test_logprobs_bad_entries_fail_alone(svm, h):
    V = 3001
    z = tu.logits(12, V, FP, 1, device="cuda")
    z[1, 7] = math.nan
    z[2, V - 1] = math.inf
    z[3] = -math.inf
    y = torch.tensor([0, 1, 2, 3, V, -2, 6, -1, 8, 9, 10, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    r = h.token_logprobs(z, y, k=2, rank=True)
    bits = h.device_status()
    assert bits == svm.STATUS_BITS["bad_logit"] | svm.STATUS_BITS["bad_token"]
    for i in (1, 2, 3, 4, 5, 11):
        assert all(x[i].isnan().all() for x in (r.logprob, r.entropy, r.lse, r.topk_logprob))
        assert int(r.rank[i]) == -1 and (r.topk_idx[i] == -1).all()
    for i in (0, 6, 8, 9, 10):
        check_entry(z[i], 1.0, int(y[i]), r, i, 2)
    # rows outside the buffer, of an entry with a token and of one without
    y = torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    y[3, 1] = -1
    off = torch.tensor([-1, 4, 11, 11], device="cuda")
    r = h.token_logprobs(z, y, k=2, row_off=off)
    assert h.device_status() == svm.STATUS_BITS["bad_row"]
    assert r.logprob.isnan().tolist() == [[True, False], [False, False], [False, True], [False, False]]
    check_entry(z[0], 1.0, 0, r, (0, 1), 2)
    check_entry(z[11], 1.0, 0, r, (3, 0), 2)
    # no row is before a sequence's first
    path = torch.tensor([[0, -1], [-1, 3]], device="cuda", dtype=torch.int32)
    r = h.token_logprobs(z, torch.zeros(2, 2, device="cuda", dtype=torch.int32), row_off=off[1:3], path=path)
    assert h.device_status() == svm.STATUS_BITS["bad_row"]
    assert r.logprob.isnan().tolist() == [[False, True], [True, True]]  # (row 14 of 12)


def test_logprobs_past_two_to_the_31(h):
    V, rows = 152064, 14200  # 2.16e9 logits
    z = torch.zeros(rows, V, dtype=BF, device="cuda")
    last = tu.logits(3, V, BF, 5, device="cuda")
    z[-3:] = last
    y = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    y[-3:] = torch.tensor([3, 77, V - 1])
    r = h.token_logprobs(z, y, k=4, rank=True)
    clean(h)
    for i in range(3):
        check_entry(last[i], 1.0, int(y[rows - 3 + i]), r, rows - 3 + i, 4)
    grad, lp, _ = h.token_logprobs_grad(z, y, torch.ones(rows, device="cuda"), grad=z)
    clean(h)
    for i in range(3):
        want, err = tu.Soft(last[i], 1.0).grad(int(y[rows - 3 + i]), 1.0, 0.0)
        assert tu.close(grad[rows - 3 + i], want, err, BF)
    assert not grad[:-3].any()


# ---------------------------------------------------------------------------
# their gradient

SIZES = [(1, 3, 0), (7, 4, 1), (1001, 70, 0), (5003, 9, 2), (50257, 37, 0), (152064, 5, 0), (256000, 2, 0)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,rows,pad", SIZES)
@pytest.mark.parametrize("ent", [False, True], ids=["", "ent"])
@pytest.mark.parametrize("in_place", [False, True], ids=["", "in_place"])
def test_logprobs_grad_sizes(h, dtype, V, rows, pad, ent, in_place):
    z = tu.logits(rows, V, dtype, V, pad=pad, device="cuda")
    y = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
    if rows > 2:
        y[1] = -1
    g, e = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda") if ent else None
    grad = z.clone(memory_format=torch.preserve_format) if not in_place else None
    keep = z.clone()
    if in_place:
        wide = torch.as_strided(z, (rows, z.stride(0)), (z.stride(0), 1))
        grad, lp, H = h.token_logprobs_grad(z, y, g, e, 0.75, grad=z)
        assert wide[:, V:].isnan().all()  # what lies between rows
    else:
        grad, lp, H = h.token_logprobs_grad(z, y, g, e, 0.75)
        assert torch.equal(z, keep)
    clean(h)
    for i in range(rows):
        s = tu.Soft(keep[i], 0.75)
        if y[i] < 0:
            assert not grad[i].any() and float(lp[i]) == float(H[i]) == 0
            continue
        want, err = s.grad(int(y[i]), float(g[i]), float(e[i]) if ent else 0.0)
        assert tu.close(grad[i], want, err, dtype), i
        assert tu.close(lp[i], s.lp[y[i]], s.lp_err(s.lp[y[i]])) and tu.close(H[i], s.entropy, s.entropy_err())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_logprobs_grad_values(h, kind, dtype):
    V = 9001
    z = tu.logits(6, V, dtype, 2, kind, device="cuda")
    y = torch.tensor([0, V - 1, 4, 1, int(z[4].float().argmax()), 5], device="cuda", dtype=torch.int32)
    g, e = torch.randn(6, device="cuda"), torch.randn(6, device="cuda")
    grad, _, _ = h.token_logprobs_grad(z, y, g, e, 1.25)
    clean(h)
    for i in range(6):
        want, err = tu.Soft(z[i], 1.25).grad(int(y[i]), float(g[i]), float(e[i]))
        assert tu.close(grad[i], want, err, dtype), i


def test_logprobs_grad_many_rows(h):
    """More rows than the GPU has room for at once, every fourth skipped."""
    V, rows = 32000, 1500
    z = tu.logits(30, V, BF, 6, device="cuda").repeat(50, 1)
    y = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
    y[::4] = -1
    g = torch.randn(rows, device="cuda")
    grad, lp, _ = h.token_logprobs_grad(z, y, g)
    clean(h)
    assert not grad[::4].any() and not lp[::4].any()
    for i in (1, 2, 303, 742, 1497, 1499):
        want, err = tu.Soft(z[i], 1.0).grad(int(y[i]), float(g[i]), 0.0)
        assert tu.close(grad[i], want, err, BF)
    # a gradient's row sums to 0: to its elements' roundings, half a step each
    ok = y >= 0
    assert (grad.float().sum(1).abs()[ok] <= 2.0 ** -8 * grad.float().abs().sum(1)[ok] + 1e-5).all()


def test_logprobs_grad_bad_rows(svm, h):
    z = tu.logits(5, 2000, BF, 1, device="cuda")
    z[1, 3], z[2], z[3, 1999] = math.nan, -math.inf, math.inf
    y = torch.tensor([0, 0, 0, 0, 2000], device="cuda", dtype=torch.int32)
    grad, lp, H = h.token_logprobs_grad(z, y, torch.ones(5, device="cuda"))
    assert h.device_status() == svm.STATUS_BITS["bad_logit"] | svm.STATUS_BITS["bad_token"]
    assert grad[1:].isnan().all() and lp[1:].isnan().all() and H[1:].isnan().all()
    want, err = tu.Soft(z[0], 1.0).grad(0, 1.0, 0.0)
    assert tu.close(grad[0], want, err, BF)


# ---------------------------------------------------------------------------
# distillation

def check_distill(h, z, ids, t, T, kind, form, beta=0.5, weight=None, in_place=False):
    rows = z.shape[0]
    loss = h.distill_loss(z, ids, t, T, kind, form=form, beta=beta)
    keep = z.clone()
    grad, same = h.distill_grad(z, ids, t, weight, T, kind, form=form, beta=beta, grad=z if in_place else None)
    clean(h)
    for i in range(rows):
        if not (ids[i] >= 0).any():
            assert float(loss[i]) == float(same[i]) == 0 and not grad[i].any()
            continue
        d = tu.Divergence(keep[i], ids[i], t[i], T, kind, form, float(torch.tensor(beta).float()))
        assert tu.close(loss[i], d.loss, d.loss_err), (i, float(loss[i]), float(d.loss), d.loss_err)
        assert tu.close(same[i], d.loss, d.loss_err), (i, float(same[i]), float(d.loss), d.loss_err)
        w = 1.0 if weight is None else float(weight[i])
        assert tu.close(grad[i], d.grad * w, d.grad_err * abs(w), z.dtype), i
    return keep


FORMS = [(d, f) for d in ("fkl", "rkl", "jsd", "tvd") for f in ("logprobs", "logits") if (d, f) != ("rkl", "logits")]


@pytest.mark.parametrize("kind,form", FORMS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,rows,K,pad", [(2, 3, 1, 0), (9, 4, 5, 1), (300, 10, 256, 0), (1001, 48, 3, 0),
                                          (5003, 7, 64, 2), (50257, 6, 33, 0)])
def test_distill_sizes(h, kind, form, dtype, V, rows, K, pad):
    z = tu.logits(rows, V, dtype, V + K, pad=pad, device="cuda")
    ids, t = tu.lists(z, K, V, form, 1.25)
    weight = torch.rand(rows, device="cuda") + 0.5
    if rows > 3:
        ids[3] = -1
        weight[2] = -0.5
    check_distill(h, z, ids, t, 1.25, kind, form, 0.3, weight)


@pytest.mark.parametrize("kind", ["fkl", "rkl", "jsd", "tvd"])
@pytest.mark.parametrize("values", KINDS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_distill_values(h, kind, values, dtype):
    z = tu.logits(6, 12345, dtype, 9, values, device="cuda")
    ids, t = tu.lists(z, 40, 9)
    check_distill(h, z, ids, t, 1.0, kind, "logprobs")


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,rows", [(152064, 6), (256000, 4), (32000, 400)])
def test_distill_large_and_in_place(h, dtype, V, rows):
    z = tu.logits(min(rows, 20), V, dtype, 3, device="cuda")
    z = z.repeat(-(-rows // 20), 1) if rows > 20 else z
    ids, t = tu.lists(z[:20], 64, 3)
    n = z.shape[0] // ids.shape[0]
    ids, t = ids.repeat(n, 1), t.repeat(n, 1)
    if rows <= 20:
        check_distill(h, z, ids, t, 1.0, "jsd", "logprobs", in_place=True)
        return
    loss, keep = h.distill_loss(z, ids, t), z.clone()
    grad, same = h.distill_grad(z, ids, t, grad=z)
    clean(h)
    for i in (0, 1, 19, 20, 205, rows - 1):
        d = tu.Divergence(keep[i], ids[i], t[i], 1.0, "fkl")
        assert tu.close(loss[i], d.loss, d.loss_err) and tu.close(same[i], d.loss, d.loss_err)
        assert tu.close(grad[i], d.grad, d.grad_err, dtype)


@pytest.mark.parametrize("kind", ["fkl", "rkl", "jsd", "tvd"])
def test_distill_edges(h, kind):
    """Whole vocabularies, lists of nothing but what the draft masks, a draft with no mass outside the list, values of -inf,
    a target sure of one token, bf16 values."""
    V = 24
    z = tu.logits(7, V, FP, 12, device="cuda")
    ids = torch.full((7, V), -1, dtype=torch.int32, device="cuda")
    t = torch.zeros(7, V, device="cuda")
    lp = torch.log_softmax(z + 0.3 * torch.sin(torch.arange(V, device="cuda").float()), 1)
    ids[0] = torch.arange(V)                         # everything is listed
    t[0] = lp[0]
    z[1, 5:] = -math.inf                             # the draft has nothing outside the list
    ids[1, :5], t[1, :5] = torch.arange(5, device="cuda", dtype=torch.int32), lp[1, :5]
    ids[2, 3] = 7                                    # sure of one token
    ids[3, 0], ids[3, 1], t[3, 1] = 2, 9, -math.inf  # a listed token that the target rules out
    ids[4, 20], t[4, 20] = 11, -0.25
    z[4, 11] = -30.0                                 # all but ruled out by the draft
    ids[5, 0], t[5, 0] = 1, -20.0                    # next to nothing listed
    ids[6, :3], t[6, :3] = torch.tensor([4, 1, 9], device="cuda", dtype=torch.int32), torch.tensor([-1.0, -2.0, -3.0]).cuda()
    if kind in ("fkl", "jsd", "tvd"):
        check_distill(h, z, ids, t, 1.0, kind, "logprobs")
    else:  # rows 0 to 3 have outcomes of (nearly) no mass on the target's side: their own test
        check_distill(h, z[4:], ids[4:].contiguous(), t[4:].contiguous(), 1.0, kind, "logprobs")
    check_distill(h, z[4:], ids[4:].contiguous(), t[4:].to(BF).contiguous(), 2.0, kind, "logprobs")


def test_distill_infinite_divergences(h):
    """A listed token that one side rules out: infinite where the formula is, finite gradients where it has them."""
    z = tu.logits(2, 50, FP, 4, device="cuda")
    z[0, 3] = -math.inf
    ids = torch.tensor([[3, 5], [3, 5]], dtype=torch.int32, device="cuda")
    t = torch.tensor([[-0.5, -1.5], [-math.inf, -1.5]], device="cuda")
    assert h.distill_loss(z, ids, t, divergence="fkl").tolist()[0] == math.inf
    assert h.distill_loss(z, ids, t, divergence="rkl").tolist()[1] == math.inf
    grad, _ = h.distill_grad(z, ids, t, divergence="fkl")
    d = tu.Divergence(z[0], ids[0], t[0], 1.0, "fkl")
    assert torch.isfinite(grad[0]).all() and tu.close(grad[0], d.grad, d.grad_err)
    for kind in ("jsd", "tvd"):
        loss, _ = h.distill_loss(z, ids, t, divergence=kind), h.device_status()
        assert torch.isfinite(loss).all()
    assert h.device_status() == 0


def test_distill_bad_rows_fail_alone(svm, h):
    V = 4001
    z = tu.logits(10, V, BF, 3, device="cuda")
    ids, t = tu.lists(z, 8, 3, short=False)
    keep = z.clone()
    z[1, int(ids[1, 2])] = math.nan          # among the listed
    z[2, 4000 if 4000 not in ids[2] else 3999] = math.nan
    z[3] = -math.inf
    ids[4, 0] = V
    ids[5, 7] = -2
    ids[6, 5] = ids[6, 1]                    # the same index twice
    t[7, 3] = math.nan
    t[8, 1] = math.inf
    loss = h.distill_loss(z, ids, t)
    bits = svm.STATUS_BITS["bad_logit"] | svm.STATUS_BITS["bad_token"]
    assert h.device_status() == bits
    grad, same = h.distill_grad(z, ids, t)
    assert h.device_status() == bits
    assert loss.isnan().tolist() == same.isnan().tolist() == [False] + [True] * 8 + [False]
    assert grad[1:9].isnan().all()
    for i in (0, 9):
        d = tu.Divergence(keep[i], ids[i], t[i], 1.0, "fkl")
        assert tu.close(grad[i], d.grad, d.grad_err, BF) and tu.close(loss[i], d.loss, d.loss_err)


@pytest.mark.parametrize("kind", ["fkl", "rkl", "jsd", "tvd"])
def test_distill_lists_of_more_than_one(svm, h, kind):
    """Log-probabilities that leave less than nothing of one: the rest has none, and the formulas hold for what is there."""
    z = tu.logits(4, 3001, FP, 5, device="cuda")
    ids, t = tu.lists(z, 6, 5, short=False)
    t[0] += 0.3 - t[0].logsumexp(0)   # 1.35 in all
    t[1, 2] = 3.0
    t[2] -= t[2].logsumexp(0)         # one, to a rounding
    t[3, 0] = 81.0
    keep = [3]
    loss = h.distill_loss(z, ids, t, 1.0, kind)
    grad, same = h.distill_grad(z, ids, t, None, 1.0, kind)
    assert h.device_status() == svm.STATUS_BITS["bad_logit"]
    assert loss.isnan().tolist() == same.isnan().tolist() == [False, False, False, True]
    for i in range(3):
        d = tu.Divergence(z[i], ids[i], t[i], 1.0, kind)
        assert tu.close(loss[i], d.loss, d.loss_err), (i, float(loss[i]), float(d.loss))
        assert tu.close(same[i], d.loss, d.loss_err)
        assert tu.close(grad[i], d.grad, d.grad_err, FP), i
    assert grad[keep].isnan().all()


# ---------------------------------------------------------------------------
# as a program runs them

def test_refusals(svm, h):
    z = tu.logits(4, 40, FP, device="cuda")
    y, g = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
    ids, t = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    odd = torch.zeros(4, 41, device="cuda")
    for call in (lambda: h.token_logprobs(z, y, 0.0), lambda: h.token_logprobs(z, y, -1.0),
                 lambda: h.token_logprobs(z, y, math.nan), lambda: h.token_logprobs(z, y, math.inf),
                 lambda: h.token_logprobs(z, y, 1e-39), lambda: h.token_logprobs(odd, y),
                 lambda: h.token_logprobs(odd[:, 1:41], y),
                 lambda: h.distill_loss(z, ids, t, divergence="rkl", form="logits"),
                 lambda: h.distill_loss(z, ids, t, divergence="jsd", beta=0.0),
                 lambda: h.distill_loss(z, ids, t, divergence="jsd", beta=math.nan),
                 lambda: h.distill_grad(z, ids, t, divergence="jsd", beta=1.0),
                 # a gradient over half of the logits, over the weights, over the list
                 lambda: h.token_logprobs_grad(z[:3], y[:3], g[:3], grad=z[1:]),
                 lambda: h.token_logprobs_grad(z, y, z.view(-1)[:4], grad=z),
                 lambda: h.distill_grad(z, ids, t, z.view(-1)[:4], grad=z)):
        with pytest.raises(svm.SpecVerifyError) as e:
            call()
        assert e.value.rc == svm.ERR_INVALID_ARG
    for call in (lambda: h.token_logprobs(z, y.long()), lambda: h.token_logprobs(z, y[:3]), lambda: h.token_logprobs(z.half(), y),
                 lambda: h.token_logprobs(z.t(), y), lambda: h.token_logprobs(z, y, k=129), lambda: h.token_logprobs(z, y, k=-1),
                 lambda: h.token_logprobs(z, y, path=y), lambda: h.token_logprobs(z, y.cpu()),
                 lambda: h.token_logprobs(z, y, k=2, out=h.token_logprobs_buffers(4, k=3)),
                 lambda: h.token_logprobs(z, y, k=0, out=h.token_logprobs_buffers(4, k=3)),
                 lambda: h.token_logprobs_grad(z, y, g, grad=odd), lambda: h.token_logprobs_grad(z, y, g.double()),
                 lambda: h.distill_loss(z, ids, t.half()), lambda: h.distill_loss(z, ids[:, :0], t[:, :0]),
                 lambda: h.distill_loss(z, ids, t, divergence="kl"), lambda: h.distill_loss(z, ids, t, form="probs"),
                 lambda: h.distill_loss(z, ids.t().contiguous().t(), t)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert h.device_status() == 0


def test_nothing_to_do(h):
    z = torch.empty(0, 100, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert h.token_logprobs(z, none, k=3).topk_idx.shape == (0, 3)
    assert h.token_logprobs_grad(z, none, torch.empty(0, device="cuda"))[0].shape == (0, 100)
    assert h.distill_loss(z, none.view(0, 1), torch.empty(0, 1, device="cuda")).shape == (0,)
    assert h.distill_grad(z, none.view(0, 1), torch.empty(0, 1, device="cuda"))[0].shape == (0, 100)
    z = tu.logits(2, 100, FP, device="cuda")  # no sequences, sequences of no entries
    off = torch.empty(0, dtype=torch.int64, device="cuda")
    assert h.token_logprobs(z, none.view(0, 4), row_off=off).logprob.shape == (0, 4)
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    assert h.token_logprobs(z, none.view(3, 0), row_off=off).logprob.shape == (3, 0)
    clean(h)


def everything(h, z, y, ids, t, stream=None):
    r = h.token_logprobs(z, y, k=7, rank=True, stream=stream)
    g, _, _ = h.token_logprobs_grad(z, y, r.logprob, r.entropy, stream=stream)
    loss = h.distill_loss(z, ids, t, divergence="jsd", stream=stream)
    d, same = h.distill_grad(z, ids, t, loss, divergence="jsd", stream=stream)
    return [*r, g, loss, d, same]


def inputs(seed, rows=21, V=20001, dtype=BF):
    z = tu.logits(rows, V, dtype, seed, device="cuda")
    ids, t = tu.lists(z, 12, seed)
    y = torch.randint(-1, V, (rows,), device="cuda", dtype=torch.int32)
    return z, y, ids, t


def test_results_repeat_on_any_stream(h):
    """The same bits from run to run, and with two streams at once on one handle."""
    a, b = inputs(1), inputs(2, rows=300, V=9999, dtype=FP)
    want = [everything(h, *a), everything(h, *b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        got.append([everything(h, *a, stream=s[0]), everything(h, *b, stream=s[1])])
    torch.cuda.synchronize()
    for x in got:
        for p, q in zip(want, x):
            assert all(torch.equal(m.nan_to_num(), n.nan_to_num()) for m, n in zip(p, q))
    clean(h)


def test_graphs_replay_beside_one_another(h):
    a, b = inputs(3), inputs(4, rows=150, V=5000, dtype=FP)
    want = [everything(h, *a), everything(h, *b)]
    s, graphs, out = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.append(everything(h, *x))
        graphs.append(g)
    for o in out:
        for x in o:
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for p, q in zip(want, out):
        assert all(torch.equal(m.nan_to_num(), n.nan_to_num()) for m, n in zip(p, q))
    clean(h)


def test_rows_past_the_last_and_between_stay(h):
    """Outputs of a call on part of a buffer touch nothing else."""
    V, rows = 1003, 6
    z = tu.logits(rows, V, FP, 1, device="cuda")
    ids, t = tu.lists(z, 5, 1)
    wide = torch.full((rows + 2, 1024), 7.0, device="cuda")
    grad = wide[1:-1, :V]
    h.distill_grad(z, ids, t, grad=grad)
    h.token_logprobs_grad(z, torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.ones(rows, device="cuda"), grad=grad)
    clean(h)
    assert (wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, V:] == 7).all()
    assert (wide[1:-1, :V] != 7).all()


def test_logprobs_of_what_a_verify_emits(svm):
    batch = workload.make_batch(1, device="cuda", seed=11)
    h = svm.SpecVerify(batch.B, batch.gamma_max, batch.V)
    n, tokens = h.verify_batch(batch, seed=3)
    r = h.token_logprobs(batch.target, tokens, batch.T, k=5, rank=True, row_off=batch.p_row_off)
    assert h.device_status() == 0
    for b in range(batch.B):
        for m in range(batch.gamma_max + 1):
            if m <= int(n[b]):
                check_entry(batch.target[int(batch.p_row_off[b]) + m], batch.T, int(tokens[b, m]), r, (b, m), 5)
            else:
                assert int(tokens[b, m]) == -1 and float(r.logprob[b, m]) == 0
    # a greedy step emits the argmax: rank 0, and the first alternative
    n, tokens = h.verify_batch(batch, greedy=True)
    r = h.token_logprobs(batch.target, tokens, k=1, rank=True, row_off=batch.p_row_off)
    live = tokens >= 0
    assert not r.rank[live].any() and torch.equal(r.topk_idx[live][:, 0], tokens[live])
    # the same drafts as trees that are chains, through the accepted path
    parent, toks = workload.draft_tree(batch, chain=True)
    tree = svm.TokenTree(batch.p_row_off, batch.gamma + 1, parent, toks)
    st = svm.SpecTree(batch.B)
    _, emitted, path = st.verify(tree, batch.target)
    r = h.token_logprobs(batch.target, emitted, k=1, rank=True, row_off=batch.p_row_off, path=path)
    live = emitted >= 0
    assert not r.rank[live].any() and torch.equal(r.topk_idx[live][:, 0], emitted[live])
    assert h.device_status() == 0 and st.device_status() == 0
    st.close()
    h.close()


def test_distillation_from_a_targets_pass(h):
    """The target's rows give the lists, the draft's rows its loss and gradient; the gradient goes on through a linear
    draft head as autograd's would, and its reverse divergence agrees with the acceptance the framework measures."""
    g = torch.Generator(device="cuda").manual_seed(5)
    V, d, rows, T = 5000, 64, 24, 1.25
    x = torch.randn(rows, d, generator=g, device="cuda")
    W = (0.3 * torch.randn(V, d, generator=g, device="cuda")).requires_grad_()
    target = (x @ W.detach().t() + torch.randn(rows, V, generator=g, device="cuda"))
    top = h.token_logprobs(target, torch.zeros(rows, dtype=torch.int32, device="cuda"), T, k=64)
    draft = x @ W.t()
    weight = torch.full((rows,), 1.0 / rows, device="cuda")
    grad, loss = h.distill_grad(draft.detach(), top.topk_idx, top.topk_logprob, weight, T, "tvd")
    draft.backward(grad)
    clean(h)
    want = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(want)
    for i in range(rows):
        D = tu.Divergence(draft[i].detach(), top.topk_idx[i], top.topk_logprob[i], T, "tvd")
        assert tu.close(loss[i], D.loss, D.loss_err)
        assert tu.close(grad[i], D.grad / rows, D.grad_err / rows)
        want += torch.outer(D.grad / rows, x[i].double())
        # the product of fp32 gradients: their error and a rounding a term
        err += torch.outer(D.grad_err / rows + 2.0 ** -20 * D.grad.abs() / rows, x[i].double().abs())
    assert ((W.grad.double() - want).abs() <= err + 1e-12).all()
    # TVD over all tokens is at least that over outcomes that put the rest together
    p, q = torch.softmax(target.double() / T, 1), torch.softmax(draft.detach().double() / T, 1)
    assert (loss.double() <= 0.5 * (p - q).abs().sum(1) + 1e-5).all()


def test_exploring_gradients_by_differences(h):
    """The calls' own values, moved by a step of the logits, give the gradients that the calls return."""
    z = tu.logits(3, 500, FP, 21, device="cuda")
    ids, t = tu.lists(z, 9, 21)
    y = torch.tensor([4, 77, 499], dtype=torch.int32, device="cuda")
    one, step = torch.ones(3, device="cuda"), 2.0 ** -6
    grad, _, _ = h.token_logprobs_grad(z, y, one, one)
    dgrad, _ = h.distill_grad(z, ids, t, divergence="rkl")
    for v in (4, 77, int(ids[0, 0]), int(ids[1, 0])):
        moved = []
        for s in (step, -step):
            x = z.clone()
            x[:, v] += s
            r = h.token_logprobs(x, y)
            moved.append((r.logprob + r.entropy, h.distill_loss(x, ids, t, divergence="rkl")))
        # a difference of fp32 values (each off by 2^-20 of a few units) over 2 steps, and a third derivative of order 10
        lim = 2.0 ** -17 / step + 10 * step * step
        assert ((moved[0][0] - moved[1][0]) / (2 * step) - grad[:, v]).abs().max() <= lim
        assert ((moved[0][1] - moved[1][1]) / (2 * step) - dgrad[:, v]).abs().max() <= lim
    clean(h)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,kind", [(64000, "rkl"), (256000, "fkl"), (262144, "jsd"), (128000, "tvd")])
def test_gradients_under_load_repeat(h, dtype, V, kind):
    """Rows enough to keep the memory busy: every element is the same in every run, and right."""
    rows, K = 200, 128
    z = torch.randn(rows, V, device="cuda").mul_(2).to(dtype)
    v, i = z.float().topk(K, 1)
    ids, t = i.to(torch.int32), v - z.float().logsumexp(1, keepdim=True) - 0.01
    y, one = ids[:, 5].contiguous(), torch.ones(rows, device="cuda")
    first = None
    for _ in range(5):
        got = (*h.distill_grad(z, ids, t, divergence=kind), *h.token_logprobs_grad(z, y, one, one))
        if first is None:
            first = [x.clone() for x in got]
        for a, b in zip(first, got):
            assert torch.equal(a, b)
    clean(h)
    for r in range(0, rows, 9):
        d = tu.Divergence(z[r], ids[r], t[r], 1.0, kind)
        assert tu.close(first[0][r], d.grad, d.grad_err, dtype) and tu.close(first[1][r], d.loss, d.loss_err)
        want, err = tu.Soft(z[r], 1.0).grad(int(y[r]), 1.0, 1.0)
        assert tu.close(first[2][r], want, err, dtype)


def test_rows_under_load_repeat(h):
    rows, V = 900, 128256
    z = torch.randn(rows, V, device="cuda").mul_(2).to(BF)
    y = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
    top = h.token_logprobs(z, y, k=64)
    first = None
    for _ in range(5):
        got = [x for k in (0, 64) for x in h.token_logprobs(z, y, k=k, rank=k == 0) if x is not None]
        got.append(h.distill_loss(z, top.topk_idx, top.topk_logprob - 0.01, divergence="jsd"))
        if first is None:
            first = [x.clone() for x in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    clean(h)
    for i in range(0, rows, 90):
        check_entry(z[i], 1.0, int(y[i]), top, i, 64)


# ---------------------------------------------------------------------------
# far from zero: logits whose neighbours in the type are many binades of weight apart, and whose products with log2(e) / T
# are rounded by as much

def steps(dtype, base, step, V=20001, rising=False):
    """Rows of base + j step: j = 0 in a row's first half and 0 or 1, or 0 to 7, behind it; or rising."""
    g = torch.Generator().manual_seed(77)
    j = torch.randint(0, 8, (3, V), generator=g).double()
    j[0] = j[0].clamp(max=1)
    j[:2, : V // 2] = 0
    if rising:
        j = torch.sort(torch.randint(0, 160, (3, V), generator=g).double(), 1)[0]
    x = base + j * step
    z = x.to(dtype)
    assert torch.equal(z.double(), x)  # the type has them all
    return torch.nn.functional.pad(z, (0, -V % 8)).cuda()[:, :V]


BF16_LAG = [(-32768.0, 128.0, 1.0), (-100.0, 0.5, 2.0 ** -7), (-100.0, 0.5, 0.25), (-1.0, 2.0 ** -8, 2.0 ** -20)]


def check_far(h, z, T):
    y = torch.tensor([7, z.shape[1] - 1, z.shape[1] // 2], dtype=torch.int32, device="cuda")
    for rows in (3, 180):
        many = torch.as_strided(z, (3, z.stride(0)), (z.stride(0), 1)).repeat(rows // 3, 1)[:, : z.shape[1]]
        for k in (0, 20):
            r = h.token_logprobs(many, y.repeat(rows // 3), T, k=k, rank=True)
            clean(h)
            for i in (0, 1, 2, rows - 1):
                check_entry(z[i % 3], T, int(y[i % 3]), r, i, k)
        g, e = torch.tensor([1.0, -0.5, 2.0], device="cuda"), torch.tensor([0.5, 1.0, -1.0], device="cuda")
        grad, _, _ = h.token_logprobs_grad(many, y.repeat(rows // 3), g.repeat(rows // 3), e.repeat(rows // 3), T)
        clean(h)
        for i in (0, 1, 2, rows - 1):
            want, err = tu.Soft(z[i % 3], T).grad(int(y[i % 3]), float(g[i % 3]), float(e[i % 3]))
            assert tu.close(grad[i], want, err, z.dtype), i
    ids, t = tu.lists(z, 9, 3, T=T)
    for kind in ("fkl", "jsd", "tvd"):
        check_distill(h, z, ids, t, T, kind, "logprobs")


@pytest.mark.parametrize("base,step,T", BF16_LAG)
def test_bf16_rows_below_zero(h, base, step, T):
    """Negative logits a step of the type above what came before them."""
    check_far(h, steps(BF, base, step), T)


# T = 1: |z| log2(e) = 2^24 between 11629080 and 11629081
FAR = [(BF, 2.0 ** 100, 2.0 ** 93, 1.0), (BF, -2.0 ** 40, 2.0 ** 33, 2.0 ** 20), (BF, -2.0 ** 40, 2.0 ** 32, 1.0),
       (FP, 2.0 ** 40, 2.0 ** 17, 1.0), (FP, -2.0 ** 40, 2.0 ** 16, 2.0 ** 12), (FP, -2.0 ** 60, 2.0 ** 36, 2.0 ** 20),
       (FP, 2.0 ** 127, 2.0 ** 104, 1.0), (FP, -2.0 ** 127, 2.0 ** 103, 2.0 ** 20), (FP, -1.0, 2.0 ** -24, 2.0 ** -20),
       (FP, 0.0, 2.0 ** -149, 1.0), (BF, 0.0, 2.0 ** -133, 1.0), (FP, 0.0, 2.0 ** -149, 2.0 ** -20),
       (FP, 20000.0, 2.0 ** -9, 2.0 ** -10)]
RISING = [(11629000.0, 1.0, 1.0), (-11629160.0, 1.0, 1.0), (11629000.0, 1.0, 1.5), (-2.0 ** 24, 1.0, 1.0)]


@pytest.mark.parametrize("dtype,base,step,T", FAR)
def test_rows_far_from_zero(h, dtype, base, step, T):
    check_far(h, steps(dtype, base, step), T)


@pytest.mark.parametrize("base,step,T", RISING)
def test_rows_that_rise_far_from_zero(h, base, step, T):
    check_far(h, steps(FP, base, step, rising=True), T)


@pytest.mark.parametrize("T", [2.0 ** -20, 0.01, 1.0, 2.0 ** 20])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_exploring_gradients_of_masked_rows_at_every_temperature(h, dtype, T):
    """Large weights of the entropy, masked tokens, cold rows: nothing times nothing's logarithm stays nothing."""
    V = 9001
    z = tu.logits(3, V, dtype, 5, "plain", device="cuda")
    z *= min(T, 1.0)
    z[:, ::3], z[:, 1::3] = -math.inf, tu.LOWEST[dtype]
    y = torch.tensor([0, 2, 8], dtype=torch.int32, device="cuda")
    g, e = torch.tensor([1.0, 0.0, 2.0 ** 16], device="cuda"), torch.tensor([2.0 ** 16, -1.0, 2.0 ** 30], device="cuda")
    for rows in (3, 180):
        many = torch.as_strided(z, (3, z.stride(0)), (z.stride(0), 1)).repeat(rows // 3, 1)[:, :V]
        grad, lp, H = h.token_logprobs_grad(many, y.repeat(rows // 3), g.repeat(rows // 3), e.repeat(rows // 3), T)
        clean(h)
        for i in (0, 1, 2, rows - 1):
            s = tu.Soft(z[i % 3], T)
            at = int(y[i % 3])
            assert tu.close(lp[i], s.lp[at], s.lp_err(s.lp[at])) and tu.close(H[i], s.entropy, s.entropy_err())
            want, err = s.grad(at, float(g[i % 3]), float(e[i % 3]))
            assert tu.close(grad[i], want, err, dtype), i


# ---------------------------------------------------------------------------
# a draft that agrees with its target

@pytest.mark.parametrize("kind", ["fkl", "rkl", "jsd", "tvd"])
@pytest.mark.parametrize("K,T", [(1, 1.9), (20, 1.9), (100, 0.7)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_small_divergences(h, kind, K, T, dtype):
    """Divergences far below one are as good as larger ones. What is off is the sum over the rest, by a share e of it: q of the
    rest is e (1 - q) q more, the others less by as much in all. Of the first three the derivative is p less q (of the rest,
    times no more than 1, 2 where a logarithm's half percent is counted in); of the TVD it is that change. The terms are
    of one sign: each a few roundings off, and by what a logarithm is (2^-37) times p less q."""
    z = tu.logits(24, 30000, dtype, 8, device="cuda")
    ids, t = tu.lists(z, K, 8, T=T, noise=0.02, short=False)
    loss = h.distill_loss(z, ids, t, T, kind)
    _, same = h.distill_grad(z, ids, t, None, T, kind)
    clean(h)
    for i in range(24):
        d = tu.Divergence(z[i], ids[i], t[i], T, kind)
        p_rest = 1.0 - float(torch.exp(t[i].double()).sum())
        q_rest = 1.0 - float(d.soft.p[ids[i].long()].sum())
        off = d.soft.sum_err * (q_rest * (1 - q_rest) if kind == "tvd" else 2 * abs(q_rest - p_rest))
        lim = off + 2.0 ** -20 * float(d.loss) + 2.0 ** -37 * 2 * (2 * float(d.loss)) ** 0.5
        assert abs(float(loss[i]) - float(d.loss)) <= lim, (i, float(loss[i]), float(d.loss), lim)
        assert abs(float(same[i]) - float(d.loss)) <= lim


@pytest.mark.parametrize("kind,form", FORMS)
@pytest.mark.parametrize("on", [0, None], ids=["listed", "rest"])
def test_gradients_of_sure_drafts(h, kind, form, on):
    """A draft with all but 2^-14 of its mass on one outcome: gradients and losses are of that size, and good to a few roundings
    of it (each term's logarithms to 2^-22 of themselves and 2^-36 of one, its factors to 2^-21) and to the share that the
    rest's sum is off by, which moves that much mass times the other's."""
    V, K = 40000, 7
    z = tu.logits(6, V, FP, 14, device="cuda") * 0.25
    ids, t = tu.lists(z, K, 14, form, noise=0.3, short=False)
    for r in range(6):
        free = next(v for v in range(V) if not (ids[r] == v).any())
        v = int(ids[r, 0]) if on == 0 else free
        others = torch.logsumexp(z[r].double(), 0)
        z[r, v] = float(others) + 9.7
        if form == "logprobs":  # the target is sure of the same
            small = torch.rand(K, device="cuda").mul_(2.0 ** -16).add_(2.0 ** -18)
            t[r] = torch.log(small)
            if on == 0:
                t[r, 0] = torch.log1p(-small[1:].sum() - 2.0 ** -15)
        elif on == 0:
            t[r] = torch.tensor([12.0] + [0.5 * k for k in range(K - 1)], device="cuda")
    grad, loss = h.distill_grad(z, ids, t, None, 1.0, kind, form=form)
    clean(h)
    for r in range(6):
        d = tu.Divergence(z[r], ids[r], t[r], 1.0, kind, form)
        q_rest = 1 - float(d.soft.p[ids[r].long()].sum())
        moved = d.soft.sum_err * q_rest * (1 - q_rest) + 2.0 ** -36
        size = d.grad.abs()
        lim = 2.0 ** -19 * size + 4 * moved * d.soft.p.clamp(min=2.0 ** -40) ** 0.5 + 2.0 ** -20 * size.max() * d.soft.p ** 0.5
        assert ((grad[r].double() - d.grad).abs() <= lim).all(), (r, float(((grad[r].double() - d.grad).abs() - lim).max()))
        assert abs(float(loss[r]) - float(d.loss)) <= 2.0 ** -20 * float(d.loss) + 16 * moved


# ---------------------------------------------------------------------------
# waits that run out

@pytest.mark.parametrize("rows,V", [(3, 50001), (60, 50001), (3, 140001)], ids=["clusters", "rows", "long"])
def test_waits_that_run_out(svm, rows, V):
    """With a limit of a nanosecond a call gives up at the first wait that lasts a microsecond, and says so; the next call,
    with the default limit, is right. (Not every call has such a wait every time.)"""
    h = svm.SpecVerify(1, 1, 1000)
    z, y, ids, t = inputs(31, rows=rows, V=V)
    one = torch.ones(rows, device="cuda")
    cold, late = torch.zeros(1 << 26, device="cuda"), 0  # more than L2 holds
    for run in (lambda: [x for x in h.token_logprobs(z, y, rank=True) if x is not None],
                lambda: [x for x in h.token_logprobs(z, y, k=9) if x is not None],
                lambda: h.token_logprobs_grad(z, y, one, one), lambda: [h.distill_loss(z, ids, t)],
                lambda: h.distill_grad(z, ids, t)):
        want = [x.clone() for x in run()]
        clean(h)
        for _ in range(20):
            cold.add_(1)
            h.set_wait_limit(1)
            run()
            status = h.device_status()
            assert status in (0, svm.STATUS_BITS["timeout"])
            h.set_wait_limit(0)
            got = run()
            clean(h)
            assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(want, got))
            late += status != 0
            if status:
                break
    assert late
    h.close()
