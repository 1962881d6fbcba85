"""Token log-probabilities and distillation on rows that leave little to choose from, or nothing between their logits, and
the kernel's promises about time."""
import math

import pytest
import torch

import token_exact as te
import token_util as tu

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


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
    h = svm.SpecVerify(1, 1, 1000)
    yield h
    h.close()


def clean(h):
    torch.cuda.synchronize()
    assert h.device_status() == 0


# ---------------------------------------------------------------------------
# the choice of top tokens

# tokens that a grammar, a choice of answers or a codebook leaves; logits with nothing or next to nothing between them
LEFT = ["few3", "few16", "few40", "side513", "side700", "side1024", "side1800", "side5000", "sides900", "equal", "ties", "zeros",
        "band_up", "band_down", "band", "sunk", "spike"]


def few_left(kind, rows, V, dtype, seed=0):
    """[rows, V] logits in rows of whole 16-byte pieces, of that kind."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(rows, V, device="cuda", generator=g) * 2
    left = None
    if kind.startswith("few"):  # this many tokens anywhere
        left = torch.zeros(rows, V, dtype=torch.bool, device="cuda")
        left.scatter_(1, torch.rand(rows, V, device="cuda", generator=g).topk(int(kind[3:]), 1)[1], True)
    elif kind.startswith("sides"):  # two runs of neighbours, the second at the row's end
        n = int(kind[5:])
        left = torch.zeros(rows, V, dtype=torch.bool, device="cuda")
        left[:, 3:3 + n] = left[:, V - n:] = True
    elif kind.startswith("side"):  # this many neighbours
        n = min(int(kind[4:]), V)
        at = (V - n) * torch.arange(1, rows + 1, device="cuda")[:, None] // (rows + 1)
        column = torch.arange(V, device="cuda")
        left = (column >= at) & (column < at + n)
    elif kind == "equal":
        z = torch.full_like(z, -2.5)
    elif kind == "ties":
        z = torch.randint(-3, 3, (rows, V), device="cuda", generator=g).float()
    elif kind == "zeros":  # of both signs, with denormals between
        z = torch.randint(-2, 3, (rows, V), device="cuda", generator=g).float() * (2.0 ** -133 if dtype is BF else 2.0 ** -149)
        z = torch.where(torch.rand(rows, V, device="cuda", generator=g) < 0.3, -0.0, z)
        z[:, ::3] = z[:, ::3].clamp(max=0.0)
    elif kind.startswith("band"):  # thousands of fp32 logits within one value of bf16, below and above zero
        z = 1 + torch.rand(rows, V, device="cuda", generator=g) * 2.0 ** -7
        z[::2].neg_()
        if kind != "band":
            z = torch.sort(z, 1, descending=kind == "band_down")[0]
    elif kind == "sunk":  # the same under a few better ones
        z = 1 + torch.rand(rows, V, device="cuda", generator=g) * 2.0 ** -8
        z[:, 5::V // 7] = 3.0
    elif kind == "spike":  # all of one chunk's better than the rest
        z[:, V // 2: V // 2 + 3000] += 40.0
    if left is not None:
        z = z.masked_fill(~left, -math.inf)
    return torch.nn.functional.pad(z.to(dtype), (0, -V % 8))[:, :V]


def check_top(z, T, y, r, at, k):
    s = tu.Soft(z, T)
    assert tu.close(r.logprob[at], s.lp[y], s.lp_err(s.lp[y])) and int(r.rank[at]) == s.rank(y)
    n = min(k, len(z))
    i = s.top(n)
    assert torch.equal(r.topk_idx[at][:n].long(), i), (at, r.topk_idx[at][:n].tolist(), i.tolist())
    assert (r.topk_idx[at][n:] == -1).all()
    assert tu.close(r.topk_logprob[at][:n], s.lp[i], s.lp_err(s.lp[i]))


@pytest.mark.parametrize("kind", LEFT)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,rows,ks", [(152064, 5, (1, 5, 20, 128)), (33001, 700, (3, 64)), (262147, 310, (20, 100)), (6001, 4, (128,))])
def test_top_tokens_of_what_is_left(h, kind, dtype, V, rows, ks):
    z = few_left(kind, rows, V, dtype, V)
    y = z.float().argmax(1).to(torch.int32)
    for k in ks:
        r = h.token_logprobs(z, y, 0.75, k=k, rank=True)
        clean(h)
        for i in sorted({0, 1, rows // 2, rows - 2, rows - 1}):
            check_top(z[i], 0.75, int(y[i]), r, i, k)


@pytest.mark.parametrize("kind", ["few16", "side700", "side1024", "side1800", "equal", "ties", "sunk", "band_up", "band"])
@pytest.mark.parametrize("dtype,k", [(BF, 5), (BF, 64), (FP, 20), (FP, 64)])
@pytest.mark.parametrize("rows", [5, 1000])
def test_rows_with_little_left_keep_to_a_wait_limit(h, kind, dtype, k, rows):
    """A limit of 8 ms is for what hangs: no row of a vocabulary takes that long, whatever is left of it, and rows that wait for
    one another (three and more a CTA) do not run into it."""
    z = few_left(kind, rows, 152064, dtype, 3)
    y = z.float().argmax(1).to(torch.int32)
    h.set_wait_limit(8_000_000)
    try:
        r = h.token_logprobs(z, y, k=k, rank=True)
        clean(h)
    finally:
        h.set_wait_limit(0)
    for i in (0, rows - 1):
        check_top(z[i], 1.0, int(y[i]), r, i, k)


# ---------------------------------------------------------------------------
# handles

RESET = r"""
import ctypes, sys
import speculative_decoding_token_gb300 as sv
lib, cuda = sv.load(), ctypes.CDLL(%r)
def bytes_of(n):
    p = ctypes.c_void_p()
    assert cuda.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(n)) == 0
    return p
def ask(k):
    h = sv.specverify_create(0, 1, 1, 100)
    z, y, lp, H, lse, top, idx = (bytes_of(1 << 20) for _ in range(7))
    for p in (z, y):
        assert cuda.cudaMemset(p, 0, ctypes.c_size_t(1 << 20)) == 0
    assert lib.specverify_token_logprobs(h, z, 0, 4, 1000, 1000, 1.0, 4, 1, y, None, None, k, lp, H, lse, None, top, idx, None) == 0
    assert sv.specverify_device_status(h) == 0
    out = (ctypes.c_float * 4)()
    assert cuda.cudaMemcpy(out, lp, ctypes.c_size_t(16), 2) == 0
    sv.specverify_destroy(h)
    return list(out)
first = [ask(0), ask(3)]
assert cuda.cudaDeviceReset() == 0
assert [ask(0), ask(3)] == first, first
assert abs(first[0][0] + 6.907755) < 1e-6, first
"""


def test_handles_after_a_device_reset(svm):
    """A reset ends a program's own context; a new handle works as the first did."""
    import os
    import subprocess
    import sys
    lib = next(l.split()[-1] for l in open("/proc/self/maps") if "libcudart.so" in l)
    r = subprocess.run([sys.executable, "-c", RESET % lib], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


CAPTURED = r"""
import torch
import speculative_decoding_token_gb300 as sv
h = sv.SpecVerify(1, 1, 1000)
z = torch.zeros(3, 1000, device="cuda")
y, g = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(3, device="cuda")
ids, t = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.full((3, 1), -1.0, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = [h.token_logprobs(z, y, k=2, rank=True).logprob, h.token_logprobs(z, y).logprob, *h.token_logprobs_grad(z, y, g),
           h.distill_loss(z, ids, t), *h.distill_grad(z, ids, t)]
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
assert h.device_status() == 0
want = [h.token_logprobs(z, y, k=2, rank=True).logprob, h.token_logprobs(z, y).logprob, *h.token_logprobs_grad(z, y, g),
        h.distill_loss(z, ids, t), *h.distill_grad(z, ids, t)]
assert all(torch.equal(a, b) for a, b in zip(out, want))
assert h.device_status() == 0
"""


def test_a_first_call_may_be_captured(svm):
    """A handle's first calls, in a program's first graph."""
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", CAPTURED], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_make_a_handles_first_calls(svm):
    import threading
    z = torch.zeros(40, 5000, device="cuda")
    y = torch.zeros(40, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(10):
        h, got = svm.SpecVerify(1, 1, 1000), []
        go = threading.Barrier(2)

        def first(h=h, got=got, go=go):
            s = torch.cuda.Stream()
            go.wait()
            got.append(h.token_logprobs(z, y, k=3, stream=s).logprob)
            s.synchronize()

        threads = [threading.Thread(target=first) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        clean(h)
        assert len(got) == 2 and torch.equal(got[0], got[1])
        assert (got[0] + math.log(5000)).abs().max() < 1e-5
        h.close()


# ---------------------------------------------------------------------------
# a given token that has nearly all of the mass

@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,many,T", [(40000, 1, 1.0), (40000, 40, 1.5), (152061, 1, 1.0), (1003, 30, 0.5), (13, 1, 1.0)])
@pytest.mark.parametrize("ent", [False, True], ids=["", "ent"])
def test_gradients_of_sure_tokens(h, dtype, V, many, T, ent):
    """The given token's gradient is w (g - h p (ln p - m)) / T with w = 1 - p what the others have and m the mean of their
    logarithms: as good as w, also where w is 2^-18 or 2^-40 and no fp32 p shows it.

    w is a sum of the others' weights, of one sign: exponents to D binades (the scale and the product rounded, each D and the 8 by
    which references lag times half a step), exponentials to 2^-22, chains of V / 1024 additions (256 threads with four sums each)
    and a tree of 32, and eight roundings on the way. ln p is good to w's error, m to its own (terms of one sign, and the sum's
    logarithm)."""
    gaps = [0.0, 4.0, 9.0, 12.5, 12.5, 12.5, 16.0, 28.0, 60.0, 120.0]
    rows = len(gaps)
    z = tu.logits(rows, V, FP, V, device="cuda")
    y = torch.tensor([0, V - 1, V // 2, 0, V - 1, min(V - 1, 8191), V // 3, 1, V - 2, 5], dtype=torch.int32, device="cuda")
    for r, gap in enumerate(gaps):
        v = int(y[r])
        z[r, v] = -math.inf
        z[r, v] = float(T * (torch.logsumexp(z[r].double() / T, 0) + gap))
    z = torch.nn.functional.pad(z.to(dtype), (0, -V % 8)).repeat(many, 1)[:, :V]
    g = torch.linspace(-2.0, 1.5, rows, device="cuda")
    e = torch.linspace(0.25, -1.0, rows, device="cuda") if ent else None
    grad, lp, H = h.token_logprobs_grad(z, y.repeat(many), g.repeat(many), None if e is None else e.repeat(many), T)
    clean(h)
    for i in [*range(rows), rows * many - 4]:
        r = i % rows
        s, at = tu.Soft(z[i], T), int(y[r])
        want, err = s.grad(at, float(g[r]), float(e[r]) if ent else 0.0)
        assert tu.close(grad[i], want, err, dtype), i
        others = torch.ones(V, dtype=torch.bool, device="cuda")
        others[at] = False
        x = s.z[others] / s.T
        lse = torch.logsumexp(x, 0)
        w = float(torch.exp(lse - s.lse))
        m = float((torch.exp(x - lse) * (x - s.lse)).sum())
        own = float(g[r]) * w - (float(e[r]) * float(s.p[at]) * w * (math.log1p(-w) - m) if ent else 0.0)
        D = float(s.z[at] - s.z[others].min()) / s.T * math.log2(math.e)
        rel = math.log(2) * (2 * D + 16) * 2.0 ** -24 + 2.0 ** -22 + (V / 1024 + 32) * 2.0 ** -24 + 2.0 ** -21
        lim = w * rel * (abs(float(g[r])) + (abs(float(e[r])) * (4 * abs(m) + 4) if ent else 0.0))
        assert tu.close(grad[i, at], own / s.T, lim / s.T, dtype), (i, float(grad[i, at]), own / s.T, lim / s.T)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,V", [(6, 152061), (600, 2001)])
def test_a_given_token_of_a_bad_logit_is_a_bad_row(svm, h, dtype, rows, V):
    """The given token's own logit is NaN or infinite, or the only one that is not masked, or masked."""
    z = tu.logits(rows, V, dtype, 3, device="cuda")
    y = (torch.arange(rows, device="cuda") * 977 % V).to(torch.int32)
    bad = []
    for r in range(0, rows, 6):
        for at, x in ((0, math.nan), (1, math.inf), (2, -math.inf)):
            z[r + at, y[r + at].long()] = x
        z[r + 3] = -math.inf
        z[r + 3, y[r + 3].long()] = -7.0
        z[r + 4] = -math.inf
        bad += [r, r + 1, r + 4]
    g, e = torch.ones(rows, device="cuda"), torch.full((rows,), 0.5, device="cuda")
    for h_ in (None, e):
        grad, lp, H = h.token_logprobs_grad(z, y, g, h_)
        assert h.device_status() == svm.STATUS_BITS["bad_logit"]
        assert lp.isnan().nonzero()[:, 0].tolist() == H.isnan().nonzero()[:, 0].tolist() == bad
        assert grad[bad].isnan().all()
        for r in (2, 3, 5, rows - 4, rows - 3, rows - 1):
            s = tu.Soft(z[r], 1.0)
            want, err = s.grad(int(y[r]), 1.0, 0.0 if h_ is None else 0.5)
            assert tu.close(grad[r], want, err, dtype), r
            assert tu.close(lp[r], s.lp[y[r]], s.lp_err(s.lp[y[r]])) and tu.close(H[r], s.entropy, s.entropy_err())


# ---------------------------------------------------------------------------
# sums that are known exactly: every token counts once

EXACT = [(1, 3), (5, 9), (1003, 400), (8193, 30), (33001, 5), (128256, 3), (152064, 330), (262144, 5), (262139, 40)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,rows", EXACT)
@pytest.mark.parametrize("top", [0, 5])
def test_sums_count_every_token_once(h, dtype, V, rows, top):
    z, w = te.counted(min(rows, 6), V, dtype, V, "cuda", top)
    n = z.shape[0]
    many = torch.as_strided(z, (n, z.stride(0)), (z.stride(0), 1)).repeat(-(-rows // n), 1)[:, :V]
    rows = many.shape[0]
    y = torch.arange(n, dtype=torch.int32, device="cuda") * 31 % V
    y[-1] = V // 2
    y = y.repeat(rows // n)
    check = sorted({*range(n), rows // 2, rows - 1})
    for k, rank in ((0, False), (0, True), (20, True)):
        r = h.token_logprobs(many, y, te.T2, k=k, rank=rank)
        clean(h)
        for i in check:
            assert te.right(z[i % n], w[i % n], int(y[i]), r.lse[i], r.logprob[i], r.entropy[i]), (i, k)
    g = torch.linspace(-1.0, 0.5, rows, device="cuda")
    for e in (None, torch.zeros(rows, device="cuda")):
        grad, lp, H = h.token_logprobs_grad(many, y, g, e, te.T2)
        clean(h)
        for i in check:
            assert te.right(z[i % n], w[i % n], int(y[i]), torch.logsumexp(z[i % n].double() / te.T2, 0), lp[i], H[i]), i
            assert te.right_gradient(grad[i], w[i % n], int(y[i]), float(g[i]), te.T2, dtype), i


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V,rows", [x for x in EXACT if x[0] > 100])
def test_the_rest_of_a_list_counts_every_token_once(h, dtype, V, rows):
    """Rows of n equal tokens, one of them listed with a half: the forward divergence is ln(n / 2) / 2 + ln(n / (2 n - 2)) / 2 and
    an unlisted token's gradient (1 / 2 - 1 / n) / (n - 1) / T. Of the loss, two terms of a few roundings; a lost token is 1 / (2 n)."""
    z, w = te.counted(min(rows, 6), V, dtype, V + 1, "cuda")
    n = z.shape[0]
    many = torch.as_strided(z, (n, z.stride(0)), (z.stride(0), 1)).repeat(-(-rows // n), 1)[:, :V]
    rows = many.shape[0]
    ids = torch.full((rows, 3), -1, dtype=torch.int32, device="cuda")
    ids[:, 1] = V // 2
    t = torch.full((rows, 3), -math.log(2.0), device="cuda")
    loss = h.distill_loss(many, ids, t, te.T2)
    grad, same = h.distill_grad(many, ids, t, None, te.T2)
    clean(h)
    for i in sorted({*range(n), rows // 2, rows - 1}):
        count = float(w[i % n].sum())
        p = math.exp(float(t[i, 1].double()))
        want = p * math.log(p * count) + (1 - p) * math.log((1 - p) * count / (count - 1))
        lim = 2.0 ** -24 * (2 * want + 8)
        assert lim < 0.4 / count
        assert abs(float(loss[i]) - want) <= lim and abs(float(same[i]) - want) <= lim, (i, float(loss[i]), want)
        d = torch.where(w[i % n] > 0, (p - 1 / count) / (count - 1), 0.0)
        d[V // 2] = -(p - 1 / count)
        assert tu.close(grad[i], d / te.T2, d.abs() / te.T2 * 2.0 ** -21, dtype), i


# ---------------------------------------------------------------------------
# the reverse divergence where a side has no mass

def test_reverse_divergence_at_its_edges(h):
    """Everything listed, a draft with nothing outside its list, a target sure of one token: the target's rest has its floor of
    2^-20, and the divergence and each element of its gradient are finite and the formula's."""
    V = 24
    for dtype in (FP, BF):
        z = tu.logits(6, V, dtype, 12, device="cuda")
        lp = torch.log_softmax(z.float() + 0.3 * torch.sin(torch.arange(V, device="cuda").float()), 1)
        ids = torch.full((6, V), -1, dtype=torch.int32, device="cuda")
        t = torch.zeros(6, V, device="cuda")
        ids[0] = torch.arange(V)                        # everything is listed
        t[0] = lp[0]
        z[1, 5:] = -math.inf                            # the draft has nothing outside the list, the target has
        ids[1, :5], t[1, :5] = torch.arange(5, device="cuda", dtype=torch.int32), lp[1, :5]
        ids[2, 3] = 7                                   # the target is sure of one token
        z[3, 1:] = -math.inf                            # the draft is, of a listed one
        ids[3, :2], t[3, :2] = torch.tensor([0, 3], device="cuda", dtype=torch.int32), torch.tensor([-1.0, -1.5], device="cuda")
        z[4, 1:] = -math.inf                            # of one that is not listed
        ids[4, :2], t[4, :2] = torch.tensor([2, 3], device="cuda", dtype=torch.int32), torch.tensor([-1.0, -1.5], device="cuda")
        z[5, 5:] = -math.inf                            # neither has anything outside
        ids[5, :5], t[5, :5] = torch.arange(5, device="cuda", dtype=torch.int32), torch.log_softmax(lp[5, :5], 0)
        for T in (1.0, 0.5):
            loss = h.distill_loss(z, ids, t, T, "rkl")
            grad, same = h.distill_grad(z, ids, t, None, T, "rkl")
            clean(h)
            for i in range(6):
                d = tu.Divergence(z[i], ids[i], t[i], T, "rkl")
                assert math.isfinite(float(d.loss)) and torch.isfinite(d.grad).all()
                assert tu.close(loss[i], d.loss, d.loss_err), (i, float(loss[i]), float(d.loss))
                assert tu.close(same[i], d.loss, d.loss_err)
                assert tu.close(grad[i], d.grad, d.grad_err, dtype), (i, grad[i].tolist(), d.grad.tolist())


# ---------------------------------------------------------------------------
# waits that run out, form by form

FORMS = {"sums": lambda h, z, y, ids, t, one: h.token_logprobs(z, y, entropy=False, lse=False)[:1],
         "entropy": lambda h, z, y, ids, t, one: h.token_logprobs(z, y)[:3],
         "rank": lambda h, z, y, ids, t, one: h.token_logprobs(z, y, rank=True)[:4],
         "top": lambda h, z, y, ids, t, one: [x for x in h.token_logprobs(z, y, k=9) if x is not None],
         "both": lambda h, z, y, ids, t, one: h.token_logprobs(z, y, k=9, rank=True),
         "grad": lambda h, z, y, ids, t, one: h.token_logprobs_grad(z, y, one, one),
         "loss": lambda h, z, y, ids, t, one: [h.distill_loss(z, ids, t)],
         "loss_grad": lambda h, z, y, ids, t, one: h.distill_grad(z, ids, t, divergence="jsd")}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,V", [(3, 140001), (700, 50001)], ids=["clusters", "rows"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_each_form_gives_up_and_recovers(svm, form, rows, V, dtype):
    """With a limit of a nanosecond each form of the kernel gives up at a first wait that lasts two microseconds (its logits come
    from memory that something else keeps busy), says so, and the next call, with the default limit, is right."""
    h = svm.SpecVerify(1, 1, 1000)
    z = tu.logits(min(rows, 20), V, dtype, 31, device="cuda")
    z = torch.as_strided(z, (z.shape[0], z.stride(0)), (z.stride(0), 1)).repeat(-(-rows // 20), 1)[:rows, :V]
    ids, t = tu.lists(z[:20], 12, 31)
    ids, t = ids.repeat(-(-rows // 20), 1)[:rows].contiguous(), t.repeat(-(-rows // 20), 1)[:rows].contiguous()
    y = torch.arange(rows, dtype=torch.int32, device="cuda")
    one = torch.ones(rows, device="cuda")
    run = lambda: FORMS[form](h, z, y, ids, t, one)  # noqa: E731
    want = [x.clone() for x in run()]
    clean(h)
    cold, side = torch.zeros(1 << 27, device="cuda"), torch.cuda.Stream()  # more than L2 holds
    for _ in range(40):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                cold.add_(1)
        h.set_wait_limit(1)
        run()
        status = h.device_status()
        assert status in (0, svm.STATUS_BITS["timeout"])
        h.set_wait_limit(0)
        got = run()
        clean(h)
        assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(want, got))
        if status:
            break
    assert status, "no call gave up"
    h.close()
