"""Host-side checks of the token log-probability and distillation calls (no GPU needed): refusals before any CUDA call,
and the restatement in 64 bits that the GPU tests compare against, pinned by worked cases and by differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

import token_util as tu


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_token_gb300 as sv
    sv.build()
    return sv.load()


def test_refusals_without_a_handle(lib):
    from speculative_decoding_token_gb300 import losses
    li = losses.SpecverifyLists(K=1)
    rows = (None, None, 0, 1, 8, 8, 1.0)
    assert lib.specverify_token_logprobs(*rows, 1, 1, None, None, None, 0, *[None] * 7) == -1
    assert lib.specverify_token_logprobs_grad(*rows, None, None, None, None, 8, None, None, None) == -1
    assert lib.specverify_distill_loss(*rows, ctypes.byref(li), None, None) == -1
    assert lib.specverify_distill_grad(*rows, ctypes.byref(li), None, None, 8, None, None) == -1


def test_struct_matches_the_header(lib):
    from speculative_decoding_token_gb300 import losses
    assert ctypes.sizeof(losses.SpecverifyLists) == 4 * 4 + 4 + 4 + 2 * 8


def test_importing_the_package_needs_no_torch():
    import subprocess
    import sys
    code = "import sys, speculative_decoding_token_gb300 as sv; assert 'torch' not in sys.modules; sv.TokenLogprobs"
    subprocess.run([sys.executable, "-c", code], check=True)


def test_binding_refuses_host_tensors_and_bad_shapes(lib):
    import speculative_decoding_token_gb300 as sv
    h = object.__new__(sv.SpecVerify)  # no CUDA here: a handle that every call refuses before using it
    h.h, h.device = None, 0
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        h.token_logprobs(z, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        h.distill_grad(z, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))


# -- the restatement

def test_log_probabilities_of_worked_rows():
    s = tu.Soft(torch.tensor([0.0, math.log(3.0)]), 1.0)
    # ln 3 in fp32 is off by up to 2^-24, a log-probability by three quarters of that
    assert abs(float(s.lp[0]) - math.log(0.25)) < 2.0 ** -24 and abs(float(s.lse) - math.log(4.0)) < 1e-7
    assert abs(float(s.entropy) - (math.log(4) - 0.75 * math.log(3))) < 1e-7
    s = tu.Soft(torch.tensor([1.0, 5.0, 5.0, -math.inf]), 2.0)
    assert [s.rank(i) for i in range(4)] == [2, 0, 1, 3] and s.top(3).tolist() == [1, 2, 0]
    u = tu.Soft(torch.full((7,), tu.LOWEST[torch.float32]), 1.0)  # masked by the lowest value, all of it: uniform
    assert abs(float(u.entropy) - math.log(7)) < 1e-12 and abs(float(u.lp[3]) + math.log(7)) < 1e-12


@pytest.mark.parametrize("T", [0.5, 1.0, 1.75])
def test_log_probability_gradient_by_differences(T):
    z = tu.logits(1, 37, torch.float32, 3)[0].double()
    for y, g, h in ((5, 1.0, 0.0), (0, -0.3, 0.7), (36, 0.0, 1.0)):
        f = lambda x: g * tu.Soft(x, T).lp[y] + h * tu.Soft(x, T).entropy  # noqa: E731, B023
        want, step = tu.Soft(z, T).grad(y, g, h)[0], 1e-5
        for v in (0, 5, 17, 36):
            e = torch.zeros_like(z)
            e[v] = step
            assert abs(float((f(z + e) - f(z - e)) / (2 * step)) - float(want[v])) < 1e-8


@pytest.mark.parametrize("kind", ["fkl", "rkl", "jsd", "tvd"])
@pytest.mark.parametrize("form", ["logprobs", "logits"])
def test_divergence_gradient_by_differences(kind, form):
    if kind == "rkl" and form == "logits":
        pytest.skip("infinite")
    z = tu.logits(2, 41, torch.float32, 5).double()
    ids, t = tu.lists(z, 6, 5, form, 1.25)
    for r in range(2):
        f = lambda x: tu.Divergence(x, ids[r], t[r], 1.25, kind, form, 0.3)  # noqa: E731, B023
        want, step = f(z[r]).grad, 1e-5
        for v in list(range(8)) + ids[r][ids[r] >= 0].tolist():
            e = torch.zeros(41, dtype=torch.float64)
            e[v] = step
            assert abs(float((f(z[r] + e).loss - f(z[r] - e).loss) / (2 * step)) - float(want[v])) < 1e-8


def test_divergences_of_worked_rows():
    # a draft of 1/2, 1/4, 1/4; the target lists the first token alone, with 3/4
    z, ids = torch.tensor([math.log(2.0), 0.0, 0.0], dtype=torch.float64), torch.tensor([0])
    t = torch.tensor([math.log(0.75)], dtype=torch.float64)
    D = lambda kind, **k: float(tu.Divergence(z, ids, t, 1.0, kind, **k).loss)  # noqa: E731
    assert abs(D("tvd") - 0.25) < 1e-9
    assert abs(D("fkl") - (0.75 * math.log(1.5) + 0.25 * math.log(0.5))) < 1e-9
    assert abs(D("rkl") - (0.5 * math.log(2 / 3) + 0.5 * math.log(2))) < 1e-9
    m = (0.625, 0.375)
    want = 0.5 * (0.75 * math.log(0.75 / m[0]) + 0.25 * math.log(0.25 / m[1])
                  + 0.5 * math.log(0.5 / m[0]) + 0.5 * math.log(0.5 / m[1]))
    assert abs(D("jsd") - want) < 1e-9
    # over the list alone the target is the first token: -ln 1/2
    assert abs(D("fkl", form="logits") - math.log(2)) < 1e-9
    # the draft's own distribution, complete or not, is at no distance
    lp = tu.Soft(z, 1.0).lp
    for kind in ("fkl", "rkl", "jsd", "tvd"):
        assert abs(float(tu.Divergence(z, torch.tensor([0, 2]), lp[[0, 2]], 1.0, kind).loss)) < 1e-9


def test_a_planted_mistake_fails_the_differences():
    """The gradient without the rest's share, or with the temperature left out, is not the difference quotient's."""
    z = tu.logits(1, 20, torch.float32, 8).double()
    ids, t = tu.lists(z, 4, 8, "logprobs", 2.0, short=False)
    d = tu.Divergence(z[0], ids[0], t[0], 2.0, "fkl")
    step, e = 1e-5, torch.zeros(20, dtype=torch.float64)
    v = next(v for v in range(20) if v not in ids[0])
    e[v] = step
    diff = float((tu.Divergence(z[0] + e, ids[0], t[0], 2.0, "fkl").loss
                  - tu.Divergence(z[0] - e, ids[0], t[0], 2.0, "fkl").loss) / (2 * step))
    q = float(d.soft.p[v])
    for wrong in (q / 2.0, float(d.grad[v]) * 2.0):
        assert abs(diff - wrong) > 1e-4 * q
    assert np.isclose(diff, float(d.grad[v]), rtol=1e-4)


# -- plans

PLANS = r"""
#include <cstdio>
#include <random>
#include "sv_token.cuh"

using namespace sv;

// What a plan has to keep to, whatever fits the device.
template <class Kd>
int check(const TokenParams &P, const int (&room)[5], Plan &p) {
    p = make_plan<Kd>(P, room);
    const int64_t vecs = ((int64_t)P.V * Kd::kSize + 15) / 16;
    const int chunks = (p.slice_vecs + Kd::kChunkVecs - 1) / Kd::kChunkVecs;
    if (p.cluster < 1 || p.cluster > kMaxCluster || p.clusters < 1 || p.slots < 2 || p.slots > kMaxSlots) return 1;
    if ((int64_t)p.slice_vecs * p.cluster < vecs || p.smem > kHalfSmem) return 2;
    if ((int64_t)p.clusters * p.cluster > INT32_MAX || (!p.dynamic && p.clusters > P.entries)) return 3;
    if (Kd::Top && (p.cluster > 1 ? P.k * p.cluster > kGathered : P.k > kMaxAlternatives)) return 4;
    if (Kd::Top && ((chunks + (1 << p.group_log) - 1) >> p.group_log) > kGroupRows) return 5;
    if (!Kd::Grad && p.cluster > 1 && p.clusters < P.entries) return 6;  // sums alone: a cluster has one row
    if (Kd::kId < 0 || Kd::kId >= 18) return 7;
    return 0;
}

int main() {
    std::mt19937_64 rng(1);
    auto spread = [&](double lo, double hi) { return (int64_t)std::exp(std::uniform_real_distribution<>(std::log(lo), std::log(hi))(rng)); };
    const int large[5] = {304, 152, 72, 36, 16}, small[5] = {60, 30, 14, 6, 2}, one[5] = {8, 4, 2, 1, 1};
    int unlike = 0;
    for (int i = 0; i < 20000; ++i) {
        TokenParams P{};
        P.V = (int32_t)(i % 50 == 0 ? INT32_MAX - i : spread(1, 400000));
        P.entries = P.rows = i % 70 == 0 ? 1ll << 34 : spread(1, 5000);
        P.k = (int32_t)spread(1, 128.9);
        P.K = (int32_t)spread(1, 256.9);
        Plan a, b;
        for (const int (*rooms)[5] : {&large, &small, &one}) {
            const int (&room)[5] = *rooms;
            const int bad[] = {check<Kind<0, false, false, false, false, false>>(P, room, a), check<Kind<1, false, false, true, false, true>>(P, room, a),
                               check<Kind<0, false, false, true, true, true>>(P, room, a), check<Kind<1, false, false, true, true, false>>(P, room, a),
                               check<Kind<0, false, true, true, false, false>>(P, room, a), check<Kind<1, false, true, false, false, false>>(P, room, a),
                               check<Kind<1, true, false, false, false, false>>(P, room, a), check<Kind<0, true, true, false, false, false>>(P, room, a)};
            for (int j = 0; j < 8; ++j)
                if (bad[j]) {
                    std::printf("kind %d: %d (V %d, entries %lld, k %d, K %d, room %d)\n", j, bad[j], P.V, (long long)P.entries, P.k, P.K, room[0]);
                    return 1;
                }
        }
        check<Kind<1, false, true, false, false, false>>(P, large, a);
        check<Kind<1, false, true, false, false, false>>(P, small, b);
        unlike += a.cluster != b.cluster;
    }
    std::printf("%d\n", unlike);
    return 0;
}
"""


def test_plans_are_a_devices_own(lib, tmp_path):
    """Every plan keeps to the kernel's limits, over the range of sizes and for large and small devices, and is made for the
    device that it is told of, not for the last that a handle was made on."""
    import subprocess

    from speculative_decoding_token_gb300 import _build
    src, exe = tmp_path / "plans.cu", tmp_path / "plans"
    src.write_text(PLANS)
    subprocess.run([_build.nvcc(), *_build.NVCC_FLAGS, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 100


def test_binding_refuses_more_rows_than_the_call_counts(lib):
    """2^32 rows of a token each would be none in 32 bits."""
    import speculative_decoding_token_gb300 as sv
    h = object.__new__(sv.SpecVerify)
    h.h, h.device = None, -1  # tensors on the host, as far as the check
    for rows in (2 ** 31, 2 ** 32, 2 ** 32 + 3):
        z = torch.zeros(8).as_strided((rows, 8), (0, 1))
        tokens = torch.zeros(1, dtype=torch.int32)
        for y, off in ((tokens.expand(rows), None), (tokens.expand(rows, 1), torch.zeros(1, dtype=torch.int64).expand(rows)),
                       (tokens.expand(1, rows), torch.zeros(1, dtype=torch.int64))):
            with pytest.raises(ValueError, match="no more than 2147483647 rows"):
                h.token_logprobs(z, y, row_off=off)


# -- rows of exact sums

@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("V", [1001, 128256, 262144])
def test_a_lost_vector_is_seen_in_exact_sums(V, top):
    """The limits of rows with exact sums let right outputs through, and no vector lost or counted twice; where all weights are one,
    no token."""
    import token_exact as te
    z, w = te.counted(2, V, torch.float32, V, top=top)
    for r in range(2):
        y = V // 2
        x = torch.where(w[r] > 0, torch.log(w[r].clamp(min=1)), 0.0)
        total, spread = w[r].sum(), (w[r] * x).sum()

        def says(sum_, t, r=r, x=x, y=y):
            lse = torch.log(sum_)
            return te.right(z[r], w[r], y, lse.float(), (x[y] - lse).float(), (lse - t / sum_).float())

        assert says(total, spread)
        at = torch.nonzero(w[r])[:, 0]
        vectors = [(int(v), int(v) // step * step, step) for v in (at[0], at[len(at) // 3], at[-1]) for step in (4, 8)]
        for v, first, step in vectors:
            lost = slice(first, min(first + step, V))
            for sign in (-1, 1):
                assert not says(total + sign * w[r][lost].sum(), spread + sign * (w[r][lost] * x[lost]).sum())
                if top == 0:
                    assert not says(total + sign * w[r][v], spread)
        g, p = -0.5, w[r] / total
        grad = -g * p
        grad[y] += g
        assert te.right_gradient((grad / te.T2).float(), w[r], y, g, te.T2, torch.float32)
        assert not te.right_gradient((grad / te.T2 * (1 + 4 / V)).float(), w[r], y, g, te.T2, torch.float32)
        wrong = grad.clone()
        wrong[at[1] if at[1] != y else at[2]] = 0
        assert not te.right_gradient((wrong / te.T2).float(), w[r], y, g, te.T2, torch.float32)
