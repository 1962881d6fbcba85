"""Rows whose sums are known exactly: logits that are whole multiples of the temperature's ln 2, few of them apart, so that every
weight is a small whole number and every sum of weights one below 2^24, which fp32 holds. What a call says of them is off by
its logarithm's last steps alone, far less than one token in a vocabulary weighs."""
import math

import numpy as np
import torch

import token_util as tu

T2 = float(np.float32(math.log2(math.e)))  # of this temperature log2(e) / T is 1 in fp32: a logit is its weight's exponent
assert np.float32(math.log2(math.e) / T2) == 1.0
CLOSE = 2.0 ** -23  # of a logarithm before its rounding: logf of 1 to 2 (a step of a number below 0.7), the rest in pairs


def counted(rows, V, dtype, seed, device="cpu", top=0):
    """[rows, V] logits 0 .. top in whole 16-byte rows, half of the tokens masked (none in the first row), and their weights."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randint(0, top + 1, (rows, V), generator=g).float()
    left = torch.rand(rows, V, generator=g) < 0.5
    left[0] = True
    left[:, V // 2] = True
    w = torch.where(left, torch.exp2(z), 0.0).double()
    z = z.masked_fill(~left, -math.inf)
    assert float(w.sum(1).max()) < 2 ** 24
    return torch.nn.functional.pad(z.to(dtype), (0, -V % 8)).to(device)[:, :V], w.to(device)


def right(z, w, y, lse, logprob, entropy):
    """Whether a row's outputs are those of its weights w; z at T2."""
    total = w.sum()
    x = torch.where(w > 0, torch.log(w.clamp(min=1.0)), 0.0)  # ln 2^z
    # 2^z to 2^-22 where z is not 0 (of 0 it is 1), and ln 2 / T2 off by 2^-26
    off = CLOSE + (2.0 ** -22 + 2.0 ** -22 if float(x.max()) > 0 else 0.0)
    want = torch.log(total)
    mean = (w * x).sum() / total
    # the mean's sums are above 2^24: six additions of parts; its division and product
    off_H = off + float(mean) * (2.0 ** -21 + 8 * 2.0 ** -24) + 2.0 ** -22
    return (tu.close(lse, want, off) and tu.close(logprob, x[y] - want if w[y] > 0 else torch.tensor(-math.inf), off)
            and tu.close(entropy, want - mean, off_H))


def right_gradient(grad, w, y, g, T, dtype):
    """Whether a row's gradient of g logprob[y] is (g / T) ([v = y] - w_v / sum w), each element to a few roundings."""
    want = -g * w / w.sum()
    want[y] = g * (w.sum() - w[y]) / w.sum()
    return tu.close(grad, want / T, want.abs() / T * (2.0 ** -22 + 8 * 2.0 ** -24 + (2.0 ** -21 if float(w.max()) > 1 else 0.0)), dtype)
