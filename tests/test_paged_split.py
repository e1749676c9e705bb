"""The splits of queries and probabilities into terms of fewer bits, on the host: their stated bounds,
and inputs that would show a lost term of the probabilities."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")


def e4m3(x):
    """Rounded to nearest even, saturated."""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).double()


def bf16_below(limit):
    v = (torch.arange(0x7F80, dtype=torch.int32) << 16).view(torch.float32).double()
    return v[v < limit]


def fine(x):
    """The decode form's split: the second term 16 times finer, of what the first leaves."""
    t1 = e4m3(x)
    return t1 + e4m3((x - t1) * 16) / 16


def level(x):
    """The chunk form's: one scale, the leading 4 bits and the other 4."""
    cut = ((x.float().view(torch.int32) >> 16 & 0xFFF0) << 16).view(torch.float32).double()
    return e4m3(cut) + e4m3(x - cut)


@pytest.mark.parametrize("split,exact_from,bound", [(fine, 2.0 ** -13, 2.0 ** -21), (level, 2.0 ** -9, 2.0 ** -16)])
def test_two_terms_of_a_query(split, exact_from, bound):
    """The row's largest value is scaled into [128, 256): relative to it, exact from `exact_from` on,
    and `bound` holds below (and is needed: half of it would not do)."""
    x = bf16_below(256.0)
    err = (x - split(x)).abs()
    assert bound / 2 * 128 < err.max() <= bound * 128  # the smallest largest value is the worst case
    for largest in (128.0, 255.0):
        assert (err[x >= exact_from * largest] == 0).all()


# ---- probabilities. Their rounding errors average out over random weights; so every 128-key tile gets
# one key M of the largest score (value 0), 41 keys A (value +1) and 86 keys B (value -1), with scores at
# which the A and the B nearly cancel: the errors of the two weights then are the output.
HEADS, N_A, N_B = 16, 41, 86


def balanced_keys(n):
    """Kind of each position: 0 M, 1 A, 2 B."""
    at = np.arange(n) % 128
    return np.where(at == 0, 0, np.where(at <= N_A, 1, 2))


def balanced_scores():
    """[HEADS, 3] scores of M, A and B before their rounding to bf16."""
    d = np.linspace(0.31, 2.93, HEADS)
    return np.stack([0 * d, -d, -d - math.log(N_B / N_A)], 1)


def bf16_round(x):
    return torch.as_tensor(x).float().bfloat16().double()


def e4m3_terms(p, terms):
    """The running maximum lies at 2^5; each term 16 times finer than the one before."""
    rest, total = p * 32, 0
    for i in range(terms):
        t = e4m3(rest * 16 ** i) / 16 ** i
        total, rest = total + t, rest - t
    return total / 32


def cut_terms(p, terms):
    """bf16: the leading 8 bits, then the rest."""
    hi = (p.float().view(torch.int32) & -65536).view(torch.float32).double()
    return hi if terms == 1 else hi + bf16_round(p - hi)


def half_terms(p, terms):
    """fp16 at 2^7 (bf16 if one bit of detail is lost)."""
    return (p * 128).half().double() / 128 if terms == 2 else bf16_round(p)


# the probabilities of a form: how they are held, terms, stated error of a weight
HELD = {"decode e4m3": (e4m3_terms, 3, 2.0 ** -12), "decode bf16": (cut_terms, 2, 2.0 ** -15),
        "chunk e4m3": (half_terms, 2, 2.0 ** -11)}


@pytest.mark.parametrize("form", HELD)
def test_probabilities_and_what_a_lost_term_would_show(form):
    held, terms, bound = HELD[form]
    p = torch.exp(bf16_round(balanced_scores()))
    mag = N_A * p[:, 1] + N_B * p[:, 2]
    out = lambda w: N_A * w[:, 1] - N_B * w[:, 2]  # noqa: E731
    tol = bound * mag + 2.0 ** -16 * mag
    assert (out(p).abs() < 0.02 * mag).all()
    assert ((out(held(p, terms)) - out(p)).abs() <= tol).all()
    lost = (out(held(p, terms - 1)) - out(p)).abs()
    assert (lost > 1.5 * tol).sum() >= 2  # of 16 heads; one is enough to be noticed
