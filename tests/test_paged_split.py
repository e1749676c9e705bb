"""The splits of queries into e4m3 terms, on the host: their stated bounds over every bf16 value."""
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
