"""The paged cache's operators where they can go wrong: refused calls, lists, scales, values at the
ends of the types' ranges. Tolerances: see test_gpu_paged.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from helpers import assert_device_ok, rope_gpu  # noqa: E402,F401
from test_gpu_paged import Case, f64  # noqa: E402,F401
from test_paged_split import HELD, balanced_keys, balanced_scores  # noqa: E402

D = 128


@pytest.fixture(scope="module")
def q3():
    import qwen3_decoder_block_b200 as m
    return m


def test_a_refused_attention_call_leaves_nothing_on_the_stream(q3):
    """A row stride that no tensor map can hold is refused; the call's own plan kernel, which would
    report the negative context, must not have been launched."""
    c = Case(q3, [1], [40], 16)
    c.t_ctx.fill_(-1)
    c.ldq = 1 << 39
    with pytest.raises(q3.Qwen3Error, match="ldq"):
        c.attend()
    assert q3.check_device_error() == q3.OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[1, 1], [200, 1], [1] * 17 + [40]])
def test_workspace_at_any_16_bytes(q3, qlens, fp8):
    """A workspace may begin at any multiple of 16 bytes."""
    c = Case(q3, qlens, [700 + 13 * b for b in range(len(qlens))], 32, fp8=fp8, seed=3)
    c.darken()
    n = q3.workspace_size(c.cfg, q3.OP_ATTENTION_PAGED, len(qlens), max(qlens), 1)
    whole = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0
    for at in (16, 48, 112, 240):
        o = c.attend(ws=whole[at:at + n])
        assert_device_ok()
        c.check(o)
        assert (whole[:at] == 0xAB).all() and (whole[at + n:] == 0xAB).all()
        whole.fill_(0xAB)


def run_writer(q3, what, c, n, s_max=100, seed=0):
    """One of the writers on random inputs: (tensors it may write, as they were before, row of each token)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    B, width = len(c.ctx), (c.hq + 2 * c.hkv) * D
    qkv, ck, cv = rnd(n, width), rnd(B, c.hkv, s_max, D), rnd(B, c.hkv, s_max, D)
    out = torch.full((n, c.hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    may = {"norm": [c.k, c.v, out], "to": [c.k, c.v], "from": [ck, cv]}[what]
    old = [raw(t).clone() for t in may]
    if what == "norm":
        q3.op_qk_norm_rope_paged(c.cfg, qkv, n, c.batch, one, one, c.pages, rope_gpu(c.cfg), out)
    elif what == "to":
        q3.op_kv_to_pages(c.cfg, q3.kv_layer(ck, cv, s_max), n, c.batch, c.pages)
    else:
        q3.op_kv_from_pages(c.cfg, c.pages, n, c.batch, q3.kv_layer(ck, cv, s_max))
    status = q3.check_device_error()
    return status, [raw(t) for t in may], old


def cells_written(c, what, now, old):
    """Positions (sequence, position) whose cells changed, from a cache writer's tensors."""
    changed = (now[0] != old[0]).any(-1).any(1)  # pages: [page, slot]; contiguous: [sequence, position]
    if what == "from":
        return {(int(b), int(p)) for b, p in changed.nonzero().tolist()}
    got = {(int(p), int(s)) for p, s in changed.nonzero().tolist()}
    where = {(int(c.table[b, p // c.page]), p % c.page): (b, p) for b in range(len(c.ctx)) for p in range(c.table.shape[1] * c.page)
             if c.table[b, p // c.page] < c.n_pages}
    return {where[x] for x in got}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["norm", "to", "from"])
@pytest.mark.parametrize("start,served", [
    ([3, 0], 0), ([-5, 3], 0), ([0, 10, 5, 20], 10), ([0, 2 ** 31 - 1], 0), ([0, 20, 15], 20), ([0, 5, -1, 20], 5), ([0, 5, 21], 5),
    ([0] + [4] * 40 + [3] + [20] * 3, 4), ([0] + [20] * 70 + [19], 20)])
def test_writers_report_bad_row_lists(q3, what, start, served, fp8):
    """Every decrease, and every entry outside [0, n_tokens], is reported, wherever it stands; the
    tokens before it are written, none at or behind it."""
    n, B = 20, len(start) - 1
    c = Case(q3, [20] * B, [16] * B, 16, fp8=fp8, seed=6)
    c.t_start.copy_(torch.tensor(start, dtype=torch.int32))
    status, now, old = run_writer(q3, what, c, n)
    assert status == q3.EINVAL
    assert cells_written(c, what, now, old) == {(0, 16 + t) for t in range(served)}
    if what == "norm":
        rows = (now[2] != old[2]).any(-1)
        assert rows[:served].all() and not rows[served:].any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["norm", "to", "from", "attend1", "attend7"])
def test_rows_before_the_first_sequence(q3, what, fp8):
    """A batch may begin behind row 0 of the token buffers (one of several batches over the same
    rows): the rows before it belong to no sequence, in all four calls."""
    one = what == "attend1"
    qlens, ctx = ([1, 1, 1] if one else [7, 0, 3]), [30, 5, 60]
    c = Case(q3, qlens, ctx, 16, fp8=fp8, seed=6)
    first, n = 4, 4 + sum(qlens) + 2
    c.t_start.add_(first)
    c.q_start = c.q_start + first
    c.n = n
    if what.startswith("attend"):
        c.q = torch.randn(n, c.hq * D, device="cuda").bfloat16()
        o = c.attend()
        assert_device_ok()
        ref, tol = c.reference()
        assert (np.abs(f64(o)[first:-2] - ref) <= tol).all() and (o[:first] == 7.0).all() and (o[-2:] == 7.0).all()
        return
    status, now, old = run_writer(q3, what, c, n)
    assert status == q3.OK
    assert cells_written(c, what, now, old) == {(b, x + t) for b, (m, x) in enumerate(zip(qlens, ctx)) for t in range(m)}
    if what == "norm":
        rows = (now[2] != old[2]).any(-1)
        assert rows[first:-2].all() and not rows[:first].any() and not rows[-2:].any()


def cells(c, pool, b, first, last):
    """View-like access to positions first..last-1 of a sequence: index tuple into a page tensor."""
    p = np.arange(first, last)
    return (torch.from_numpy(c.table[b, p // c.page]).long().cuda(), slice(None), torch.from_numpy(p % c.page).cuda())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q", [1, 3])
@pytest.mark.parametrize("ctx,first", [(130, 128), (258, 256), (2, 0), (40000, 39936)])
def test_nan_keys_of_one_tile_reach_the_output(q3, q, ctx, first, fp8):
    """A KV tile of which every key is NaN, alone in its partial maximum: the row is NaN, not the mean
    over the other tiles."""
    c = Case(q3, [q], [ctx], 128, fp8=fp8, seed=2)
    c.darken()
    c.k.view(torch.uint8)[cells(c, c.k, 0, first, ctx + q)] = 0x7F if fp8 else 0xFF
    o = c.attend()
    assert_device_ok()
    assert torch.isnan(o).all()


@pytest.mark.parametrize("qlens,ctx", [([1], [200]), ([1, 1], [9000, 40]), ([5], [700]), ([200], [100]), ([1] * 17 + [30], [300] * 18)])
def test_attended_infinities(q3, qlens, ctx):
    """bf16 values of +inf and -inf, in dims of their own and in keys whose weights have any bits: the
    outputs of those dims are the infinities, the others are right."""
    c = Case(q3, qlens, ctx, 32, seed=5, sharp=0.5)
    c.darken()
    ref, tol = c.reference()
    inf = float("inf")
    for b, x in enumerate(ctx):
        for p in (0, 3, x // 2, x - 1):
            at = cells(c, c.v, b, p, p + 1)
            v = c.v[at]
            v[..., 17], v[..., 90] = inf, -inf
            c.v[at] = v
    got = f64(c.attend()).reshape(-1, c.hq, D)
    assert_device_ok()
    assert (got[..., 17] == inf).all() and (got[..., 90] == -inf).all()
    keep = np.ones(D, dtype=bool)
    keep[[17, 90]] = False
    assert (np.abs(got - ref.reshape(got.shape)) <= tol.reshape(got.shape))[..., keep].all()


@pytest.mark.parametrize("ks", [2.0 ** -126, 1e-9, 1.0, 1e18])
@pytest.mark.parametrize("qlens", [[1, 1], [200, 3], [1] * 17 + [40]])
def test_zero_and_tiny_queries_under_any_scale(q3, qlens, ks):
    """Rows of zeros and of the smallest normal values attend evenly, whatever the keys' scale."""
    c = Case(q3, qlens, [150 + b for b in range(len(qlens))], 16, fp8=True, seed=4)
    c.darken()
    c.ks.fill_(ks)
    c.ks64 = f64(c.ks)
    c.q.zero_()
    c.q[1::2, ::3] = 2.0 ** -126
    c.q[1::2, 1::3] = -(2.0 ** -120)
    o = c.attend()
    assert_device_ok()
    c.check(o)


@pytest.mark.parametrize("qlens", [[1, 1], [130, 1]])
def test_queries_at_the_end_of_bf16(q3, qlens):
    """Queries of 2^127 and above (up to bf16's largest, 3.4e38) over e4m3 keys that bring their
    scores to a few units: they are scaled into e4m3's range, not past it."""
    c = Case(q3, qlens, [170, 40], 32, fp8=True, seed=7)
    sign = torch.where(torch.rand(c.q.shape, device="cuda") < 0.5, -1.0, 1.0)
    c.q.copy_(sign * (1.75 + 0.24 * torch.rand(c.q.shape, device="cuda")) * 2.0 ** 127)
    assert torch.isfinite(c.q).all() and float(c.q.abs().max()) > 3.35e38
    c.ks.fill_(2.0 ** -126)
    c.ks64 = f64(c.ks)
    c.k.copy_((torch.randn(c.k.shape, device="cuda") * 0.5).to(c.k.dtype))
    c.darken()
    o = c.attend()
    assert_device_ok()
    c.check(o)


def one_hot_values(c, b, n):
    """V of position p < 128 is 1 in dim p: output dim p is the weight of position p."""
    at = cells(c, c.v, b, 0, n)
    v = torch.zeros(n, c.hkv, D, device="cuda")
    v[torch.arange(D), :, torch.arange(D)] = 1.0
    c.v[at] = v.to(c.v.dtype)
    c.vs.fill_(1.0)
    c.vs64 = f64(c.vs)


@pytest.mark.parametrize("qlen,bound", [(1, 2.0 ** -21), (2, 2.0 ** -16)])
def test_small_parts_of_a_query_reach_the_scores(q3, qlen, bound):
    """Weights read back one by one: the score of key p is q_p alone, a value far below the query's
    largest, which the two e4m3 terms hold to `bound` of that largest (decode and chunk form)."""
    c = Case(q3, [qlen], [127], 128, fp8=True, seed=1)
    hq, n = c.hq, 127 + qlen
    # key p: 448 in dim p (dims 1 to 127), position 0 all zeros
    k = torch.zeros(n, c.hkv, D, device="cuda")
    p = torch.arange(1, 127)
    k[p, :, p] = 448.0
    c.k.view(torch.uint8).zero_()
    c.k[cells(c, c.k, 0, 0, n)] = k.to(c.k.dtype)
    one_hot_values(c, 0, n)
    # a scale at which an error of the bound moves a score by 0.25
    ks = 0.25 / (bound * 448 / D ** 0.5)
    c.ks.fill_(ks)
    ks = float(c.ks[0])
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    size = bound * 2.0 ** (4 * torch.rand(qlen, hq, D, generator=g, device="cuda"))  # scores of 0.25 to 4
    q = torch.where(torch.rand(qlen, hq, D, generator=g, device="cuda") < 0.5, -size, size)
    q[..., 0] = 1.0  # the largest value: scaled to 128, the worst case
    c.q = q.reshape(qlen, -1).bfloat16()
    w = f64(c.attend()).reshape(qlen, hq, D)[0]
    assert_device_ok()
    got = np.log(w[:, 1:127] / w[:, :1])
    want = f64(c.q).reshape(qlen, hq, D)[0][:, 1:127] * 448 * ks / D ** 0.5
    # two outputs in bf16 (2^-8 each, in the logarithm 1.01 times that), the probability's terms (2^-11)
    assert np.abs(got - want).max() <= 0.25 + 2.02 * 2.0 ** -8 + 2.0 ** -10


@pytest.mark.parametrize("form,qlens,ctx", [("decode e4m3", [1], [2047]), ("decode e4m3", [1, 1], [127, 30000]),
                                            ("decode bf16", [1], [2047]), ("decode bf16", [1, 1], [127, 30000]),
                                            ("chunk e4m3", [2], [126]), ("chunk e4m3", [2, 1], [2046, 127])])
def test_stated_error_of_the_probabilities(q3, form, qlens, ctx):
    """Values of two groups of keys that nearly cancel: what is left is the error of the weights, which
    must stay within what the form states (a lost term would not; see test_paged_split.py)."""
    fp8 = form.endswith("e4m3")
    c = Case(q3, qlens, ctx, 128, fp8=fp8, gemm_f16=1, seed=2)
    c.darken()
    if fp8:
        c.ks.fill_(D ** 0.5)
        c.vs.fill_(1.0)
        c.ks64, c.vs64 = f64(c.ks), f64(c.vs)
    one = 1.0 if fp8 else D ** 0.5  # a score is the query's value in the dim of the key's kind
    for b, (t, x) in enumerate(zip(qlens, ctx)):
        kind = torch.from_numpy(balanced_keys(x + t)).cuda()
        k = torch.zeros(x + t, c.hkv, D, device="cuda")
        k.scatter_(2, kind[:, None, None].expand(-1, c.hkv, 1), one)
        v = torch.tensor([0.0, 1.0, -1.0], device="cuda")[kind][:, None, None].expand(-1, c.hkv, D).clone()
        v[..., 1::2] *= -1
        at = cells(c, c.k, b, 0, x + t)
        c.k[at], c.v[at] = k.to(c.k.dtype), v.to(c.v.dtype)
    q = torch.zeros(c.n, c.hq, D, device="cuda")
    q[..., :3] = torch.from_numpy(balanced_scores()).float().cuda()
    c.q = q.reshape(c.n, -1).bfloat16()
    got = f64(c.attend())
    assert_device_ok()
    ref, loose = c.reference()
    mag = (loose - 2.0 ** -11 * np.abs(ref) - 1e-7) / (2.0 ** -8 + 2.0 ** -10)
    # the weights' stated error; e4m3 terms end at 2^-23 of the largest weight (1 in each tile of 128
    # keys: 2^-16 of it summed over a tile); scores, exponentials and fp32 sums below 2^-16; fp16 output
    tol = HELD[form][2] * mag + 2.0 ** -16 * mag + (2.0 ** -16 if fp8 else 0) + 2.0 ** -11 * np.abs(ref)
    assert (np.abs(ref) < 0.03 * mag).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(6, 3), (20, 5), (7, 7), (16, 1)])
def test_odd_head_counts(q3, hq, hkv, fp8):
    """All four calls with KV heads that no power of two divides."""
    for qlens, ctx in (([1, 1, 1], [40, 700, 3]), ([90, 1, 150], [0, 260, 33])):
        c = Case(q3, qlens, ctx, 16, hq=hq, hkv=hkv, fp8=fp8, seed=hq, pad=1)
        c.darken()
        o = c.attend()
        assert_device_ok()
        c.check(o)
        for what in ("norm", "to", "from"):
            # (pages of their own: read back from pages just filled from it, a cache would not change)
            c = Case(q3, qlens, ctx, 16, hq=hq, hkv=hkv, fp8=fp8, seed=hq, pad=1)
            status, now, old = run_writer(q3, what, c, c.n, s_max=800)
            assert status == q3.OK
            want = {(b, x + t) for b, (m, x) in enumerate(zip(qlens, ctx)) for t in range(m)}
            assert cells_written(c, what, now, old) == want
            # every head of every written cell
            heads = (now[0] != old[0]).any(-1)
            heads = heads if what != "from" else heads.transpose(1, 2)
            per_cell = heads.sum(1 if what != "from" else 2)
            assert set(per_cell.unique().tolist()) <= {0, hkv}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,max_q", [(1, 1), (5, 1), (3, 40), (20, 40)])
def test_batches_without_a_token(q3, B, max_q, fp8):
    """Every sequence empty, rows that belong to none: nothing is written, nothing reported; every
    form of the attention."""
    c = Case(q3, [0] * B, [50] * B, 16, fp8=fp8, pad=4, spare=8)
    o = c.attend(max_q=max_q)
    assert_device_ok()
    assert (o == 7.0).all()
    for what in ("norm", "to", "from"):
        status, now, old = run_writer(q3, what, c, c.n)
        assert status == q3.OK and all(torch.equal(a, b) for a, b in zip(now, old))


@pytest.mark.parametrize("vs", [2.0 ** -126, 1e-30, 1e35])
@pytest.mark.parametrize("qlens,ctx", [([1, 1], [30000, 700]), ([1], [60]), ([300, 1], [0, 40]), ([40], [9000]), ([1] * 17 + [40], [300] * 18)])
def test_values_of_any_scale(q3, qlens, ctx, vs):
    """The values' scale from the smallest normal number to one that brings 448 near fp32's end: whole
    rows and rows joined from partials."""
    c = Case(q3, qlens, ctx, 32, fp8=True, seed=9)
    c.darken()
    c.vs.fill_(vs)
    c.vs64 = np.ones(c.hkv)  # the reference in units of the scale
    ref, tol = c.reference()
    got = f64(c.attend()) / float(c.vs[0])
    assert_device_ok()
    assert (np.abs(got - ref) <= tol + 2.0 ** -134 / vs).all()  # bf16 ends at steps of 2^-133
