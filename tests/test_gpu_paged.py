"""The paged KV cache's operators against float64: norm + rotation + write, attention over
pages, moves between pages and a contiguous cache; bf16 and e4m3 pages.

Tolerances. A 16-bit output is off by at most half a step of its type, relative to the value
(bf16 2^-8, fp16 2^-11). Inside the attention the probabilities are rounded to bf16 or finer,
at most 2^-8 of each, so the output moves by at most 2^-8 sum_j w_j |v_j|; scores in fp32 (a sum
of 128 products, error under 128 * 2^-24 of sum |q k| / sqrt(128), far below 2^-10 in the exponent
for these inputs) and the approximate exponential add less than 2^-10 of the same sum."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from helpers import assert_device_ok, rope_gpu  # noqa: E402

D = 128


@pytest.fixture(scope="module")
def q3():
    import qwen3_decoder_block_b200 as m
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    """A ragged batch over shuffled pages; every cell that no sequence has reached holds NaN."""

    def __init__(self, q3, qlens, ctx, page=16, hq=16, hkv=8, fp8=False, seed=0, pad=0, spare=2, ldq_extra=0,
                 gemm_f16=0, sharp=2.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.q3, self.qlens, self.ctx, self.page, self.hq, self.hkv, self.fp8 = q3, qlens, ctx, page, hq, hkv, fp8
        self.cfg = q3.make_config(n_q_heads=hq, n_kv_heads=hkv, gemm_f16=gemm_f16)
        B = len(qlens)
        need = [-(-(a + b) // page) for a, b in zip(qlens, ctx)]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((B, max(max(need), 1)), self.n_pages + 7, dtype=np.int32)  # bad ids where nothing reads
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        self.n = int(self.q_start[-1]) + pad
        self.t_start, self.t_ctx = (torch.tensor(x, dtype=torch.int32).cuda() for x in (self.q_start, np.array(ctx)))
        self.t_table = torch.from_numpy(self.table).cuda()
        self.batch = q3.paged_batch(self.t_start, self.t_ctx, self.t_table)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        k, v = rnd(self.n_pages, hkv, page, D), rnd(self.n_pages, hkv, page, D)
        self.ks = self.vs = None
        self.ks64 = self.vs64 = np.ones(hkv)
        if fp8:
            self.ks = (5 + torch.rand(hkv, generator=g, device="cuda")) / 448
            self.vs = (5 + torch.rand(hkv, generator=g, device="cuda")) / 448
            self.ks64, self.vs64 = f64(self.ks), f64(self.vs)
            k = (k.float() / self.ks[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            v = (v.float() / self.vs[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        self.k, self.v = k, v
        width = hq * D
        self.ldq = width + ldq_extra
        self.q = torch.full((max(self.n, 1), self.ldq), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.q[:self.n, :width] = (sharp * rnd(self.n, width).float()).to(torch.bfloat16)
        self.otype = torch.float16 if gemm_f16 else torch.bfloat16
        self.pages = q3.kv_pages(self.k, self.v, self.ks, self.vs)

    def darken(self):
        seen = np.zeros((self.n_pages, self.page), dtype=bool)
        for b, (t, c) in enumerate(zip(self.qlens, self.ctx)):
            p = np.arange(t + c if t else 0)
            seen[self.table[b, p // self.page], p % self.page] = True
        dark = ~torch.from_numpy(seen).cuda()[:, None, :, None]
        raw, nan = (torch.uint8, 0x7F) if self.fp8 else (torch.int16, 0x7FC0)
        self.k.view(raw).masked_fill_(dark, nan)
        self.v.view(raw).masked_fill_(dark, nan)

    def rows(self, pool, scale, b, n):
        """float64 [n, hkv, D] of a sequence's first n cached positions."""
        p = np.arange(n)
        page, slot = (torch.from_numpy(x).long().cuda() for x in (self.table[b, p // self.page], p % self.page))
        raw = pool.view(torch.uint8) if self.fp8 else pool
        cells = raw[page, :, slot].view(pool.dtype)
        return f64(cells.float() if self.fp8 else cells) * scale[:, None]

    def attend(self, max_q=None, ldo_extra=0, ws=None, stream=None, out=None):
        q3 = self.q3
        width = self.hq * D
        max_q = max_q or max(max(self.qlens), 1)
        o = out if out is not None else torch.full((self.n, width + ldo_extra), 7.0, dtype=self.otype, device="cuda")
        if ws is None:
            n = q3.workspace_size(self.cfg, q3.OP_ATTENTION_PAGED, len(self.qlens), max_q, 1)
            ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
        q3.op_attention_paged(self.cfg, self.q, self.n, max_q, self.batch, self.pages, o, ws, ldq=self.ldq,
                              ldo=width + ldo_extra, stream=stream)
        return o

    def reference(self):
        """Outputs and tolerances [q_start[B], hq * D]."""
        G = self.hq // self.hkv
        refs, mags = [], []
        for b, (t, c) in enumerate(zip(self.qlens, self.ctx)):
            if not t:
                continue
            K, V = self.rows(self.k, self.ks64, b, c + t), self.rows(self.v, self.vs64, b, c + t)
            r0 = self.q_start[b]
            Q = f64(self.q[r0:r0 + t, :self.hq * D]).reshape(t, self.hkv, G, D)
            s = np.einsum("thgd,shd->thgs", Q, K) / np.sqrt(D)
            mask = np.arange(c + t)[None, :] > c + np.arange(t)[:, None]
            s = np.where(mask[:, None, None, :], -np.inf, s)
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            refs.append(np.einsum("thgs,shd->thgd", w, V).reshape(t, -1))
            mags.append(np.einsum("thgs,shd->thgd", w, np.abs(V)).reshape(t, -1))
        ref, mag = np.concatenate(refs), np.concatenate(mags)
        half = 2.0 ** -11 if self.otype == torch.float16 else 2.0 ** -8
        return ref, half * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag + 1e-7

    def check(self, o, pad_value=7.0):
        ref, tol = self.reference()
        width = self.hq * D
        got = f64(o)
        n = len(ref)
        bad = np.abs(got[:n, :width] - ref) > tol
        assert not bad.any() and np.isfinite(got[:n, :width]).all(), (
            np.argwhere(bad)[:5], float(np.nanmax(np.abs(got[:n, :width] - ref) / tol)))
        assert (got[n:] == pad_value).all() and (got[:, width:] == pad_value).all()


# one token: lengths around tile and page borders, empty sequences, a long axis
ONE = [([1], [0], 16), ([1], [15], 16), ([1], [127], 128), ([1, 1, 1], [128, 129, 255], 32), ([1], [500], 64),
       ([1, 0, 1, 1], [3000, 50, 17, 1], 256), ([1] * 9, [5, 700, 64, 63, 65, 1023, 2, 383, 384], 16), ([1], [20011], 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens,ctx,page", ONE)
def test_attention_one_token(q3, qlens, ctx, page, fp8):
    c = Case(q3, qlens, ctx, page, fp8=fp8, pad=3, seed=len(ctx) + sum(ctx))
    c.darken()
    o = c.attend()
    assert_device_ok()
    c.check(o)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(16, 16), (16, 8), (16, 4), (32, 4), (16, 1)])
@pytest.mark.parametrize("qmax", [1, 70])
def test_attention_group_sizes(q3, hq, hkv, fp8, qmax):
    qlens = [1, 1, 1] if qmax == 1 else [1, 70, 33]
    c = Case(q3, qlens, [300, 45, 1000], 64, hq=hq, hkv=hkv, fp8=fp8, seed=hq * 7 + hkv)
    c.darken()
    o = c.attend()
    assert_device_ok()
    c.check(o)


# chunks: one row to several tiles, contexts of none to many pages, mixed with decode rows
CHUNKS = [([2], [0], 16), ([64], [0], 16), ([65], [63], 32), ([128], [128], 128), ([129], [1], 256),
          ([300], [0], 64), ([1, 200, 0, 3, 77], [900, 33, 40, 0, 129], 16), ([7, 7, 7], [2000, 3, 500], 128),
          ([1000], [1500], 64), ([17], [9000], 32),
          ([1, 90, 1, 1, 0, 1, 2, 1, 1, 64, 1, 1, 1, 1, 1, 1, 3, 1], [700, 300, 0, 5, 9, 2000, 127, 128, 64, 0, 31, 1, 900, 77, 255, 256, 10, 63], 16),
          ([1] * 16 + [2], [40 * i for i in range(17)], 128), ([5] * 20, [33 * i for i in range(20)], 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens,ctx,page", CHUNKS)
def test_attention_chunks(q3, qlens, ctx, page, fp8):
    c = Case(q3, qlens, ctx, page, fp8=fp8, pad=5, seed=3 * len(ctx) + sum(ctx) + sum(qlens))
    c.darken()
    o = c.attend()
    assert_device_ok()
    c.check(o)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[1, 1], [40, 1]])
def test_attention_strides_f16_and_loose_bound(q3, qlens, fp8):
    c = Case(q3, qlens, [200, 77], 32, fp8=fp8, ldq_extra=2048, gemm_f16=1)
    c.darken()
    for max_q in (max(qlens), 512):
        o = c.attend(max_q=max_q, ldo_extra=64)
        assert_device_ok()
        c.check(o)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[1, 1, 1], [100, 1, 20]])
def test_attention_sharp_and_flat_rows(q3, qlens, fp8):
    """Scores spread over hundreds (one key takes all), all equal (zero queries), and one key far
    above thousands of equal ones, whose small weights still add up."""
    for sharp in (40.0, 0.0):
        c = Case(q3, qlens, [2000, 1300, 64], 64, fp8=fp8, sharp=sharp)
        c.darken()
        o = c.attend()
        assert_device_ok()
        c.check(o)
    c = Case(q3, qlens, [6000, 6000, 6000], 64, fp8=fp8)
    # keys all zero but position 0 along dim 0; queries give it a lead of about ln(2^13)
    one = (c.k[:1, :1, :1, :1].float() * 0 + 1).to(c.k.dtype)
    c.k.view(torch.uint8).zero_()
    for b in range(3):
        c.k[int(c.table[b, 0]), :, 0, 0] = one[0, 0, 0, 0]
    lead = 13 * np.log(2) * np.sqrt(D)
    c.q.zero_()
    c.q.view(-1, D)[:, 0] = float(lead if not fp8 else lead / c.ks64.mean())
    o = c.attend()
    assert_device_ok()
    c.check(o)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[1, 1, 1], [130, 2, 1]])
def test_attention_repeats_bit_for_bit_and_replays(q3, qlens, fp8):
    """The same call twice, and from a graph on another stream, gives the same bits; the graph
    follows lengths and queries that change between replays; dirty workspaces do not matter."""
    c = Case(q3, qlens, [5000, 700, 90], 32, fp8=fp8)
    c.darken()
    a, b = c.attend(), c.attend()
    assert torch.equal(a, b)
    n = q3.workspace_size(c.cfg, q3.OP_ATTENTION_PAGED, 3, max(qlens), 1)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full_like(a, 7.0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.attend(ws=ws, out=o)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, o)
    c.ctx = [4000, 31, 0]
    c.t_ctx.copy_(torch.tensor(c.ctx, dtype=torch.int32))
    c.q.copy_(c.q.flip(0))
    o.fill_(7.0)
    for _ in range(3):
        graph.replay()
    assert_device_ok()
    c.check(o)


def test_attention_two_calls_at_once(q3):
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    cases = [Case(q3, [1, 1], [9000, 800], 64, fp8=False, seed=1), Case(q3, [300, 1], [3000, 50], 16, fp8=True, seed=2)]
    alone = [c.attend() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs, keep = [torch.full_like(a, 7.0) for a in alone], []
    for c in cases:
        n = q3.workspace_size(c.cfg, q3.OP_ATTENTION_PAGED, 2, max(c.qlens), 1)
        keep.append(torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, o, ws in zip(cases, streams, outs, keep):
            c.attend(stream=s, out=o, ws=ws)
    torch.cuda.synchronize()
    assert_device_ok()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[1, 1, 1], [20, 9, 1]])
def test_attention_reports_bad_sequences(q3, qlens, fp8):
    """A bad sequence is reported and left alone; the others come out right."""
    def run(status, change, hurt, same_rows=True):
        c = Case(q3, qlens, [100, 200, 300], 16, fp8=fp8, seed=5)
        kw = change(c) or {}
        o = c.attend(**kw)
        assert q3.check_device_error() == status
        assert q3.check_device_error() == q3.OK
        got = f64(o)
        ref, tol = c.reference()
        for b in range(3):
            r = slice(c.q_start[b], c.q_start[b + 1])
            if b != hurt:
                assert (np.abs(got[r] - ref[r]) <= tol[r]).all()
            elif same_rows:
                assert (got[r] == 7.0).all()

    def set_ctx(b, value):
        def f(c):
            c.t_ctx[b] = value
        return f

    run(q3.EINVAL, set_ctx(1, -1), 1)
    run(q3.ECAPACITY, set_ctx(1, 16 * 20), 1)  # the table holds 19 or 20 pages a sequence
    run(q3.ECAPACITY, set_ctx(0, 2 ** 31 - 5), 0)

    def page(value):
        def f(c):
            c.t_table[1, 2] = value
        return f

    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        run(q3.EINVAL, page(bad), 1, same_rows=False)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_mixed_batch_reports_and_serves(q3, fp8):
    """A batch large enough for both forms of the kernel, with bad decode and chunk sequences."""
    qlens = [1, 40, 1, 1, 9, 1, 1, 200, 1, 1, 1, 0, 1, 1, 2, 1, 1, 1]
    ctx = [50 * i + 3 for i in range(18)]
    c = Case(q3, qlens, ctx, 32, fp8=fp8, seed=8, pad=2)
    c.t_ctx[2] = -7
    c.t_ctx[7] = 10 ** 6
    o = c.attend()
    assert q3.check_device_error() in (q3.EINVAL, q3.ECAPACITY)
    got, (ref, tol) = f64(o), c.reference()
    for b in range(18):
        r = slice(c.q_start[b], c.q_start[b + 1])
        if b in (2, 7):
            assert (got[r] == 7.0).all()
        else:
            assert (np.abs(got[r] - ref[r]) <= tol[r]).all(), b
    assert (got[c.q_start[-1]:] == 7.0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q", [1, 2])
def test_attention_many_sequences(q3, q, fp8):
    """More sequences than the plan keeps in shared memory."""
    B = 1100
    c = Case(q3, [q if b % 7 else 0 for b in range(B)], [(37 * b) % 200 for b in range(B)], 16, hq=4, hkv=2, fp8=fp8)
    c.darken()
    o = c.attend()
    assert_device_ok()
    c.check(o)


@pytest.mark.parametrize("qlens", [[1, 1], [150, 1]])
def test_attention_graphs_share_a_workspace(q3, qlens):
    """Two captured calls with one workspace, replayed in turn on one stream."""
    cases = [Case(q3, qlens, [4000, 100], 32, seed=1), Case(q3, qlens, [10, 2500], 32, fp8=True, seed=2)]
    want = [c.attend() for c in cases]
    n = q3.workspace_size(cases[0].cfg, q3.OP_ATTENTION_PAGED, 2, max(qlens), 1)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.full_like(w, 7.0) for w in want], []
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.attend(ws=ws, out=o)
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    assert_device_ok()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)


def test_attention_nan_and_huge_keys_behind_a_token(q3):
    """Keys of later tokens of the same call may hold anything: their scores are masked."""
    for fp8 in (False, True):
        c = Case(q3, [6], [130], 32, fp8=fp8)
        c.darken()
        ref, tol = c.reference()
        p = 135  # the last token's position
        c.k[int(c.table[0, p // 32]), :, p % 32].view(torch.uint8).fill_(0x7F)
        o = f64(c.attend())
        assert_device_ok()
        assert (np.abs(o[:5] - ref[:5]) <= tol[:5]).all()
        # the bytes are NaN in e4m3 (and 3.4e38 in bf16, a score like any other)
        assert not fp8 or np.isnan(o[5]).all()


def test_attention_reports_too_many_tokens(q3):
    c = Case(q3, [3, 20], [100, 200], 16)
    o = c.attend(max_q=8)
    assert q3.check_device_error() == q3.EINVAL
    got, (ref, tol) = f64(o), c.reference()
    assert (np.abs(got[:3] - ref[:3]) <= tol[:3]).all() and (got[3:] == 7.0).all()
    c = Case(q3, [1, 2], [100, 200], 16)
    o = c.attend(max_q=1)
    assert q3.check_device_error() == q3.EINVAL
    got, (ref, tol) = f64(o), c.reference()
    assert (np.abs(got[:1] - ref[:1]) <= tol[:1]).all() and (got[1:] == 7.0).all()


# ------------------------------------------------------------------------- norm, rotation, write
def half_step_e4m3(x):
    """Half a step of e4m3 at |x| (values up to 448): steps of 2^-9 below 2^-6."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return 2.0 ** (e - 4)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens,ctx,page,hq,hkv", [
    ([1], [0], 16, 16, 8), ([1, 1, 1, 1, 1], [0, 15, 16, 17, 4000], 16, 16, 8), ([5, 0, 1, 130], [3, 9, 127, 250], 64, 32, 4),
    ([40, 2], [0, 300], 256, 16, 1), ([33], [31], 32, 16, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_qk_norm_rope_paged(q3, qlens, ctx, page, hq, hkv, fp8, in_place):
    import oracle.qwen3_ref as R
    c = Case(q3, qlens, ctx, page, hq, hkv, fp8=fp8, pad=4)
    n, width = c.n, (hq + 2 * hkv) * D
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    qkv = rnd(n, width + 8)
    qw, kw = (1 + 0.1 * rnd(D).float()).bfloat16(), (1 + 0.1 * rnd(D).float()).bfloat16()
    rope = rope_gpu(c.cfg)
    x = f64(qkv)
    k0, v0 = f64(c.k.float()), f64(c.v.float())
    if in_place:
        out, ldq = qkv, width + 8
    else:
        out, ldq = torch.full((n, hq * D + 16), 7.0, dtype=torch.bfloat16, device="cuda"), hq * D + 16
    q3.op_qk_norm_rope_paged(c.cfg, qkv, n, c.batch, qw, kw, c.pages, rope, out, ldqkv=width + 8, ldq=ldq)
    assert_device_ok()
    got = f64(out)
    k1, v1 = f64(c.k.float()), f64(c.v.float())
    eps = float(np.float32(1e-6))
    touched = np.zeros((c.n_pages, page), dtype=bool)
    for b, (t, cx) in enumerate(zip(qlens, ctx)):
        if not t:
            continue
        r = slice(c.q_start[b], c.q_start[b + 1])
        pos = np.arange(cx, cx + t)
        h = x[r, :width].reshape(t, hq + 2 * hkv, D)
        cos, sin = R.rope_tables(pos, D, 1e6) if hasattr(R, "rope_tables") else (None, None)
        if cos is None or cos.shape[-1] != D // 2:
            a = pos[:, None] * 1e6 ** (-2.0 * np.arange(D // 2) / D)
            cos, sin = np.cos(a), np.sin(a)

        def turn(y, w):
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * f64(w)
            lo, hi = y[..., :64], y[..., 64:]
            co, si = cos[:, None], sin[:, None]
            return np.concatenate([lo * co - hi * si, lo * si + hi * co], -1)

        q = turn(h[:, :hq], qw).reshape(t, -1)
        assert (np.abs(got[r, :hq * D] - q) <= 2.0 ** -8 * np.abs(q) + 4e-6).all()
        pg, slot = c.table[b, pos // page], pos % page
        touched[pg, slot] = True
        for new, want, scale in ((k1, turn(h[:, hq:hq + hkv], kw), c.ks64), (v1, h[:, hq + hkv:], c.vs64)):
            cell = new[pg, :, slot]
            want = want / scale[:, None]
            if fp8:  # fp32 rounding of the value may move it across a border: a hair more than half a step
                want = np.clip(want, -448, 448)
                assert (np.abs(cell - want) <= half_step_e4m3(want) * (1 + 1e-4) + 1e-5 * np.abs(want)).all()
            else:
                assert (np.abs(cell - want) <= 2.0 ** -8 * np.abs(want) + 4e-6).all()
    for new, old in ((k1, k0), (v1, v0)):
        assert np.array_equal(new.transpose(0, 2, 1, 3)[~touched], old.transpose(0, 2, 1, 3)[~touched])
    last = c.q_start[-1]
    if in_place:
        assert np.array_equal(got[last:], x[last:]) and np.array_equal(got[:, hq * D:], x[:, hq * D:])
    else:
        assert (got[last:] == 7.0).all() and (got[:, hq * D:] == 7.0).all()


def test_e4m3_write_saturates_and_keeps_nan(q3):
    c = Case(q3, [2], [0], 16, fp8=True)
    qkv = torch.zeros(2, 32 * D, dtype=torch.bfloat16, device="cuda")
    v = qkv.view(2, 32, D)[:, 24:]
    v[0, 0, :4] = torch.tensor([1e30, -1e30, float("inf"), float("nan")], dtype=torch.bfloat16, device="cuda")
    v[1, 7, :2] = torch.tensor([-float("inf"), 2.0 ** -40], dtype=torch.bfloat16, device="cuda")
    one = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2, 16 * D, dtype=torch.bfloat16, device="cuda")
    q3.op_qk_norm_rope_paged(c.cfg, qkv, 2, c.batch, one, one, c.pages, rope_gpu(c.cfg), out)
    assert_device_ok()
    cell = c.v[int(c.table[0, 0])].float()
    assert cell[0, 0, :3].tolist() == [448.0, -448.0, 448.0] and torch.isnan(cell[0, 0, 3])
    assert cell[7, 1, :2].tolist() == [-448.0, 0.0]


@pytest.mark.parametrize("what", ["norm", "to", "from"])
def test_writers_report_bad_positions(q3, what):
    """Bad lists are reported; the token's cells and rows stay as they were."""
    for status, change in ((q3.EINVAL, lambda c: c.t_ctx.fill_(-5)), (q3.ECAPACITY, lambda c: c.t_ctx.fill_(10 ** 5)),
                           (q3.EINVAL, lambda c: c.t_table.fill_(-3)), (q3.EINVAL, lambda c: c.t_table.fill_(10 ** 6)),
                           (q3.ECAPACITY, lambda c: c.t_ctx.fill_(64)),
                           (q3.EINVAL, lambda c: c.t_start.copy_(torch.tensor([3, 0], dtype=torch.int32)))):
        c = Case(q3, [3], [20], 16, seed=4)
        qkv = torch.randn(3, 32 * D, device="cuda").bfloat16()
        ck = torch.randn(1, 8, 5000, D, device="cuda").bfloat16()
        kv = q3.kv_layer(ck, ck, 5000)
        out = torch.full((3, 16 * D), 7.0, dtype=torch.bfloat16, device="cuda")
        one = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        rope = rope_gpu(c.cfg)
        before = c.k.clone(), c.v.clone(), ck.clone()
        change(c)
        if what == "norm":
            q3.op_qk_norm_rope_paged(c.cfg, qkv, 3, c.batch, one, one, c.pages, rope, out)
        elif what == "to":
            q3.op_kv_to_pages(c.cfg, kv, 3, c.batch, c.pages)
        else:
            q3.op_kv_from_pages(c.cfg, c.pages, 3, c.batch, kv)
        st = q3.check_device_error()
        if change(c) is not None and int(c.t_start[0]) == 3:
            assert st in (q3.OK, q3.EINVAL)  # [3, 0]: every row lies behind the last sequence
        else:
            assert st == status, (status, st)
        assert torch.equal(before[0], c.k) and torch.equal(before[1], c.v) and torch.equal(before[2], ck)
        assert (out == 7.0).all()


# ------------------------------------------------------------------------- moves
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens,ctx,page,hkv", [([1], [0], 16, 8), ([100, 0, 37, 1], [0, 5, 200, 127], 32, 4),
                                                ([513], [3], 256, 1), ([70, 70], [0, 1], 64, 16)])
def test_moves_both_ways(q3, qlens, ctx, page, hkv, fp8):
    c = Case(q3, qlens, ctx, page, 16, hkv, fp8=fp8, pad=6)
    B, s_max = len(qlens), max(a + b for a, b in zip(qlens, ctx)) + 5
    src = [torch.randn(B, hkv, s_max, D, device="cuda").bfloat16() for _ in range(2)]
    dst = [torch.full_like(src[0], 7.0) for _ in range(2)]
    old = [f64(c.k.float()), f64(c.v.float())]
    q3.op_kv_to_pages(c.cfg, q3.kv_layer(*src, s_max), c.n, c.batch, c.pages)
    q3.op_kv_from_pages(c.cfg, c.pages, c.n, c.batch, q3.kv_layer(*dst, s_max))
    assert_device_ok()
    new = [f64(c.k.float()), f64(c.v.float())]
    touched = np.zeros((c.n_pages, page), dtype=bool)
    for b, (t, cx) in enumerate(zip(qlens, ctx)):
        pos = np.arange(cx, cx + t)
        pg, slot = c.table[b, pos // page], pos % page
        touched[pg, slot] = True
        for i, scale in ((0, c.ks), (1, c.vs)):
            x = src[i][b, :, cx:cx + t].transpose(0, 1).float()
            want = (x * (1 / scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float() if fp8 else x
            assert np.array_equal(new[i][pg, :, slot], f64(want))
            back = (want * scale[:, None]).bfloat16() if fp8 else x.bfloat16()
            assert torch.equal(dst[i][b, :, cx:cx + t].transpose(0, 1), back)
        keep = np.ones(s_max, dtype=bool)
        keep[cx:cx + t] = False
        for d in dst:
            assert (f64(d[b])[:, keep] == 7.0).all()
    for n, o in zip(new, old):
        assert np.array_equal(n.transpose(0, 2, 1, 3)[~touched], o.transpose(0, 2, 1, 3)[~touched])


def test_far_pages(q3):
    """Pages whose byte offsets pass 2^32: write, attend, read back."""
    n_pages, page, hkv = (1 << 24) // (8 * 128) + 300, 128, 8
    cfg = q3.make_config(n_q_heads=16, n_kv_heads=hkv)
    k = torch.empty(n_pages, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[n_pages - 1, n_pages - 7]], dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    src = [torch.randn(1, hkv, 200, D, device="cuda").bfloat16() for _ in range(2)]
    dst = [torch.zeros_like(src[0]) for _ in range(2)]
    pages = q3.kv_pages(k, v)
    start, zero = i32(0, 200), i32(0)
    fill = q3.paged_batch(start, zero, table)
    q3.op_kv_to_pages(cfg, q3.kv_layer(*src, 200), 200, fill, pages)
    q3.op_kv_from_pages(cfg, pages, 200, fill, q3.kv_layer(*dst, 200))
    assert torch.equal(src[0], dst[0]) and torch.equal(src[1], dst[1])
    kv = q3.kv_layer(*src, 200)
    for nq in (1, 130):
        q = torch.randn(nq, 16 * D, device="cuda").bfloat16()
        s2, c2 = i32(0, nq), i32(200 - nq)
        o = torch.empty(nq, 16 * D, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(q3.workspace_size(cfg, q3.OP_ATTENTION_PAGED, 1, nq, 200), dtype=torch.uint8, device="cuda")
        q3.op_attention_paged(cfg, q, nq, nq, q3.paged_batch(s2, c2, table), pages, o, ws)
        w = torch.empty_like(o)
        q3.op_attention_prefill(cfg, torch.cat([q, q], 1).contiguous(), 1, nq, c2, kv, w)
        assert_device_ok()
        assert (o.float() - w.float()).abs().max() <= 2.0 ** -6 * w.float().abs().max()


# ------------------------------------------------------------------------- together
@pytest.mark.parametrize("fp8", [False, True])
def test_serving_run_of_the_operators(q3, fp8):
    """Three prompts cached by the contiguous path move into pages; the batch then takes a chunk
    and two decode tokens through norm + write + attention, in three calls; each call's output
    matches float64 over everything cached so far, and the pages read back feed the contiguous
    decode attention."""
    import oracle.qwen3_ref as R  # noqa: F401
    hq, hkv, page = 16, 8, 32
    c = Case(q3, [60, 1, 200], [150, 99, 0], page, hq, hkv, fp8=fp8, spare=40)
    B, s_max = 3, 512
    cfg, rope = c.cfg, rope_gpu(c.cfg)
    full = torch.arange(3 * 14, dtype=torch.int32).view(3, 14)
    c.table = full.numpy()
    assert c.n_pages >= 42
    c.t_table = full.cuda()
    c.k.view(torch.uint8).zero_()
    c.v.view(torch.uint8).zero_()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    one = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    # prompts of 150, 99 and 0 tokens in a contiguous cache
    kv_t = [torch.randn(B, hkv, s_max, D, device="cuda").bfloat16() for _ in range(2)]
    start, ctx = i32([0, 150, 249, 249]), i32([0, 0, 0])
    q3.op_kv_to_pages(cfg, q3.kv_layer(*kv_t, s_max), 249, q3.paged_batch(start, ctx, c.t_table), c.pages)
    lens = [150, 99, 0]
    for qlens in ([60, 1, 200], [1, 1, 1], [1, 0, 1]):
        n = sum(qlens)
        c.qlens, c.ctx, c.n = qlens, list(lens), n
        c.q_start = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        start, ctx = i32(c.q_start.tolist()), i32(lens)
        c.batch = q3.paged_batch(start, ctx, c.t_table)
        qkv = torch.randn(n, (hq + 2 * hkv) * D, device="cuda").bfloat16()
        c.q, c.ldq = torch.empty(n, hq * D, dtype=torch.bfloat16, device="cuda"), hq * D
        q3.op_qk_norm_rope_paged(cfg, qkv, n, c.batch, one, one, c.pages, rope, c.q)
        o = c.attend()
        assert_device_ok()
        c.check(o)
        lens = [a + b for a, b in zip(lens, qlens)]
    # back to a contiguous cache: its decode attention agrees with the paged one
    start, ctx = i32([0, lens[0], lens[0] + lens[1], sum(lens)]), i32([0, 0, 0])
    back = [torch.zeros(B, hkv, s_max, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv = q3.kv_layer(*back, s_max)
    q3.op_kv_from_pages(cfg, c.pages, sum(lens), q3.paged_batch(start, ctx, c.t_table), kv)
    q = torch.randn(B, hq * D, device="cuda").bfloat16()
    last = i32([x - 1 for x in lens])
    ws = torch.empty(q3.workspace_size(cfg, q3.OP_BLOCK_DECODE, B, 1, s_max), dtype=torch.uint8, device="cuda")
    want = torch.empty(B, hq * D, dtype=torch.bfloat16, device="cuda")
    q3.op_attention_decode(cfg, q, B, last, kv, want, ws, ldqkv=hq * D)
    c.q, c.qlens, c.ctx, c.n = q, [1, 1, 1], [x - 1 for x in lens], 3
    c.q_start = np.arange(4, dtype=np.int32)
    start = i32([0, 1, 2, 3])
    c.batch = q3.paged_batch(start, last, c.t_table)
    o = c.attend()
    assert_device_ok()
    c.check(o)
    # bf16 read-back of e4m3 rounds K and V once more (2^-8 of each); the outputs stay that near
    assert (o.float() - want.float()).norm() <= 2.0 ** -5 * want.float().norm()
