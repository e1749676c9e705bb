"""The paged KV cache's operators as they are measured: real sizes, plain forms, exact results.

Four operators belong together: the per-head QK norm with the rotation that writes a
ragged batch's keys and values into pages (``qk_norm_rope_paged``), the attention of the
batch's new tokens over those pages (``attention_paged``), and the moves between the pages
and a contiguous cache (``kv_to_pages``, ``kv_from_pages``). Pages hold bf16, or e4m3 with
one fp32 scale per KV head.
"""
from __future__ import annotations

import random

import torch

own = False

HEAD_DIM = 128
MAX_POS = 40960
THETA = 1.0e6
EPS = 1.0e-6
OPS = ("attention", "norm_rope", "to_pages", "from_pages")


def _case(name, op, fp8, page, B, ctx_lo, ctx_hi, q_lo, q_hi, n_single=0, pad=0, hq=16, hkv=8, lens=1):
    """One case. ctx_lo..ctx_hi: cached tokens of a sequence before the call; q_lo..q_hi: its new
    tokens; n_single: how many of the B sequences bring one token instead; pad: rows of the token
    buffers behind the last sequence; lens: seed of the lengths."""
    c = {"op": op, "fp8": fp8, "page": page, "B": B, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "q_lo": q_lo, "q_hi": q_hi,
         "n_single": n_single, "pad": pad, "hq": hq, "hkv": hkv, "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a chat turn of one user: one token over a short history, where the launches' latency counts
        _case("decode_one_ctx500", "attention", False, 16, 1, 500, 500, 1, 1),
        # a full decode batch at 4096 cached tokens, the two cache types
        _case("decode_B64_ctx4096", "attention", False, 64, 64, 4096, 4096, 1, 1),
        _case("decode_B64_ragged_fp8", "attention", True, 16, 64, 257, 8191, 1, 1, pad=5),
        # one user's long document, decoded: few rows over a long axis
        _case("decode_B2_ctx32700_fp8", "attention", True, 128, 2, 32500, 32700, 1, 1),
        # a serving step: 30 sequences decode while two prompts are prefilled in chunks
        _case("mixed_B32", "attention", False, 32, 32, 100, 4000, 300, 512, n_single=30),
        # chunked prefill of four prompts, second chunk, quantised cache
        _case("chunk_B4xT2048_fp8", "attention", True, 64, 4, 2048, 2048, 2048, 2048),
        # the last chunk of a long document
        _case("chunk_T2048_ctx30000", "attention", False, 256, 1, 30011, 30011, 2048, 2048),
        # norm, rotation and cache write: a prefill, and a decode step on a quantised cache
        _case("norm_rope_B4xT2048", "norm_rope", False, 64, 4, 0, 0, 2048, 2048),
        _case("norm_rope_decode_B64_fp8", "norm_rope", True, 16, 64, 100, 1000, 1, 1),
        # a prompt prefilled into a contiguous cache moves into quantised pages
        _case("to_pages_B8_fp8", "to_pages", True, 32, 8, 0, 0, 1500, 4096),
        # pages read back into a contiguous cache: a long quantised sequence, and short bf16 ones
        _case("from_pages_32k_fp8", "from_pages", True, 128, 1, 0, 0, 32768, 32768),
        _case("from_pages_B16", "from_pages", False, 16, 16, 0, 300, 1, 700),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "norm_rope", "to_pages", "from_pages"))
    hq, hkv = rng.choice(((16, 8), (16, 8), (32, 4), (32, 8), (16, 16), (16, 1)))
    page, fp8, lens = rng.choice((16, 32, 64, 128, 256)), rng.random() < 0.5, rng.randrange(1 << 30)
    pad = rng.choice((0, 0, rng.randrange(1, 40)))
    while True:
        B = _log_int(rng, 1, 96)
        ctx_hi = _log_int(rng, 1, 32000)
        ctx_lo = rng.randrange(0, ctx_hi + 1)
        kind = rng.choice(("single", "single", "few", "chunk", "mixed")) if op in ("attention", "norm_rope") else "chunk"
        q_hi = 1 if kind == "single" else rng.randrange(2, 17) if kind == "few" else _log_int(rng, 17, 4096)
        q_lo = q_hi if rng.random() < 0.3 else rng.randrange(1, q_hi + 1)
        n_single = rng.randrange(0, B) if kind == "mixed" else 0
        if op != "attention":
            ctx_hi = min(ctx_hi, 4096)
            ctx_lo = min(ctx_lo, ctx_hi)
        c = _case("", op, fp8, page, B, ctx_lo, ctx_hi, q_lo, q_hi, n_single, pad, hq, hkv, lens)
        q, ctx = _lengths(c)
        rows, longest = max(q), max(a + b for a, b in zip(q, ctx))
        if op == "attention":
            if B * hq * rows * longest <= 1 << 30 and B * hkv * longest <= 1 << 22 and work(c)["flops"] < 5e11:
                return c
        elif B * hkv * longest <= 1 << 19 and sum(q) * hkv <= 1 << 18:
            return c


# ------------------------------------------------------------------------- sizes of a case
def _lengths(case):
    """New tokens and cached tokens of each sequence."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    for b in r.sample(range(case["B"]), case["n_single"]):
        q[b] = 1
    return q, ctx


def work(case):
    q, ctx = _lengths(case)
    hq, hkv, D, n = case["hq"], case["hkv"], HEAD_DIM, sum(q)
    cell = 1 if case["fp8"] else 2
    pages = sum(-(-(a + b) // case["page"]) for a, b in zip(q, ctx))
    lists = 4 * (2 * case["B"] + 1 + pages)
    if case["op"] == "attention":
        pairs = sum(t * c + t * (t + 1) // 2 for t, c in zip(q, ctx))
        return {"bytes": 2 * 2 * n * hq * D + 2 * cell * hkv * D * sum(a + b for a, b in zip(q, ctx)) + lists,
                "flops": 4 * hq * D * pairs}
    if case["op"] == "norm_rope":
        rot = 4 * D * len({c + i for t, c in zip(q, ctx) for i in range(t)})
        return {"bytes": 2 * n * (hq + 2 * hkv) * D + 2 * n * hq * D + 2 * cell * n * hkv * D + rot + lists,
                "flops": 8 * n * (hq + hkv) * D}
    return {"bytes": (2 + cell) * 2 * n * hkv * D + lists, "flops": 2 * n * hkv * D if case["fp8"] else 0}


# ------------------------------------------------------------------------- inputs
def _layout(case, g):
    """The batch's lists on the GPU: token offsets, cached lengths, shuffled page table."""
    q, ctx = _lengths(case)
    dev, ps = "cuda", case["page"]
    need = [-(-(a + b) // ps) for a, b in zip(q, ctx)]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int32)
    table = torch.zeros((case["B"], max(need)), dtype=torch.int32)
    at = 0
    order = order.cpu()
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    start = torch.tensor([0] + q).cumsum(0).to(torch.int32)
    return {"q_start": start.to(dev), "ctx_len": torch.tensor(ctx, dtype=torch.int32).to(dev), "table": table.to(dev),
            "n_pages": n_pages, "n_tokens": sum(q) + case["pad"], "max_q": max(q), "page": ps,
            "longest": max(a + b for a, b in zip(q, ctx)), "hq": case["hq"], "hkv": case["hkv"], "op": case["op"],
            "fp8": case["fp8"]}


def _rope_table():
    f = THETA ** (-torch.arange(0, HEAD_DIM, 2, dtype=torch.float64, device="cuda") / HEAD_DIM)
    a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = _layout(case, g)
    hq, hkv, n, ps, D = case["hq"], case["hkv"], s["n_tokens"], case["page"], HEAD_DIM
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    k, v = normal(s["n_pages"], hkv, ps, D), normal(s["n_pages"], hkv, ps, D)
    s["k_scale"] = s["v_scale"] = None
    if case["fp8"]:
        # scales that put the largest of N(0, 1) values near e4m3's largest, another one for each head
        s["k_scale"] = (5.0 + torch.rand(hkv, generator=g, device="cuda")) / 448.0
        s["v_scale"] = (5.0 + torch.rand(hkv, generator=g, device="cuda")) / 448.0
        k = (k.float() / s["k_scale"][:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v.float() / s["v_scale"][:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    s["k"], s["v"] = k, v
    if case["op"] == "attention":
        # what no sequence has written yet holds anything, NaN too
        q, ctx = _lengths(case)
        seen = torch.zeros((s["n_pages"], ps), dtype=torch.bool)
        table = s["table"].cpu()
        for b, (t, c) in enumerate(zip(q, ctx)):
            full, rest = divmod(t + c, ps)
            seen[table[b, :full].long()] = True
            if rest:
                seen[int(table[b, full]), :rest] = True
        dark = ~seen.cuda()[:, None, :, None]
        nan = 0x7F if case["fp8"] else 0x7FC0
        raw = torch.uint8 if case["fp8"] else torch.int16
        k.view(raw).masked_fill_(dark, nan)
        v.view(raw).masked_fill_(dark, nan)
        # queries after their norm and rotation, sharp enough for peaked rows
        s["q"] = (2.0 * normal(n, hq * D).float()).to(torch.bfloat16)
        s["o"] = torch.zeros((n, hq * D), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "norm_rope":
        s["qkv"] = normal(n, (hq + 2 * hkv) * D)
        s["q_norm"] = (1.0 + 0.1 * normal(D).float()).to(torch.bfloat16)
        s["k_norm"] = (1.0 + 0.1 * normal(D).float()).to(torch.bfloat16)
        s["rope"] = _rope_table()
        s["q"] = torch.zeros((n, hq * D), dtype=torch.bfloat16, device="cuda")
    else:
        s["s_max"] = s["longest"] + 7
        s["ck"], s["cv"] = normal(case["B"], hkv, s["s_max"], D), normal(case["B"], hkv, s["s_max"], D)
    return s


# ------------------------------------------------------------------------- the framework's calls
def _handles(s):
    """The descriptors and the workspace that a program keeps beside its cache."""
    if "handles" not in s:
        import qwen3_decoder_block_b200 as q3
        cfg = q3.make_config(n_q_heads=s["hq"], n_kv_heads=s["hkv"], max_pos=MAX_POS)
        pages = q3.kv_pages(s["k"], s["v"], s["k_scale"], s["v_scale"])
        batch = q3.paged_batch(s["q_start"], s["ctx_len"], s["table"])
        ws = kv = None
        if s["op"] == "attention":
            B = s["ctx_len"].numel()
            size = q3.workspace_size(cfg, q3.OP_ATTENTION_PAGED, B, s["max_q"], s["longest"])
            ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        if "ck" in s:
            kv = q3.kv_layer(s["ck"], s["cv"], s["s_max"])
        s["handles"] = q3, cfg, pages, batch, ws, kv
    return s["handles"]


def _run_own(s):
    q3, cfg, pages, batch, ws, kv = _handles(s)
    if s["op"] == "attention":
        q3.op_attention_paged(cfg, s["q"], s["n_tokens"], s["max_q"], batch, pages, s["o"], ws)
        return {"o": s["o"]}
    if s["op"] == "norm_rope":
        q3.op_qk_norm_rope_paged(cfg, s["qkv"], s["n_tokens"], batch, s["q_norm"], s["k_norm"], pages, s["rope"], s["q"])
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    if s["op"] == "to_pages":
        q3.op_kv_to_pages(cfg, kv, s["n_tokens"], batch, pages)
        return {"k": s["k"], "v": s["v"]}
    q3.op_kv_from_pages(cfg, pages, s["n_tokens"], batch, kv)
    return {"k": s["ck"], "v": s["cv"]}


# ------------------------------------------------------------------------- the plain forms
def _tokens(s):
    """Sequence, position and validity of each row of the token buffers."""
    at = torch.arange(s["n_tokens"], device="cuda", dtype=torch.int32)
    start = s["q_start"]
    b = torch.searchsorted(start[1:].contiguous(), at, right=True).clamp(max=s["ctx_len"].numel() - 1)
    t = at - start[b]
    return b, t, s["ctx_len"][b] + t, at < start[-1]


def _widen(x, scale):
    return x.float() if scale is None else x.float() * scale[:, None, None]


def _narrow(x, scale):
    """fp32 [.., hkv, D] as the pages hold it."""
    if scale is None:
        return x.to(torch.bfloat16)
    return (x * (1.0 / scale)[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _put(s, pool, b, pos, ok, rows):
    """rows [tokens, hkv, D] into the pages, in place."""
    page = s["table"][b, (pos // s["page"]).long().clamp(max=s["table"].shape[1] - 1)].long()
    slot = (pos % s["page"]).long()
    raw, new = _raw(pool), _raw(rows)
    # a row behind the last sequence writes what the first row writes, where it writes it
    page, slot = torch.where(ok, page, page[0]), torch.where(ok, slot, slot[0])
    raw[page, :, slot] = torch.where(ok[:, None, None], new, new[:1])


def _plain_attention(s):
    B, hq, hkv, D, T = s["ctx_len"].numel(), s["hq"], s["hkv"], HEAD_DIM, s["max_q"]
    G, S = hq // hkv, s["table"].shape[1] * s["page"]
    total = (s["ctx_len"] + s["q_start"][1:] - s["q_start"][:-1])[:, None]
    key = torch.arange(S, device="cuda", dtype=torch.int32)
    gather = lambda pool, scale: torch.where(  # noqa: E731
        (key < total)[:, None, :, None],
        _widen(_raw(pool)[s["table"].long()].view(pool.dtype), scale).transpose(1, 2).reshape(B, hkv, S, D), 0.0)
    at = (s["q_start"][:-1, None] + torch.arange(T, device="cuda", dtype=torch.int32)).clamp(max=s["n_tokens"] - 1)
    q = s["q"][at.long()].float().view(B, T, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * T, D)
    p = (q * D ** -0.5) @ gather(s["k"], s["k_scale"]).transpose(2, 3)
    limit = s["ctx_len"][:, None] + torch.arange(T, device="cuda", dtype=torch.int32)
    seen = (key <= limit[:, :, None]).repeat(1, G, 1)[:, None]
    p = p.masked_fill_(~seen, float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    o = (p @ gather(s["v"], s["v_scale"])) / p.sum(-1, keepdim=True)
    o = o.view(B, hkv, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, hq * D)
    b, t, _, ok = _tokens(s)
    rows = o[b, t.long().clamp(max=T - 1)].to(torch.bfloat16)
    s["o"] = torch.where(ok[:, None], rows, s["o"])
    return {"o": s["o"]}


def _plain_norm_rope(s):
    hq, hkv, D = s["hq"], s["hkv"], HEAD_DIM
    b, _, pos, ok = _tokens(s)
    x = s["qkv"].view(-1, hq + 2 * hkv, D)
    qk = x[:, :hq + hkv].float()
    qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS)
    qk = torch.cat((qk[:, :hq] * s["q_norm"].float(), qk[:, hq:] * s["k_norm"].float()), 1)
    cos, sin = s["rope"][pos.long().clamp(max=MAX_POS - 1)].unbind(-1)
    lo, hi = qk.chunk(2, -1)
    cos, sin = cos[:, None], sin[:, None]
    qk = torch.cat((lo * cos - hi * sin, lo * sin + hi * cos), -1)
    q = qk[:, :hq].reshape(-1, hq * D).to(torch.bfloat16)
    s["q"] = torch.where(ok[:, None], q, s["q"])
    _put(s, s["k"], b, pos, ok, _narrow(qk[:, hq:], s["k_scale"]))
    _put(s, s["v"], b, pos, ok, _narrow(x[:, hq + hkv:].float(), s["v_scale"]))
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _plain_to_pages(s):
    b, _, pos, ok = _tokens(s)
    at = pos.long().clamp(max=s["s_max"] - 1)
    _put(s, s["k"], b, pos, ok, _narrow(s["ck"][b, :, at].float(), s["k_scale"]))
    _put(s, s["v"], b, pos, ok, _narrow(s["cv"][b, :, at].float(), s["v_scale"]))
    return {"k": s["k"], "v": s["v"]}


def _plain_from_pages(s):
    S = min(s["table"].shape[1] * s["page"], s["s_max"])
    key = torch.arange(S, device="cuda", dtype=torch.int32)
    first = s["ctx_len"][:, None]
    last = first + (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    ok = ((key >= first) & (key < last))[:, None, :, None]
    back = lambda pool, scale: _widen(_raw(pool)[s["table"].long()].view(pool.dtype), scale).transpose(1, 2).flatten(2, 3)[:, :, :S]  # noqa: E731
    s["ck"][:, :, :S] = torch.where(ok, back(s["k"], s["k_scale"]).to(torch.bfloat16), s["ck"][:, :, :S])
    s["cv"][:, :, :S] = torch.where(ok, back(s["v"], s["v_scale"]).to(torch.bfloat16), s["cv"][:, :, :S])
    return {"k": s["ck"], "v": s["cv"]}


def run(state):
    if own:
        return _run_own(state)
    plain = {"attention": _plain_attention, "norm_rope": _plain_norm_rope, "to_pages": _plain_to_pages,
             "from_pages": _plain_from_pages}
    return plain[state["op"]](state)


# ------------------------------------------------------------------------- the definitions in 64 bits
def _cells(table, page, first, last):
    """Page and slot of the positions first..last-1 of one sequence."""
    p = torch.arange(first, last, device="cuda")
    return table[p // page].long(), p % page


def exact(case, seed):
    s = prepare(case, seed)
    q, ctx = _lengths(case)
    hq, hkv, D, page = case["hq"], case["hkv"], HEAD_DIM, case["page"]
    unit = torch.ones(hkv, dtype=torch.float64, device="cuda")
    ks, vs = (s["k_scale"].double(), s["v_scale"].double()) if case["fp8"] else (unit, unit)

    def cache(pool, scale, b, first, last):
        pg, slot = _cells(s["table"][b], page, first, last)
        raw = pool.view(torch.uint8) if case["fp8"] else pool
        return raw[pg, :, slot].view(pool.dtype).double() * scale[:, None]

    def held(x, scale):
        if not case["fp8"]:
            return x.to(torch.bfloat16)
        return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)

    def store(pool, b, first, last, rows):
        pg, slot = _cells(s["table"][b], page, first, last)
        pool[pg, :, slot] = rows.double()

    row = 0
    if case["op"] == "attention":
        out = s["o"].double()
        for b, (t, c) in enumerate(zip(q, ctx)):
            K, V = cache(s["k"], ks, b, 0, c + t), cache(s["v"], vs, b, 0, c + t)
            Q = s["q"][row:row + t].double().view(t, hkv, hq // hkv, D)
            mask = torch.arange(c + t, device="cuda")[None] > c + torch.arange(t, device="cuda")[:, None]
            for h in range(hkv):
                w = torch.einsum("tgd,sd->gts", Q[:, h], K[:, h]) / D ** 0.5
                w = torch.softmax(w.masked_fill(mask, float("-inf")), -1)
                out[row:row + t].view(t, hkv, hq // hkv, D)[:, h] = torch.einsum("gts,sd->tgd", w, V[:, h])
            row += t
        return {"o": out}
    if case["op"] == "from_pages":
        outs = [s["ck"].double(), s["cv"].double()]
        for b, (t, c) in enumerate(zip(q, ctx)):
            for dst, pool, scale in ((outs[0], s["k"], ks), (outs[1], s["v"], vs)):
                dst[b, :, c:c + t] = cache(pool, scale, b, c, c + t).transpose(0, 1)
        return {"k": outs[0], "v": outs[1]}
    k, v = s["k"].double(), s["v"].double()
    if case["op"] == "to_pages":
        for b, (t, c) in enumerate(zip(q, ctx)):
            store(k, b, c, c + t, held(s["ck"][b, :, c:c + t].transpose(0, 1).double(), ks))
            store(v, b, c, c + t, held(s["cv"][b, :, c:c + t].transpose(0, 1).double(), vs))
        return {"k": k, "v": v}
    qo = s["q"].double()
    f = torch.tensor([THETA ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")
    for b, (t, c) in enumerate(zip(q, ctx)):
        x = s["qkv"][row:row + t].double().view(t, hq + 2 * hkv, D)
        z = torch.polar(torch.ones(t, D // 2, dtype=torch.float64, device="cuda"),
                        torch.arange(c, c + t, dtype=torch.float64, device="cuda")[:, None] * f)[:, None]

        def turned(y, w):
            y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
            y = torch.complex(y[..., :D // 2].contiguous(), y[..., D // 2:].contiguous()) * z
            return torch.cat((y.real, y.imag), -1)

        qo[row:row + t] = turned(x[:, :hq], s["q_norm"]).reshape(t, hq * D)
        store(k, b, c, c + t, held(turned(x[:, hq:hq + hkv], s["k_norm"]), ks))
        store(v, b, c, c + t, held(x[:, hq + hkv:], vs))
        row += t
    return {"q": qo, "k": k, "v": v}
