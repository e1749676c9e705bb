"""CPU checks of the paged-cache calls: bad arguments are refused on the host, with a message
that names them, before anything could be launched."""
import ctypes

import pytest

FAKE = 1 << 44


@pytest.fixture(scope="module")
def q3():
    import __graft_entry__
    __graft_entry__.build()
    import qwen3_decoder_block_b200 as m
    return m


def good(q3, fp8=0, **kw):
    pages = q3.KVPages(FAKE, FAKE + (1 << 36), FAKE, FAKE, 64, 16, fp8)
    batch = q3.PagedBatch(FAKE, FAKE, FAKE, 4, 8)
    a = dict(q=FAKE, ldq=2048, qkv=FAKE, ldqkv=4096, n=64, max_q=16, o=FAKE, ldo=2048, ws=FAKE, ws_bytes=1 << 30,
             q_norm=FAKE, k_norm=FAKE, rope=FAKE, q_out=FAKE + (1 << 30), kv=q3.KVLayer(FAKE, FAKE + (1 << 36), 4096))
    for k, v in kw.items():
        if k in dict(q3.KVPages._fields_) and k not in a:
            setattr(pages, k, v)
        elif k in dict(q3.PagedBatch._fields_):
            setattr(batch, k, v)
        else:
            a[k] = v
    return pages, batch, a


def calls(q3, fp8=0, **kw):
    """Status and message of the four calls with the given arguments changed."""
    c = ctypes.byref(q3.config_qwen3_0_6b())
    p, b, a = good(q3, fp8, **kw)
    p, b, kv = ctypes.byref(p), ctypes.byref(b), ctypes.byref(a["kv"])
    L = q3.lib
    out = {}
    for name, f in (
            ("norm", lambda: L.qwen3_op_qk_norm_rope_paged(c, a["qkv"], a["ldqkv"], a["n"], b, a["q_norm"], a["k_norm"],
                                                           p, a["rope"], a["q_out"], a["ldq"], None)),
            ("attn", lambda: L.qwen3_op_attention_paged(c, a["q"], a["ldq"], a["n"], a["max_q"], b, p, a["o"], a["ldo"],
                                                        a["ws"], a["ws_bytes"], None)),
            ("to", lambda: L.qwen3_op_kv_to_pages(c, kv, a["n"], b, p, None)),
            ("from", lambda: L.qwen3_op_kv_from_pages(c, p, a["n"], b, kv, None))):
        out[name] = (f(), L.qwen3_last_error().decode())
    return out


ALL = ("norm", "attn", "to", "from")


@pytest.mark.parametrize("change,status,word,who", [
    (dict(k=None), "EINVAL", "pages->k", ALL), (dict(v=None), "EINVAL", "pages->v", ALL),
    (dict(k=FAKE + 8), "EALIGN", "16-byte", ALL), (dict(n_pages=0), "EINVAL", "n_pages", ALL),
    (dict(page_size=8), "ESHAPE", "page_size", ALL), (dict(page_size=48), "ESHAPE", "page_size", ALL),
    (dict(page_size=512), "ESHAPE", "page_size", ALL), (dict(page_size=0), "ESHAPE", "page_size", ALL),
    (dict(n_pages=1 << 25), "ESHAPE", "2^31", ALL), (dict(max_pages=1 << 28), "ESHAPE", "2^31", ALL),
    (dict(q_start=None), "EINVAL", "q_start", ALL), (dict(ctx_len=None), "EINVAL", "ctx_len", ALL),
    (dict(page_table=None), "EINVAL", "page_table", ALL), (dict(page_table=FAKE + 2), "EALIGN", "4-byte", ALL),
    (dict(B=0), "EINVAL", "B", ALL), (dict(max_pages=0), "EINVAL", "max_pages", ALL),
    (dict(n=0), "EINVAL", "n_tokens", ALL), (dict(n=-3), "EINVAL", "n_tokens", ALL),
    (dict(qkv=None), "EINVAL", "NULL", ("norm",)), (dict(rope=None), "EINVAL", "NULL", ("norm",)),
    (dict(q_out=FAKE + 2), "EALIGN", "misaligned", ("norm",)), (dict(ldqkv=4088), "EALIGN", "ldqkv", ("norm",)),
    (dict(ldq=2052), "EALIGN", "ldq", ("norm", "attn")), (dict(ldq=2040), "EALIGN", "ldq", ("norm", "attn")),
    (dict(q_out=FAKE), "EINVAL", "in place", ("norm",)),
    (dict(q=None), "EINVAL", "NULL", ("attn",)), (dict(o=FAKE + 4), "EALIGN", "misaligned", ("attn",)),
    (dict(ldo=-2048), "EALIGN", "ldo", ("attn",)), (dict(max_q=0), "EINVAL", "max_q", ("attn",)),
    (dict(ws=None), "EINVAL", "NULL", ("attn",)), (dict(ws_bytes=16), "EWORKSPACE", "workspace", ("attn",)),
])
def test_bad_arguments_are_refused(q3, change, status, word, who):
    for name, (st, msg) in calls(q3, **change).items():
        if name in who:
            assert st == getattr(q3, status) and word in msg, (name, st, msg)


def test_e4m3_pages_need_scales(q3):
    for change in (dict(k_scale=None), dict(v_scale=None)):
        for st, msg in calls(q3, fp8=1, **change).values():
            assert st == q3.EINVAL and "scale" in msg
    for st, msg in calls(q3, fp8=1, k_scale=FAKE + 2).values():
        assert st == q3.EALIGN and "scale" in msg
    for st, msg in calls(q3, fp8=2).values():
        assert st == q3.EINVAL and "fp8" in msg


def test_contiguous_side_checked(q3):
    for kv, status in ((q3.KVLayer(None, FAKE, 16), q3.EINVAL), (q3.KVLayer(FAKE + 8, FAKE, 16), q3.EALIGN),
                       (q3.KVLayer(FAKE, FAKE, 0), q3.EINVAL)):
        out = calls(q3, kv=kv)
        assert out["to"][0] == status and out["from"][0] == status


def test_null_descriptors_and_bad_config(q3):
    c = q3.config_qwen3_0_6b()
    p, b, a = good(q3)
    st = q3.lib.qwen3_op_attention_paged(ctypes.byref(c), FAKE, 2048, 64, 1, None, ctypes.byref(p), FAKE, 2048, FAKE,
                                         1 << 30, None)
    assert st == q3.EINVAL
    st = q3.lib.qwen3_op_kv_to_pages(ctypes.byref(c), None, 64, ctypes.byref(b), ctypes.byref(p), None)
    assert st == q3.EINVAL
    c.head_dim = 64
    st = q3.lib.qwen3_op_kv_to_pages(ctypes.byref(c), ctypes.byref(a["kv"]), 64, ctypes.byref(b), ctypes.byref(p), None)
    assert st == q3.ESHAPE


def test_workspace_size(q3):
    c = q3.config_qwen3_0_6b()
    assert q3.workspace_size(c, q3.OP_ATTENTION_PAGED, 64, 1, 4096) > 0
    assert q3.workspace_size(c, q3.OP_ATTENTION_PAGED, 64, 512, 4096) > 0
    assert q3.workspace_size(c, q3.OP_ATTENTION_PAGED, 0, 1, 4096) == 0
    assert q3.workspace_size(c, q3.OP_ATTENTION_PAGED, 4, 0, 4096) == 0


def test_binding_refuses_wrong_tensors(q3):
    torch = pytest.importorskip("torch")
    k = torch.zeros(4, 8, 16, 128, dtype=torch.bfloat16)
    s = torch.ones(8)
    assert q3.kv_pages(k, k).page_size == 16 and q3.kv_pages(k, k).fp8 == 0
    k8 = k.to(torch.float8_e4m3fn)
    assert q3.kv_pages(k8, k8, s, s).fp8 == 1
    for bad in ((k, k[:2]), (k.half(), k.half()), (k[..., :64], k[..., :64]), (k8, k8), (k8, k8, s, s[:4]),
                (k8, k8, s.double(), s), (k.transpose(0, 1), k.transpose(0, 1))):
        with pytest.raises(ValueError):
            q3.kv_pages(*bad)
    i = torch.zeros(5, dtype=torch.int32)
    t = torch.zeros(4, 8, dtype=torch.int32)
    assert q3.paged_batch(i, i[:4], t).max_pages == 8
    for bad in ((i, i, t), (i.long(), i[:4], t), (i, i[:4], t.t()), (i, i[:4], t[:2])):
        with pytest.raises(ValueError):
            q3.paged_batch(*bad)
