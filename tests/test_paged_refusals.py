"""CPU checks of the paged-cache calls' limits and of what the binding refuses."""
import pytest

from test_paged_abi import ALL, calls, q3  # noqa: F401


@pytest.mark.parametrize("B", [1 << 26, (1 << 27) + 5, 2 ** 31 - 20, 2 ** 31 - 1])
def test_too_many_sequences_are_refused(q3, B):  # noqa: F811
    """Beyond 2^30 (sequence, query head) rows 32-bit coordinates end; near 2^31 sequences a scan over
    them would not."""
    for name, (st, msg) in calls(q3, B=B, ws_bytes=1 << 62).items():
        assert name in ALL and st == q3.ESHAPE and "2^30" in msg, (name, st, msg)


def test_many_sequences_pass_the_limit(q3):  # noqa: F811
    """(the next check is the workspace's, or the device's)"""
    for st, msg in calls(q3, B=(1 << 26) - 1, ws_bytes=16).values():
        assert "2^30" not in msg and st != q3.ESHAPE


@pytest.mark.parametrize("heads", [4, 16])
def test_pages_of_another_head_count_are_refused(q3, heads):  # noqa: F811
    """A pool made for other KV heads than the configuration's would be read and written past its
    end (or in the wrong places). Refused before the stream or the library are looked at."""
    torch = pytest.importorskip("torch")
    cfg = q3.config_qwen3_0_6b()
    assert cfg.n_kv_heads == 8
    t = torch.zeros(4, heads, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    batch = q3.paged_batch(i, i[:4], torch.zeros(4, 8, dtype=torch.int32))
    x, kv = torch.zeros(64), q3.kv_layer(t, t, 16)
    for dtype in (torch.bfloat16, torch.float8_e4m3fn):
        s = torch.ones(heads)
        pages = q3.kv_pages(t.to(dtype), t.to(dtype), s, s)
        for call in (lambda: q3.op_qk_norm_rope_paged(cfg, x, 4, batch, x, x, pages, x, x),
                     lambda: q3.op_attention_paged(cfg, x, 4, 1, batch, pages, x, x),
                     lambda: q3.op_kv_to_pages(cfg, kv, 4, batch, pages),
                     lambda: q3.op_kv_from_pages(cfg, pages, 4, batch, kv)):
            with pytest.raises(ValueError, match=f"{heads} KV heads"):
                call()


def test_pages_of_the_right_head_count_reach_the_library(q3):  # noqa: F811
    torch = pytest.importorskip("torch")
    cfg = q3.config_qwen3_0_6b()
    t = torch.zeros(4, 8, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    batch = q3.paged_batch(i, i[:4], torch.zeros(4, 8, dtype=torch.int32))
    for pages in (q3.kv_pages(t, t), q3.KVPages(t.data_ptr(), t.data_ptr(), None, None, 4, 16, 0)):
        with pytest.raises(q3.Qwen3Error, match="max_q"):  # the library's own refusal
            q3.op_attention_paged(cfg, t, 4, 0, batch, pages, t, t, stream=0)
