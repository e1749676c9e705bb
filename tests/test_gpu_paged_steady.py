"""The paged attention in its steady state: CTAs that finish one pair of Q tiles after another, and
large mixed batches replayed with other lengths, against float64."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from helpers import assert_device_ok  # noqa: E402
from test_gpu_paged import Case  # noqa: E402
from test_paged_pairs import STEADY  # noqa: E402


@pytest.fixture(scope="module")
def q3():
    import qwen3_decoder_block_b200 as m
    return m


class GpuCase(Case):
    """The same reference and tolerances, computed on the GPU (many tokens)."""

    def reference(self):
        G, out = self.hq // self.hkv, []
        for b, (t, c) in enumerate(zip(self.qlens, self.ctx)):
            if not t:
                continue
            K, V = (torch.from_numpy(self.rows(x, s, b, c + t)).cuda() for x, s in ((self.k, self.ks64), (self.v, self.vs64)))
            r0 = self.q_start[b]
            Q = self.q[r0:r0 + t, :self.hq * 128].double().view(t, self.hkv, G, 128)
            s = torch.einsum("thgd,shd->thgs", Q, K) / 128 ** 0.5
            key, at = torch.arange(c + t, device="cuda"), torch.arange(t, device="cuda")
            s.masked_fill_((key[None] > c + at[:, None])[:, None, None], float("-inf"))
            w = torch.softmax(s, -1)
            out.append([torch.einsum("thgs,shd->thgd", w, v).reshape(t, -1).cpu().numpy() for v in (V, V.abs())])
        ref, mag = (np.concatenate(x) for x in zip(*out))
        half = 2.0 ** -11 if self.otype == torch.float16 else 2.0 ** -8
        return ref, half * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag + 1e-7


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens,ctx,page,hq,hkv", STEADY)
def test_attention_pair_after_pair(q3, qlens, ctx, page, hq, hkv, fp8):
    """Finished rows are staged over the Q tile that the next item's q goes to."""
    c = GpuCase(q3, qlens, ctx, page, hq=hq, hkv=hkv, fp8=fp8, pad=3, seed=sum(qlens))
    c.darken()
    o = c.attend()
    assert_device_ok()
    c.check(o)
    for _ in range(20):
        assert torch.equal(o, c.attend())
    assert_device_ok()


def other_lengths(c, ctx, qlens):
    """The same batch object with other lengths: its lists, its queries."""
    c.ctx, c.qlens = list(ctx), list(qlens)
    c.q_start = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    c.t_ctx.copy_(torch.tensor(c.ctx, dtype=torch.int32))
    c.t_start.copy_(torch.from_numpy(c.q_start))


@pytest.mark.parametrize("fp8", [False, True])
def test_large_mixed_batch_replays_with_other_lengths(q3, fp8):
    """Both forms of the kernel in one captured call: every replay follows the lengths of its own step
    (decode sequences become chunks and the other way round), and none the work list of the last one."""
    first_q = [1, 60, 1, 1, 130, 1, 0, 1, 1, 300, 1, 1, 2, 1, 1, 1, 1, 1, 33, 1]
    c = GpuCase(q3, first_q, [640] * 20, 32, fp8=fp8, seed=4, pad=40)  # pages for what the replays bring
    n = q3.workspace_size(c.cfg, q3.OP_ATTENTION_PAGED, 20, 300, 1)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    o = torch.full((c.n, 16 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    c.attend(max_q=300, ws=ws, out=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(max_q=300, ws=ws, out=o)
    rng = np.random.default_rng(9)
    c.q.copy_(torch.randn(c.q.shape, device="cuda").bfloat16())
    for step in range(6):
        order = rng.permutation(20)
        other_lengths(c, rng.integers(0, 341, 20).tolist(), [first_q[i] for i in order])
        o.fill_(7.0)
        graph.replay()
        assert_device_ok()
        c.check(o)
