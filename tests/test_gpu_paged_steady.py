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
