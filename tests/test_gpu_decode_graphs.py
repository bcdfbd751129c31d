"""The paged cache's steps replayed from CUDA graphs: rows stored and attended by the captured calls of all layers, against
the definition in 64 bits and against the same cache without graphs, long after the captured step is gone."""
import gc

import pytest
import torch

from nvfp4_block_scaled_11_b200 import kvcache as kc
from tests import kvref
from tests.test_gpu_decode_path import _sides

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
L, H, D = 2, 2, 64


def _pair(gen, prompts, **kw):
    """Two caches with the same sequences."""
    cs = [kc.NVFP4PagedKVCache(L, 4, H, D, 60, 16, **kw) for _ in range(2)]
    for T in prompts:
        ks, vs = ([torch.randn(H, T, D, generator=gen).to(BF).cuda() for _ in range(L)] for _ in range(2))
        for c in cs:
            c.prefill(c.alloc(), ks, vs)
    return cs


class Captured:
    """store and attend of every layer for the sequences `slots` and n tokens, captured around a step that is then dropped."""

    def __init__(self, c, slots, n, rows):
        self.k, self.v, self.q = (torch.zeros(L, len(slots), h, n, D, dtype=BF, device="cuda") for h in (H, H, 3 * H))
        self.load(rows)
        st = c.step(slots, n)
        torch.cuda.synchronize()
        self.g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.g):
            self.outs = []
            for layer in range(L):
                c.store(st, layer, self.k[layer], self.v[layer])
                self.outs.append(c.attend(st, layer, self.q[layer], want_lse=True))

    def load(self, rows):
        for t, x in zip((self.k, self.v, self.q), rows):
            t.copy_(x)


def _rows(gen, B, n):
    return [torch.randn(L, B, h, n, D, generator=gen).to(BF).cuda() for h in (H, H, 3 * H)]


@pytest.mark.parametrize("recent", [16, 5])
def test_replayed_steps_store_and_attend_their_own_rows(recent):
    gen = torch.Generator().manual_seed(recent)
    a, b = _pair(gen, (90, 16 + recent, 50), recent=recent)
    warm = _pair(gen, (60,))[0]                                       # kernels loaded outside the captures
    for n in (1, 3):
        st, (k, v, q) = warm.step([0], n), _rows(gen, 1, n)
        warm.store(st, 0, k[0], v[0])
        warm.attend(st, 0, q[0])

    def eager(slots, n, rows):
        st = b.step(slots, n)
        for layer in range(L):
            b.store(st, layer, rows[0][layer], rows[1][layer])

    graphs = []
    for slots, n in (([2, 0], 1), ([0, 1, 2], 3)):
        rows = _rows(gen, len(slots), n)
        graphs.append((slots, n, Captured(a, slots, n, rows)))        # a capture runs nothing: its step is replayed first
        graphs[-1][2].g.replay()
        eager(slots, n, rows)
    gc.collect()
    junk = [torch.full((4096,), 0x7F7F7F7F7F7F, dtype=torch.int64, device="cuda") for _ in range(64)]   # where a step's were
    for i in range(40):
        slots, n, cap = graphs[i % 2]
        rows = _rows(gen, len(slots), n)
        a.step(slots, n)
        cap.load(rows)
        cap.g.replay()
        eager(slots, n, rows)
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(a, t), getattr(b, t)) for t in ("lens", "table", "window", "codes", "scales"))
        if i % 5 < 2:
            for layer in range(L):
                kvref.check(*cap.outs[layer], kvref.attention(rows[2][layer].cpu(), *_sides(b, layer), b.lens.tolist(), b.table.cpu(),
                                                              slots))
    assert len(junk) == 64


def test_books_are_refused_in_a_real_capture():
    gen = torch.Generator().manual_seed(1)
    a, b = _pair(gen, (60,))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(g):
        x += 1                                                        # (a graph is not left empty)
        for call in (lambda: a.step([0]), lambda: a.fork(0), lambda: a.free(0), lambda: a.compact()):
            with pytest.raises(RuntimeError, match="capture"):
                call()
    g.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [1.0] * 4 and torch.equal(a.lens, b.lens) and a.length(0) == 60
