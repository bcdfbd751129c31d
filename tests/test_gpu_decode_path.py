"""The decode operators together, as a program uses them: rotary positions, prefill, forks, steps with draft tokens,
attention, compaction -- against plain attention in 64 bits over the cache's own contents, and (loosely) over the
unquantized tokens."""
import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv
from nvfp4_block_scaled_11_b200 import kvcache as kc
from tests import kvref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class _Copy(kvref.Side):
    """One side of a cache's device buffers, on the CPU."""

    def __init__(self, sink, window, codes, scales, gscale, rotate):
        self.H, self.D, self.rotate, self.tile = codes.shape[1], 2 * codes.shape[3], rotate, False
        self.sink, self.window, self.codes = sink.cpu(), window.cpu(), codes.cpu()
        self.scales, self.gscale = scales.cpu(), gscale.cpu()


def _sides(c, layer):
    return [_Copy(c.sink[layer, i], c.window[layer, i], c.codes[layer, i], c.scales[layer, i], c.gscale[layer, i], c.rotate)
            for i in (0, 1)]


@pytest.mark.parametrize("D,page,rotate", [(128, 32, True), (64, 48, True), (128, 16, False)])
def test_serving_loop(D, page, rotate):
    gen = torch.Generator(device="cuda").manual_seed(D + page)
    L, H, G = 2, 2, 3
    c = kc.NVFP4PagedKVCache(L, 6, H, D, 40, page, rotate=rotate)
    freqs, m = nv.rope_frequencies(D // 2, scaling=dict(type="yarn", factor=4, original=64))
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF)  # noqa: E731
    plain = {}                                        # slot -> per layer [K, V] of all tokens so far, BF16

    def qkv(B, n, pos):
        """A projection's output [B, n, ...], q and k turned to their positions."""
        x = r(B, n, (H * G + 2 * H) * D).unflatten(-1, (-1, D)).transpose(1, 2)
        q, k = nv.rope([x[:, :H * G], x[:, H * G:H * G + H]], pos, freqs, interleaved=True, mscale=m)
        return q, k, x[:, H * G + H:]

    def start(T):
        s = c.alloc()
        ks, vs = zip(*[qkv(1, T, torch.arange(T, device="cuda"))[1:] for _ in range(L)])
        c.prefill(s, ks, vs)
        plain[s] = [[ks[i][0], vs[i][0]] for i in range(L)]
        return s

    def step(slots, n):
        st = c.step(slots, n)
        pos = torch.tensor([[c.length(s) - n + i for i in range(n)] for s in slots], device="cuda")
        for layer in range(L):
            q, k, v = qkv(len(slots), n, pos)
            c.store(st, layer, k, v)
            out, lse = c.attend(st, layer, q, want_lse=True)
            for i, s in enumerate(slots):
                kv = plain[s][layer]
                plain[s][layer] = [torch.cat([kv[0], k[i]], 1), torch.cat([kv[1], v[i]], 1)]
            torch.cuda.synchronize()
            lens = c.lens.tolist()
            kvref.check(out, lse, kvref.attention(q.cpu(), *_sides(c, layer), lens, c.table.cpu(), slots))
            for i, s in enumerate(slots):              # near the attention over the tokens as they were
                kf, vf = (t.double().repeat_interleave(G, 0) for t in plain[s][layer])
                T = kf.shape[1]
                x = q[i].double() @ kf.transpose(1, 2) * D ** -0.5
                x.masked_fill_(torch.arange(T, device="cuda") > T - n + torch.arange(n, device="cuda")[:, None], -torch.inf)
                want = x.softmax(-1) @ vf
                assert (out[i].double() - want).norm() < 0.35 * want.norm()   # FP4 keys and values

    a, b = start(32 + page + 5), start(32)
    step([a, b], 1)
    (f,) = c.fork(a)
    plain[f] = [list(kv) for kv in plain[a]]
    for _ in range(6):
        step([b, f, a], 4)
    c.free(a)
    d = start(100)
    assert c.compact() == c.n_pages - c.pages_free
    for _ in range(5):
        step([f, d], 7)
        step([b], 1)
    # the rows of a sequence outside the step are left as they were
    before = [t.clone() for t in (c.window[:, :, d], c.lens[d], c.table[d])]
    step([b, f], 16)
    assert all(torch.equal(x, y) for x, y in zip(before, (c.window[:, :, d], c.lens[d], c.table[d])))


def test_paged_and_contiguous_caches_agree():
    """The same tokens through NVFP4KVCache + attend and through the paged cache: the same bytes, so the same output."""
    gen = torch.Generator().manual_seed(1)
    H, D, T = 2, 128, 203
    k, v = (torch.randn(1, H, T, D, generator=gen).to(BF).cuda() for _ in range(2))
    ck, cv = (kc.NVFP4KVCache(1, H, D, capacity=301) for _ in range(2))
    ck.prefill(k), cv.prefill(v)
    p = kc.NVFP4PagedKVCache(1, 2, H, D, 20, 32)
    s = p.alloc()
    p.prefill(s, [k], [v])
    for i in range(40):
        kn, vn, q = (torch.randn(1, h, 1, D, generator=gen).to(BF).cuda() for h in (H, H, 8))
        ck.append(kn), cv.append(vn)
        st = p.step([s])
        p.store(st, 0, kn, vn)
        want, wl = kc.attend(q, ck, cv, want_lse=True)
        got, gl = p.attend(st, 0, q, want_lse=True)
        assert (ck.n_sink, ck.n_mid, ck.head, ck.n_window) == tuple(p.lens[s].tolist())
        # one range here, perhaps another count there: FP32 sums in another order
        assert (got.double() - want.double()).abs().max() <= 2.0 ** -7 * want.abs().max() and (gl - wl).abs().max() < 1e-5
    tiles = kc.NVFP4KVCache(1, H, D, capacity=301, tile_layout=True)
    tiles.prefill(k)
    rows = kc.NVFP4KVCache(1, H, D, capacity=301)
    rows.prefill(k)
    q = torch.randn(1, 4, 1, D, generator=gen).to(BF).cuda()
    assert torch.equal(kc.attend(q, tiles, tiles), kc.attend(q, rows, rows))


def test_steps_replayed_from_a_graph():
    """The layers of a step captured once: later steps only change lengths, tables and inputs on the device."""
    gen = torch.Generator().manual_seed(2)
    H, D = 2, 64
    c = kc.NVFP4PagedKVCache(1, 2, H, D, 20, 16)
    for T in (90, 50):
        s = c.alloc()
        c.prefill(s, [torch.randn(H, T, D, generator=gen).to(BF).cuda()], [torch.randn(H, T, D, generator=gen).to(BF).cuda()])
    st = c.step([0, 1])
    k, v, q = (torch.randn(2, h, 1, D, generator=gen).to(BF).cuda() for h in (H, H, 4))
    ids = torch.arange(2, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    stores = c.stores(0)
    c.store(st, 0, k, v)
    nv.kv_attention(q, *stores, c.lens, c.table, ids, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.kv_attention(q, *stores, c.lens, c.table, ids, out=out)
    for _ in range(40):
        st = c.step([0, 1])
        c.store(st, 0, k, v)
        q.copy_(torch.randn(2, 4, 1, D, generator=gen))
        g.replay()
        assert torch.equal(out, nv.kv_attention(q, *stores, c.lens, c.table, ids))


def test_prompt_is_quantized_as_the_contiguous_cache_does():
    gen = torch.Generator().manual_seed(3)
    H, D, T = 3, 64, 32 + 130
    k = torch.randn(1, H, T, D, generator=gen).to(BF).cuda()
    ref = kc.NVFP4KVCache(1, H, D, capacity=130)
    ref.prefill(k)
    c = kc.NVFP4PagedKVCache(1, 1, H, D, 4, 48)
    c.prefill(c.alloc(), [k], [2 * k])
    rows = lambda t: t[0, 0, :3].transpose(0, 1).flatten(1, 2)[:, :130]  # noqa: E731
    assert torch.equal(rows(c.codes), ref.codes[0]) and torch.equal(rows(c.scales), ref.scales[0])
    assert c.gscale[0, 0, 0] == ref.gscale[0] and c.gscale[0, 1, 0] == 2 * ref.gscale[0]
    assert torch.equal(c.sink[0, 0, 0], ref.sink[0]) and torch.equal(c.window[0, 0, 0], ref.window[0])
