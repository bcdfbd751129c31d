"""Attention over the NVFP4 K/V cache against the definition in 64 bits: head layouts, lengths from none to
many ranges, ring positions, pages that end inside a tile, scale layouts, masks, poisoned and hidden tokens."""
import math

import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv
from tests import kvref

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def _q(gen, B, Hq, Tq, D, dt, amp=2.0):
    return (amp * torch.randn(B, Hq, Tq, D, generator=gen)).to(dt)


def _run(q, k, v, lens, table=None, slots=None, host=False, **kw):
    dev = lambda t, dt=torch.int32: None if t is None else torch.as_tensor(t, dtype=dt).cuda()  # noqa: E731
    out, lse = nv.kv_attention(q.cuda(), k.store(nv), v.store(nv), tuple(lens[0]) if host else dev(lens), dev(table), dev(slots),
                               want_lse=True, **kw)
    torch.cuda.synchronize()
    ref = kvref.attention(q, k, v, lens, table if table is None else torch.as_tensor(table), slots, kw.get("causal", True),
                          kw.get("scale"))
    kvref.check(out, lse, ref)
    return out, lse, ref


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 8, 11])
@pytest.mark.parametrize("dt", [BF, F16])
def test_heads_and_types(D, G, dt):
    gen = torch.Generator().manual_seed(D + G)
    k = kvref.Side(gen, 2, 2, D, 16, 32, 2, 333)
    v = kvref.Side(gen, 2, 2, D, 16, 32, 2, 333)
    _run(_q(gen, 2, 2 * G, 1, D, dt), k, v, [(16, 301, 16, 29), (16, 333, 0, 16)])


@pytest.mark.parametrize("lens", [(0, 0, 0, 0), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 31, 1), (7, 0, 0, 0), (16, 15, 5, 16),
                                  (16, 16, 17, 31), (16, 31, 31, 32), (3, 32, 0, 17), (16, 33, 30, 5), (0, 47, 0, 0),
                                  (16, 255, 16, 20), (16, 256, 0, 32), (16, 257, 1, 1), (16, 600, 16, 31)])
@pytest.mark.parametrize("D", [64, 128])
def test_lengths(lens, D):
    """No token, one token of each part, tiles and ranges that end anywhere, rings that wrap."""
    gen = torch.Generator().manual_seed(sum(lens) + D)
    k = kvref.Side(gen, 1, 1, D, 16, 32, 1, 601)
    v = kvref.Side(gen, 1, 1, D, 16, 32, 1, 601)
    out, lse, _ = _run(_q(gen, 1, 4, 1, D, BF), k, v, [lens], host=True)
    if sum(lens) - lens[2] == 0:
        assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("D,G,page", [(128, 4, 16), (128, 8, 64), (64, 3, 48), (256, 16, 32), (256, 2, 128), (64, 1, 16)])
@pytest.mark.parametrize("splits", [1, 3, None])
def test_pages(D, G, page, splits):
    """Ragged sequences over a shuffled pool, with per-slot tensor scales; tables with unused entries of -1."""
    gen = torch.Generator().manual_seed(page + D)
    mids = [700, 0, 33, 257, page]
    need = [-(-m // page) for m in mids]
    pages, cols = sum(need) + 5, max(need) + 1
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((5, cols), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    k = kvref.Side(gen, 5, 2, D, 16, 32, pages, page, per_slot=True)
    v = kvref.Side(gen, 5, 2, D, 16, 32, pages, page, per_slot=True)
    lens = [(16, 700, 16, 20), (9, 0, 0, 0), (16, 33, 16, 17), (16, 257, 0, 32), (16, page, 0, 16)]
    _run(_q(gen, 5, 2 * G, 1, D, BF), k, v, lens, table, splits=splits)


@pytest.mark.parametrize("rk,rv", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rotation_of_each_side(rk, rv, D):
    gen = torch.Generator().manual_seed(5 + D)
    k = kvref.Side(gen, 1, 2, D, 16, 32, 1, 200, rotate=rk)
    v = kvref.Side(gen, 1, 2, D, 16, 32, 1, 200, rotate=rv)
    _run(_q(gen, 1, 6, 1, D, F16), k, v, [(16, 190, 0, 20)], host=True)


@pytest.mark.parametrize("D,cap", [(64, 129), (128, 300), (128, 1), (256, 127)])
def test_tile_layout_of_the_scales(D, cap):
    gen = torch.Generator().manual_seed(cap)
    k = kvref.Side(gen, 2, 3, D, 16, 32, 2, cap, tile=True)
    v = kvref.Side(gen, 2, 3, D, 16, 32, 2, cap, tile=True)
    _run(_q(gen, 2, 3, 1, D, BF), k, v, [(16, cap, 0, 16), (16, cap - 1, 16, 32)])


@pytest.mark.parametrize("D,cap", [(64, 77), (128, 333), (64, 2)])
def test_odd_capacities(D, cap):
    """Rows of scale bytes whose heads begin at any multiple of 4 bytes."""
    gen = torch.Generator().manual_seed(cap)
    k = kvref.Side(gen, 2, 3, D, 0, 32, 2, cap)
    v = kvref.Side(gen, 2, 3, D, 0, 32, 2, cap)
    _run(_q(gen, 2, 6, 1, D, BF), k, v, [(0, cap, 0, 16), (0, cap - 1, 16, 0)])


@pytest.mark.parametrize("Tq", [2, 5, 8, 33])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_several_query_tokens(Tq, G, causal, D):
    """Draft tokens see one another causally, in the window, in the middle and across both; the sequence shorter than
    the draft leaves its first rows empty."""
    gen = torch.Generator().manual_seed(Tq + G)
    k = kvref.Side(gen, 4, 1, D, 16, 32, 4, 90)
    v = kvref.Side(gen, 4, 1, D, 16, 32, 4, 90)
    lens = [(16, 70, 5, 20), (16, 90, 0, 1), (2, 0, 0, 1), (0, 44, 0, 0)]
    out, lse, _ = _run(_q(gen, 4, G, Tq, D, BF), k, v, lens, causal=causal)
    if causal and Tq > 3:
        assert not out[2, :, :Tq - 3].any() and torch.isneginf(lse[2, :, :Tq - 3]).all()


def test_slots_choose_sequences_and_padding_rows_are_empty():
    gen = torch.Generator().manual_seed(3)
    k = kvref.Side(gen, 4, 2, 128, 16, 32, 4, 100, per_slot=True)
    v = kvref.Side(gen, 4, 2, 128, 16, 32, 4, 100, per_slot=True)
    lens = [(16, 100, 0, 16), (16, 40, 0, 16), (5, 0, 0, 0), (16, 99, 16, 31)]
    out, lse, _ = _run(_q(gen, 6, 4, 1, 128, BF), k, v, lens, slots=[3, -1, 0, 0, 4, 2])
    assert not out[1].any() and not out[4].any() and torch.isneginf(lse[1]).all()


def test_bad_pages_and_lengths_on_the_device_stay_in_the_buffers():
    """Table entries outside the pool hide their tokens; lengths outside the buffers are bounded by them."""
    gen = torch.Generator().manual_seed(4)
    k = kvref.Side(gen, 2, 2, 128, 16, 32, 6, 32)
    v = kvref.Side(gen, 2, 2, 128, 16, 32, 6, 32)
    table = [[0, 6, 2, 1 << 30], [-5, 4, 5, -2147483648]]
    _run(_q(gen, 2, 8, 1, 128, BF), k, v, [(16, 128, 0, 16), (16, 120, 16, 20)], table)
    st = [s.store(nv) for s in (k, v)]
    tab = torch.tensor([[0, 1, 2, 3], [4, 5, 4, 5]], dtype=torch.int32, device="cuda")
    q = _q(gen, 2, 8, 1, 128, BF).cuda()
    wild = torch.tensor([[99, 1 << 30, 40, 99], [-1, -7, -1, -3]], dtype=torch.int32, device="cuda")
    sane = torch.tensor([[16, 128, 8, 32], [0, 0, 0, 0]], dtype=torch.int32, device="cuda")
    assert torch.equal(nv.kv_attention(q, *st, wild, tab), nv.kv_attention(q, *st, sane, tab))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_hidden_tokens_reach_no_row(D):
    """NaN and infinities past the lengths, in unused pages and ring slots, and in tokens that only later rows see."""
    gen = torch.Generator().manual_seed(6)
    k = kvref.Side(gen, 1, 2, D, 16, 32, 4, 48)
    v = kvref.Side(gen, 1, 2, D, 16, 32, 4, 48)
    table = [[2, 0, 3]]
    lens = [(10, 100, 28, 9)]
    q = _q(gen, 1, 8, 4, D, BF)
    base = _run(q, k, v, lens, table)[0]
    for s in (k, v):
        s.sink[:, :, 10:] = math.nan
        s.window[:, :, 5:28] = math.inf
        s.scales[1], s.scales[3, :, 4:] = 0x7F, 0xFF
    assert torch.equal(_run(q, k, v, lens, table)[0], base)
    # the newest token (ring slot 36 % 32 = 4) is seen by the last query alone, the one before by the last two
    for s, a, b in ((k, math.nan, -math.inf), (v, math.inf, math.nan)):
        s.window[:, :, 4, 3], s.window[:, 1, 3, 5] = a, b
    got = _run(q, k, v, lens, table)[0]
    assert torch.equal(got[:, :, :2], base[:, :, :2]) and torch.isnan(got[:, :, 3].float()).any()
    assert torch.equal(got[:, :4, 2], base[:, :4, 2]) and torch.isnan(got[:, 4:, 2].float()).any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_poisoned_middle_tokens_of_later_rows(D):
    """The same with the newest tokens in the NVFP4 middle: a NaN block scale reaches the rows that see it, in the
    channels of its (rotated) block, and no other."""
    gen = torch.Generator().manual_seed(7)
    k = kvref.Side(gen, 1, 1, D, 16, 32, 1, 77)
    v = kvref.Side(gen, 1, 1, D, 16, 32, 1, 77)
    lens, q = [(16, 77, 0, 0)], _q(gen, 1, 3, 4, D, BF)
    base = _run(q, k, v, lens)[0]
    v.scales[0, 0, 75, 1] = 0x7F                    # seen by the last two queries
    v.scales[0, 0, 76, 2] = 0xFF                    # by the last
    got = _run(q, k, v, lens)[0]
    assert torch.equal(got[:, :, :2], base[:, :, :2])
    assert torch.isnan(got[0, :, 2].float()).any(0).nonzero().flatten().tolist() == list(range(16, 32))
    assert torch.isnan(got[0, :, 3].float()).any(0).nonzero().flatten().tolist() == list(range(16, 48))
    k.scales[0, 0, 76, 0] = 0x7F
    got = _run(q, k, v, lens)[0]
    assert torch.equal(got[:, :, :2], base[:, :, :2]) and torch.isnan(got[:, :, 3].float()).all()


def test_sharp_and_flat_rows_and_large_scores():
    """One token taking all the weight, all tokens alike, scores beyond exp's range, tiny and huge queries."""
    gen = torch.Generator().manual_seed(8)
    k = kvref.Side(gen, 1, 1, 128, 16, 32, 1, 500)
    v = kvref.Side(gen, 1, 1, 128, 16, 32, 1, 500)
    q = _q(gen, 1, 6, 1, 128, BF)
    q[0, 0] *= 0
    q[0, 1] *= 60
    q[0, 2] *= 1e-30
    q[0, 3] *= 200
    q[0, 4, 0, 5:] = 0
    _run(q, k, v, [(16, 500, 3, 32)], host=True)
    _run(q, k, v, [(16, 500, 3, 32)], host=True, scale=-0.3)
    _run(q, k, v, [(16, 500, 3, 32)], host=True, scale=0.0)


def test_large_window_is_spread_over_ranges():
    gen = torch.Generator().manual_seed(9)
    k = kvref.Side(gen, 1, 2, 128, 40, 1000, 1, 900)
    v = kvref.Side(gen, 1, 2, 128, 40, 1000, 1, 900)
    _run(_q(gen, 1, 4, 2, 128, BF), k, v, [(40, 900, 700, 990)], splits=3)
    _run(_q(gen, 1, 4, 1, 128, F16), k, v, [(40, 0, 700, 1000)])


@pytest.mark.parametrize("splits", [1, 2, 7, 128, 1000])
def test_every_split_count_gives_the_answer(splits):
    gen = torch.Generator().manual_seed(10)
    k = kvref.Side(gen, 2, 1, 128, 16, 32, 2, 2100)
    v = kvref.Side(gen, 2, 1, 128, 16, 32, 2, 2100)
    q = _q(gen, 2, 3, 1, 128, BF)
    a = _run(q, k, v, [(16, 2099, 0, 16), (16, 300, 0, 16)], splits=splits)[0]
    b = _run(q, k, v, [(16, 2099, 0, 16), (16, 300, 0, 16)], splits=splits)[0]
    assert torch.equal(a, b)


def test_strided_queries_and_outputs():
    """q as a projection leaves it (token-major slices of a wider buffer), out into a strided buffer, unaligned."""
    gen = torch.Generator().manual_seed(11)
    k = kvref.Side(gen, 2, 2, 64, 16, 32, 2, 100)
    v = kvref.Side(gen, 2, 2, 64, 16, 32, 2, 100)
    lens = torch.tensor([(16, 90, 0, 20), (16, 100, 16, 31)], dtype=torch.int32).cuda()
    st = [s.store(nv) for s in (k, v)]
    q = _q(gen, 2, 4, 3, 64, BF).cuda()
    ref, rl = nv.kv_attention(q, *st, lens, want_lse=True)
    for pad in (0, 1, 8):
        wide = torch.zeros(2, 3, 4 * 64 + 64 + pad, dtype=BF, device="cuda")
        qs = wide[:, :, 64:64 + 256].unflatten(-1, (4, 64)).transpose(1, 2)
        qs.copy_(q)
        ob = torch.full((2, 3, 5 * 64 + pad), 7.0, dtype=BF, device="cuda")
        o = ob[:, :, :256].unflatten(-1, (4, 64)).transpose(1, 2)
        lse = torch.empty(2, 4, 3, device="cuda")
        nv.kv_attention(qs, *st, lens, out=o, lse=lse)
        assert torch.equal(o, ref) and torch.equal(lse, rl) and (ob[:, :, 256:] == 7).all()


def test_captured_call_follows_lengths_and_pages_and_streams_do_not_interfere():
    gen = torch.Generator().manual_seed(12)
    k = kvref.Side(gen, 3, 2, 128, 16, 32, 40, 32)
    v = kvref.Side(gen, 3, 2, 128, 16, 32, 40, 32)
    st = [s.store(nv) for s in (k, v)]
    q = _q(gen, 3, 8, 1, 128, BF).cuda()
    table = torch.randperm(39, generator=gen)[:39].view(3, 13).int().cuda()
    lens = torch.tensor([(16, 300, 0, 20)] * 3, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        nv.kv_attention(q, *st, lens, table, out=out)                # warm up outside the capture
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    out2 = torch.empty_like(q)
    with torch.cuda.graph(g1):
        nv.kv_attention(q, *st, lens, table, out=out)
    with torch.cuda.graph(g2):
        nv.kv_attention(q, *st, lens, table, out=out2)
    for mid in (300, 0, 416, 5):
        lens[:, 1] = mid
        table.copy_(table.roll(1, 0))
        torch.cuda.synchronize()
        want = nv.kv_attention(q, *st, lens, table)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want)


def test_offsets_past_32_bits():
    """A contiguous cache whose code bytes pass 4 GiB: the last slot is read, not a wrapped one."""
    gen = torch.Generator().manual_seed(13)
    cap, slots = 1 << 18, 260                       # 260 x 2^18 rows x 64 bytes = 4.06 GiB a side
    small = kvref.Side(gen, 1, 1, 128, 16, 32, 1, 100), kvref.Side(gen, 1, 1, 128, 16, 32, 1, 100)
    stores = []
    for s in small:
        codes = torch.zeros(slots, 1, cap, 64, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(slots, 1, cap, 8, dtype=torch.uint8, device="cuda")
        codes[-1, :, :100], scales[-1, :, :100] = s.codes[0].cuda(), s.scales[0].cuda()
        sink, win = torch.zeros(slots, 1, 16, 128, dtype=BF, device="cuda"), torch.zeros(slots, 1, 32, 128, dtype=BF, device="cuda")
        sink[-1], win[-1] = s.sink[0].cuda(), s.window[0].cuda()
        stores.append(nv.KvStore(sink, win, codes, scales, s.gscale.cuda()))
    q = _q(gen, 1, 4, 1, 128, BF)
    out, lse = nv.kv_attention(q.cuda(), *stores, (16, 100, 0, 20), slots=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"),
                               want_lse=True)
    kvref.check(out, lse, kvref.attention(q, *small, [(16, 100, 0, 20)]))


def test_refusals():
    gen = torch.Generator().manual_seed(14)
    k = kvref.Side(gen, 2, 2, 128, 16, 32, 4, 24)
    s = k.store(nv)
    q = _q(gen, 2, 4, 1, 128, BF).cuda()
    lens = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        nv.kv_attention(q.float(), s, s, lens)
    with pytest.raises(TypeError):
        nv.kv_attention(q.cpu(), s, s, lens)
    with pytest.raises(ValueError):
        nv.kv_attention(q[:, :3], s, s, lens)                       # 3 query heads on 2
    with pytest.raises(ValueError):
        nv.kv_attention(q[..., :64], s, s, lens)                    # head_dim
    with pytest.raises(ValueError):
        nv.kv_attention(torch.cat([q, q], -1)[..., ::2], s, s, lens)   # channels not contiguous
    with pytest.raises(ValueError):
        nv.kv_attention(q, s, s, lens.long())
    with pytest.raises(ValueError):
        nv.kv_attention(q, s, s, lens[:1])
    with pytest.raises(nv.NVFP4Error):
        nv.kv_attention(q, s, s, lens, table)                       # pages of 24 rows
    with pytest.raises(nv.NVFP4Error):
        nv.kv_attention(q, s, s, (16, 25, 0, 0))                    # more than a page
    with pytest.raises(nv.NVFP4Error):
        nv.kv_attention(q, s, s, (16, 1, 32, 0))                    # head outside the ring
    with pytest.raises(ValueError):
        nv.kv_attention(torch.cat([q, q]), s, s, lens)              # more rows than slots
    with pytest.raises(ValueError):
        nv.kv_attention(q, s, s, lens, out=q)
    with pytest.raises(ValueError):
        nv.kv_attention(q, s, s, lens, out=q[:1].expand(2, 4, 1, 128))
    with pytest.raises(ValueError):
        nv.kv_attention(q, s, s, lens, splits=4, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(nv.NVFP4Error):
        nv.kv_attention(q, s, s, lens, splits=65536)
    with pytest.raises(ValueError):
        nv.KvStore(k.sink.cuda(), k.window[:1].cuda(), k.codes.cuda(), k.scales.cuda(), k.gscale.cuda())
    with pytest.raises(ValueError):
        nv.KvStore(k.sink.cuda(), k.window.cuda(), k.codes.cuda(), k.scales[:3].cuda(), k.gscale.cuda())
    assert nv.kv_attention(q[:0], s, s, lens).shape == (0, 4, 1, 128)
    assert nv.kv_attention(q[:, :, :0], s, s, lens).shape == (2, 4, 0, 128)


@pytest.mark.parametrize("p", [-112, 60, 112])
@pytest.mark.parametrize("D", [64, 256])
def test_far_ranges_of_query_and_keys_cancel(p, D):
    """q times 2^p against keys times 2^-p: every product is the same, so is every bit."""
    gen = torch.Generator().manual_seed(D)
    q = _q(gen, 2, 4, 1, D, BF).cuda()
    lens = torch.tensor([(16, 301, 16, 29), (16, 33, 0, 16)], dtype=torch.int32).cuda()
    k, v = (kvref.Side(gen, 2, 1, D, 16, 32, 2, 333) for _ in (0, 1))
    want = nv.kv_attention(q, k.store(nv), v.store(nv), lens, want_lse=True)
    k.sink, k.window, k.gscale = (t * 2.0 ** -p for t in (k.sink, k.window, k.gscale))
    got = nv.kv_attention(q * 2.0 ** p, k.store(nv), v.store(nv), lens, want_lse=True)
    assert torch.isfinite(got[0]).all() and all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_of_sizes_in_words():
    gen = torch.Generator().manual_seed(0)
    k = kvref.Side(gen, 1, 1, 80, 0, 16, 1, 16).store(nv)
    with pytest.raises(ValueError, match="head_dim"):
        nv.kv_attention(torch.zeros(1, 1, 1, 80, dtype=BF, device="cuda"), k, k, (0, 16, 0, 16))
    k = kvref.Side(gen, 1, 1, 64, 0, 16, 1, 16).store(nv)
    for lens in ((0, 2 ** 32 + 5, 0, 1), (0, -1, 0, 1), (0, 5, 2 ** 31, 1)):
        with pytest.raises(ValueError, match="lengths"):
            nv.kv_attention(torch.zeros(1, 1, 1, 64, dtype=BF, device="cuda"), k, k, lens)
