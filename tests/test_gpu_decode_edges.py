"""Edges of attention over the cache and of the calls around it: pools and batches without entries, the far end of a long
cache, layouts in combination, large batches, many query rows."""
import ctypes
import math

import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv
from nvfp4_block_scaled_11_b200 import kvcache as kc
from tests import kvref

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def test_no_slots_make_every_sequence_empty():
    """Slot indexes into a cache of no slots, through the C entry point: nothing is read of lengths that hold no entry
    (here 4 words that would give every sequence tokens, did they count)."""
    q = torch.randn(3, 4, 1, 128).to(BF).cuda()
    out, lse = torch.full_like(q, 7), torch.full((3, 4, 1), 7.0, device="cuda")
    lens = torch.tensor([16, 64, 0, 16], dtype=torch.int32, device="cuda")
    slot = torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda")
    d = nv._KvAttentionDesc()
    for name, x in dict(q=q.data_ptr(), out=out.data_ptr(), lse=lse.data_ptr(), q_sb=512, q_sh=128, q_st=128, out_sb=512, out_sh=128,
                        out_st=128, B=3, Hq=4, Hkv=2, Tq=1, D=128, slots=0, pages=0, page_rows=0, lens=lens.data_ptr(),
                        slot=slot.data_ptr(), dtype=1, causal=1, scale=0.1).items():
        setattr(d, name, x)
    assert nv.lib().nvfp4_kv_attention(ctypes.byref(d), 1, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert not out.any() and torch.isneginf(lse).all()


def test_scale_tiles_past_32_bits():
    """One sequence of more than 2^28 tokens of 256 channels, scales in tiles: its last tokens are read with their own scales
    (those bytes begin at 2^32 of the matrix).  All tokens but the last 128 are zeros: scores 0, values 0."""
    gen = torch.Generator().manual_seed(21)
    D, n, far = 256, 128, 1 << 28
    s = kvref.Side(gen, 1, 1, D, 0, 16, 1, n, rotate=False)
    codes = torch.zeros(1, 1, far + n, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(nv.sf_mma_bytes(far + n, D, 1), dtype=torch.uint8, device="cuda")
    codes[0, 0, far:], scales[-n * D // 16:] = s.codes[0, 0].cuda(), kvref.tile_scales(s.scales.flatten(0, 1)).cuda()
    st = nv.KvStore(s.sink.cuda(), s.window.cuda(), codes, scales, s.gscale.cuda(), False, True)
    val = s.tokens(0, (0, n, 0, 0), None)[0][0]                       # [128, 256] in 64 bits
    q = (torch.randn(1, 2, 1, D, generator=gen) * 12).to(BF)
    x = q[0, :, 0].double() @ val.T * D ** -0.5
    assert x.max() > 20                                               # enough to be seen beside e^0 2^28 times
    m = x.amax(1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(1, keepdim=True) + far * torch.exp(-m)
    want, mag = p @ val / l, p @ val.abs() / l
    out, lse = nv.kv_attention(q.cuda(), st, st, (0, far + n, 0, 0), want_lse=True)
    # FP32 scores of up to |x| and sums of the parts (2^28 tokens over at least 148 * 4 warps' 8 lanes a row), FP16 numerators
    rel = float(2 * x.abs().max() * 2.0 ** -20 + (far / (148 * 32) + 64) * 2.0 ** -24)
    assert ((out[0, :, 0].cpu().double() - want).abs() <= mag * (rel + 2.0 ** -11) + 2.0 ** -8 * want.abs() + 1e-9).all()
    assert ((lse[0, :, 0].cpu().double() - (m + torch.log(l))[:, 0]).abs() <= rel + 2.0 ** -20).all()
    assert want.abs().max() > 0.5


def _run(q, k, v, lens, table=None, slots=None, **kw):
    dev = lambda t: None if t is None else torch.as_tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    out, lse = nv.kv_attention(q.cuda(), k.store(nv), v.store(nv), dev(lens), dev(table), dev(slots), want_lse=True, **kw)
    torch.cuda.synchronize()
    kvref.check(out, lse, kvref.attention(q, k, v, lens, table if table is None else torch.as_tensor(table), slots,
                                          kw.get("causal", True)))
    return out


@pytest.mark.parametrize("tk,tv", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 48), (256, 16), (64, 32), (128, 64), (256, 128), (128, 160)])
def test_scale_tiles_in_pages_and_on_one_side(D, page, tk, tv):
    """Each page's scales in tiles of their own, for both sides or one: pages that end inside a tile, inside 32 rows of one,
    and that hold several."""
    gen = torch.Generator().manual_seed(D + page)
    mids = [333, page, 0, 31]
    need = [-(-m // page) for m in mids]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((4, max(need)), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    k, v = (kvref.Side(gen, 4, 2, D, 16, 32, pages, page, tile=t, per_slot=True) for t in (tk, tv))
    _run((2 * torch.randn(4, 6, 1, D, generator=gen)).to(BF), k, v, [(16, m, 16, 17) for m in mids], table)


@pytest.mark.parametrize("tk,tv", [(True, False), (False, True)])
@pytest.mark.parametrize("D,cap", [(64, 129), (128, 300), (256, 130)])
def test_scale_tiles_on_one_side_of_a_contiguous_cache(D, cap, tk, tv):
    gen = torch.Generator().manual_seed(D + cap)
    k, v = (kvref.Side(gen, 2, 2, D, 16, 32, 2, cap, tile=t) for t in (tk, tv))
    _run((2 * torch.randn(2, 4, 2, D, generator=gen)).to(F16), k, v, [(16, cap, 0, 16), (3, cap - 1, 16, 32)])


@pytest.mark.parametrize("B", [128, 129, 300])
def test_more_sequences_than_threads_of_a_cta(B):
    """Ragged batches whose rows are shared out to the threads that add their work up: one, two and three rows each, some
    of them empty or of slots that do not exist."""
    gen = torch.Generator().manual_seed(B)
    k, v = (kvref.Side(gen, 40, 1, 64, 16, 32, 90, 32, per_slot=True) for _ in (0, 1))
    table = torch.randint(0, 90, (40, 9), generator=gen).int()
    lens = [(int(a), int(m), 0, int(w)) for a, m, w in zip(torch.randint(0, 17, (40,), generator=gen),
                                                          torch.randint(0, 289, (40,), generator=gen) * torch.randint(0, 2, (40,), generator=gen),
                                                          torch.randint(0, 33, (40,), generator=gen))]
    slots = torch.randint(-1, 42, (B,), generator=gen).tolist()
    q = (2 * torch.randn(B, 2, 1, 64, generator=gen)).to(BF)
    a = _run(q, k, v, lens, table, slots, max_mid=288)
    assert torch.equal(a, _run(q, k, v, lens, table, slots, max_mid=288))
    _run(q, k, v, lens, table, slots, splits=5)


@pytest.mark.parametrize("D,G,Tq,dt", [(256, 12, 3, BF), (256, 12, 3, F16), (256, 4, 8, F16), (256, 1, 17, BF), (128, 4, 4, F16),
                                       (128, 16, 8, F16), (128, 3, 43, BF), (64, 8, 16, F16)])
def test_many_query_rows(D, G, Tq, dt):
    """Rows in several tiles of 16 and a rest, at every head_dim, for both types; the newest tokens in the window, in the
    middle and in both."""
    gen = torch.Generator().manual_seed(D + G * Tq)
    k, v = (kvref.Side(gen, 3, 2, D, 16, 32, 3, 300, per_slot=True) for _ in (0, 1))
    _run((1.5 * torch.randn(3, 2 * G, Tq, D, generator=gen)).to(dt), k, v, [(16, 270, 5, 32), (16, 299, 0, 2), (7, 0, 31, 9)])

def test_a_dominating_middle_token_under_an_older_reference():
    """Numerators of the middle are rounded to FP16 once, by up to half a step of 11 significant bits: 2^-11.  A token that
    holds nearly all of the weight, 2^4 (1 + 0.51 2^-10) of the reference (under its limit of 2^5, so that the reference
    stays), is rounded up by 0.49 2^-10, its share of the denominator not at all; the output's own rounding adds up to
    half a step, in the same direction here."""
    w = 16 * (1 + 0.51 * 2.0 ** -10)
    key, value = torch.full((160,), 15, dtype=torch.uint8), torch.zeros(160, dtype=torch.uint8)
    key[0], key[130], value[130] = 0, 2, 2                            # E2M1: -6 (far below) but for 0 and 1; 0 but for 1
    scales = torch.full((1, 1, 160, 4), 0x38, dtype=torch.uint8)      # 1
    scales[0, 0, key == 15] = 0x50                                    # 8: e^-133 of the first token's weight each
    sides = []
    # tokens 0 and 130 lie in the first and the fifth tile, which one warp takes; the result is 1 + 0.02 2^-10
    for codes, g in ((key, 1.0), (value, (1 + w) / w * (1 + 0.02 * 2.0 ** -10))):
        s = kvref.Side(torch.Generator().manual_seed(0), 1, 1, 64, 0, 16, 1, 160, rotate=False)
        s.codes, s.scales, s.gscale = torch.zeros_like(s.codes), scales, torch.tensor([g])
        s.codes[..., 0] = codes                                       # channel 0
        sides.append(s)
    q = torch.zeros(1, 1, 1, 64, dtype=F16)
    q[..., 0] = 1
    scale = math.log(w)
    out, lse = nv.kv_attention(q.cuda(), *(s.store(nv) for s in sides), (0, 160, 0, 0), scale=scale, splits=1, want_lse=True)
    want, l, _, _ = kvref.attention(q, *sides, [(0, 160, 0, 0)], scale=scale)
    assert abs(float(want[..., 0]) - (1 + 0.02 * 2.0 ** -10)) < 2.0 ** -22 and not want[..., 1:].any()
    off = (out.cpu().double() - want).abs()
    assert (off <= want * (2.0 ** -11 + 2.0 ** -17) * (1 + 2.0 ** -10) + 2.0 ** -11).all(), float(off.max())
    assert not out[..., 1:].any() and abs(float(lse) - float(l)) < 2.0 ** -19    # scores of 4 in FP32


def test_caches_that_start_without_a_middle():
    """The shortest prompt, then tokens that fill pages: the contiguous cache against the definition, and the same bytes as
    the paged one."""
    gen = torch.Generator().manual_seed(22)
    H, D, T = 2, 64, 32
    rows = lambda n: torch.randn(1, H, n, D, generator=gen).to(BF).cuda()  # noqa: E731
    k, v = rows(T), rows(T)
    one = [kc.NVFP4KVCache(1, H, D, capacity=96) for _ in (0, 1)]
    many = kc.NVFP4PagedKVCache(1, 1, H, D, 4, 32)
    one[0].prefill(k), one[1].prefill(v)
    many.prefill(many.alloc(), [k], [v])
    for _ in range(70):
        k, v = rows(1), rows(1)
        one[0].append(k), one[1].append(v)
        st = many.step([0])
        many.store(st, 0, k, v)
    q = torch.randn(1, 6, 1, D, generator=gen).to(BF)
    out, lse = kc.attend(q.cuda(), *one, want_lse=True)
    sides = []
    for i, c in enumerate(one):
        s = kvref.Side(gen, 1, H, D, 16, 32, 1, 96)
        s.sink, s.window, s.codes, s.scales, s.gscale = (t.cpu() for t in (c.sink, c.window, c.codes, c.scales, c.gscale))
        sides.append(s)
        n = c.n_mid
        assert n == 64 and float(s.gscale) > 0 and (s.codes[0, :, :n] != 0).any(2).all()
        paged = many.codes[0, i, many.table[0, :2].long()].transpose(0, 1).flatten(1, 2).cpu()
        assert torch.equal(paged[:, :n], s.codes[0, :, :n]) and float(many.gscale[0, i, 0]) == float(s.gscale)
    c = one[0]
    kvref.check(out, lse, kvref.attention(q, *sides, [(c.n_sink, c.n_mid, c.head, c.n_window)]))


def test_written_buffers_share_no_memory():
    """lse and workspace inside q, out or each other are refused; side by side in one buffer they are not."""
    gen = torch.Generator().manual_seed(23)
    k, v = (kvref.Side(gen, 2, 2, 64, 16, 32, 2, 100).store(nv) for _ in (0, 1))
    lens = (16, 90, 0, 20)
    need = nv.lib().nvfp4_kv_attention_workspace_bytes(2, 64, 4)
    buf = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    at = lambda a, n, dt=BF: buf[a:a + n].view(dt)  # noqa: E731
    q, out, lse, ws = at(0, 1024).view(2, 4, 1, 64), at(1024, 1024).view(2, 4, 1, 64), at(2048, 32, torch.float32), buf[2560:2560 + need]
    q.copy_(torch.randn(2, 4, 1, 64, generator=gen))
    want, wl = nv.kv_attention(q.clone(), k, v, lens, splits=4, want_lse=True)
    nv.kv_attention(q, k, v, lens, splits=4, out=out, lse=lse, workspace=ws)
    assert torch.equal(out, want) and torch.equal(lse.view(2, 4, 1), wl)
    for kw in (dict(lse=at(64, 32, torch.float32)), dict(lse=at(1024 + 992, 32, torch.float32)), dict(workspace=buf[1024:]),
               dict(workspace=buf[:need]), dict(workspace=buf[2064:]), dict(workspace=buf[:need].view(BF)),
               dict(lse=lse.view(2, 4, 1), workspace=buf[2064:2064 + need].view(torch.float32))):
        with pytest.raises(ValueError, match="overlap"):
            nv.kv_attention(q, k, v, lens, splits=4, **(dict(out=out, lse=lse, workspace=ws) | kw))
    assert torch.equal(out, want)
