"""Decode cache and its calls without a GPU: tensors on other devices, refused calls that change nothing.  Launches are
replaced by recorders; a `meta` tensor stands for one on another device."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv
import nvfp4_block_scaled_11_b200.kvcache as kc
from nvfp4_block_scaled_11_b200 import build as nvbuild

BF = torch.bfloat16


class _Library:
    """Every entry point records its call and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name == "nvfp4_sf_mma_bytes":
            return lambda *a: 512
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def launches(monkeypatch):
    """(device, entry point) of every launch; CPU tensors pass as the device's."""
    lib, out = _Library(), []

    def launch(device, fn, *args):
        fn(*args, None)
        out.append((device, lib.calls[-1][0]))
    monkeypatch.setattr(nv, "_cuda", lambda t, name: t)
    monkeypatch.setattr(nv, "lib", lambda: lib)
    monkeypatch.setattr(nv, "_launch", launch)
    return out


def test_quantizing_calls_refuse_tensors_of_another_device(launches):
    k, g = torch.zeros(1, 2, 40, 32, dtype=BF), torch.zeros(1)
    codes, scales = torch.zeros(1, 2, 64, 16, dtype=torch.uint8), torch.zeros(1, 2, 64, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="is on"):
        nv.kv_gscale(k, 4, 4, out=g.to("meta"))
    with pytest.raises(ValueError, match="is on"):
        nv.kv_gscale(k.to("meta"), 4, 4, out=g)
    for bad in (dict(k=k.to("meta")), dict(g=g.to("meta")), dict(codes=codes.to("meta")), dict(scales=scales.to("meta"))):
        a = dict(k=k, g=g, codes=codes, scales=scales) | bad
        with pytest.raises(ValueError, match="is on"):
            nv.kv_append(a["k"], 0, 16, a["g"], a["codes"], a["scales"], 0)
    assert not launches


def test_quantizing_calls_run_on_their_tensors_device(launches):
    """Whatever device is current: the launch goes through the one place that switches to the tensors' device."""
    k, g = torch.zeros(1, 2, 40, 32, dtype=BF), torch.zeros(1)
    codes, scales = torch.zeros(1, 2, 64, 16, dtype=torch.uint8), torch.zeros(1, 2, 64, 2, dtype=torch.uint8)
    nv.kv_gscale(k, 4, 4, out=g)
    nv.kv_append(k, 0, 16, g, codes, scales, 0)
    nv.KvAppendBatch([(k, g, codes, scales, True, False)])(0, 16, 0)
    assert launches == [(k.device, n) for n in ("nvfp4_kv_gscale", "nvfp4_kv_append", "nvfp4_kv_append_batch")]


# ---- the paged cache ----
H, D, PAGE = 2, 32, 32


@pytest.fixture
def log(monkeypatch):
    """What the cache would launch; `fail` names the call that raises instead."""
    out = dict(append=[], copies=[], fail=None)

    def call(name, *a):
        if out["fail"] == name:
            raise RuntimeError("launch")
        out.setdefault(name, []).append(a)
    monkeypatch.setattr(kc, "_append_records", lambda recs, lo, hi, dev: call("append", recs.copy()))
    monkeypatch.setattr(kc, "kv_gscale", lambda k, s, r, rot, out: call("gscale") or out.fill_(0.5))
    monkeypatch.setattr(kc, "copy_pages", lambda arrays, src, dst: call("copies", list(src), list(dst)))
    return out


def _cache(pages=12, slots=4, layers=2, **kw):
    return kc.NVFP4PagedKVCache(layers, slots, H, D, pages, PAGE, device="cpu", **kw)


def _prompt(T, layers=2):
    return [torch.zeros(H, T, D, dtype=BF) for _ in range(layers)]


def test_prompts_on_another_device_are_refused(log):
    c = _cache()
    s = c.alloc()
    good, away = _prompt(100), [x.to("meta") for x in _prompt(100)]
    for ks, vs in ((away, good), (good, away), (good, [good[0], away[1]])):
        with pytest.raises(ValueError, match="on meta"):
            c.prefill(s, ks, vs)
    for bad in (1.0, None, [0.0]):
        with pytest.raises(TypeError):
            c.prefill(s, [bad, bad], good)
    with pytest.raises(ValueError):
        c.prefill(s, [x[0] for x in good], good)                     # no heads
    assert c.pages_free == 12 and c.length(s) == 0
    c.prefill(s, good, good)
    assert c.length(s) == 100


@pytest.mark.parametrize("call", ["gscale", "append"])
def test_a_prefill_that_fails_gives_its_pages_back(log, call):
    c = _cache()
    a, s = c.alloc(), c.alloc()
    c.prefill(a, _prompt(100), _prompt(100))
    log["fail"] = call
    with pytest.raises(RuntimeError, match="launch"):
        c.prefill(s, _prompt(32 + 40), _prompt(32 + 40))
    assert c.pages_free == 12 - 3 and c.length(s) == 0 and c._held[s] == [] and (c._table[s] == -1).all()
    log["fail"] = None
    c.prefill(s, _prompt(32 + 40), _prompt(32 + 40))                 # the slot can be used again at once
    assert c.length(s) == 72 and c.table[s, :3].tolist() == [3, 4, -1]


def test_a_step_whose_flush_fails_can_be_made_again(log):
    c = _cache()
    s = c.alloc()
    c.prefill(s, _prompt(32 + 24), _prompt(32 + 24))
    for _ in range(16):
        c.step([s])
    before, log["fail"] = c._lens.copy(), "append"
    with pytest.raises(RuntimeError, match="launch"):
        c.step([s])
    assert (c._lens == before).all() and c.length(s) == 72
    log["fail"], log["append"] = None, []
    c.step([s])
    ((recs,),) = log["append"]
    assert recs["first"].tolist() == [0, 8] * 4 and recs["t0"].tolist() == [24, 0] * 4
    assert c.lens[s].tolist() == [16, 40, 16, 17]


def test_refused_rows_are_not_stored(log):
    """Neither side's when one is refused, and no layer's that there is not (-1 is not the last one)."""
    c = _cache()
    s = c.alloc()
    c.prefill(s, _prompt(40), _prompt(40))
    st, before = c.step([s]), c.window.clone()
    x = torch.ones(1, H, 1, D, dtype=BF)
    for k, v in ((x, x[:, :1]), (x, x.float()), (x, x.to("meta")), (x[:, :, :0], x)):
        with pytest.raises(ValueError):
            c.store(st, 0, k, v)
    for layer in (-1, 2):
        with pytest.raises(IndexError):
            c.store(st, layer, x, x)
    assert torch.equal(c.window, before)


def test_caches_hold_no_graph(log):
    """Rows of a projection whose weights train: the buffers stay plain, so no graph grows with the sequence."""
    c = _cache()
    s = c.alloc()
    p = [x.requires_grad_() for x in _prompt(40)]
    c.prefill(s, p, p)
    x = torch.ones(1, H, 1, D, dtype=BF, requires_grad=True)
    c.store(c.step([s]), 1, x, x * 2)
    assert not c.window.requires_grad and not c.sink.requires_grad and c.window[1, 1, s, 0, 16, 0] == 2
    one = kc.NVFP4KVCache(1, H, D, capacity=16, device="cpu")
    one.prefill(p[0][None][:, :, :32])
    one.append(x)
    assert not one.window.requires_grad and not one.sink.requires_grad and one.length == 33


def test_replaced_buffers_are_read(monkeypatch):
    """A cache whose buffer is replaced gives attention the new one, and the same view again while none is."""
    monkeypatch.setattr(kc, "KvStore", lambda *a: a)
    one, many = kc.NVFP4KVCache(1, H, D, capacity=16, device="cpu"), _cache()
    for c, get in ((one, one.store), (many, lambda: many.stores(1)[1])):
        for i, name in enumerate(("sink", "window", "codes", "scales", "gscale")):
            old = get()
            assert get() is old
            setattr(c, name, getattr(c, name).clone())
            new = get()
            assert [a.data_ptr() == b.data_ptr() for a, b in zip(old[:5], new[:5])] == [j != i for j in range(5)]
        old = get()
        c.codes.data = c.codes.clone()                               # the same tensor, its memory moved
        assert get() is not old and get() is get()


# ---- the C entry points, on fake pointers: everything here is decided on the host ----
ARG, SIZE = -1, -2


@pytest.fixture(scope="module")
def L():
    nvbuild.build()
    return nv.lib()


def _desc(k=None, v=None, **kw):
    store = dict(sink=0x10000, window=0x20000, codes=0x30000, scales=0x40000, gscale=0x50000, gscale_stride=0, rotate=1,
                 scale_layout=0)
    d = nv._KvAttentionDesc()
    for name, x in (dict(q=0x60000, out=0x70000, B=1, Hq=8, Hkv=2, Tq=1, D=128, slots=1, sink_rows=16, window_rows=32, pages=4,
                         page_rows=64, n_sink=16, n_window=16, dtype=1, causal=1, scale=0.1) | kw).items():
        setattr(d, name, x)
    for name, s in (("k", store | (k or {})), ("v", store | (v or {}))):
        setattr(d, name, nv._KvStore(*(s[f] for f, _ in nv._KvStore._fields_)))
    return d


@pytest.mark.parametrize("side", ["k", "v"])
def test_a_pool_without_pages_still_needs_the_tensor_scale(L, side):
    """Tokens of pages outside the pool are hidden, but the kernel reads their sequence's tensor scale."""
    paged = dict(table=0x80000, table_cols=4, lens=0x90000)
    for kw in (dict(pages=0), dict(pages=4)):
        assert L.nvfp4_kv_attention(ctypes.byref(_desc(**{side: dict(gscale=None)}, **paged, **kw)), 1, None, 0, None) == ARG
    # nothing to read where no middle can be: past the check of the stores, to a size that is refused after it
    none = dict(paged, table_cols=0, pages=0, Hq=1 << 30, Hkv=1, Tq=4)
    assert L.nvfp4_kv_attention(ctypes.byref(_desc(**{side: dict(gscale=None, codes=None, scales=None)}, **none)), 1, None, 0,
                                None) == SIZE


# ---- the paged cache under capture (see test_gpu_decode_graphs for the graphs themselves) ----
def test_books_are_not_kept_in_a_graph(log, monkeypatch):
    """Calls that change the host's lengths and pages are refused while a graph is captured, and change nothing."""
    c = _cache()
    s, e = c.alloc(), c.alloc()
    c.prefill(s, _prompt(100), _prompt(100))
    before, free = c._lens.copy(), c.pages_free
    monkeypatch.setattr(c, "_capturing", lambda: True)
    for call in (lambda: c.step([s]), lambda: c.free(s), lambda: c.fork(s), lambda: c.compact(),
                 lambda: c.prefill(e, _prompt(100), _prompt(100))):
        with pytest.raises(RuntimeError, match="capture"):
            call()
    assert (c._lens == before).all() and c.pages_free == free and c._held[s] == [0, 1, 2] and not log["copies"]


@pytest.mark.parametrize("n", [1, 3, 16])
def test_captured_rows_go_where_the_lengths_on_the_device_say(log, monkeypatch, n):
    """store's captured form, run with each step's lengths and the FIRST step's object, against store with each step's
    own: the same windows, through flushes and around the ring."""
    a, b = _cache(pages=40), _cache(pages=40)
    for c in (a, b):
        for T in (32, 32 + 20, 32 + 7):
            c.prefill(c.alloc(), _prompt(T), _prompt(T))
    first = b.step([2, 0], n)
    for i in range(20):
        st = a.step([2, 0], n)
        if i:
            b.step([2, 0], n)
        for layer in range(2):
            x = torch.randn(2, H, n, D).to(BF)
            a.store(st, layer, x, -x)
            with monkeypatch.context() as m:
                m.setattr(b, "_capturing", lambda: True)
                b.store(first, layer, x, -x)
        assert torch.equal(a.window, b.window) and torch.equal(a.lens, b.lens)
    assert any(t is first.slot_ids for t in b._captured)              # kept for the graph that reads it


@pytest.mark.parametrize("T,ends", [(32, (0, 0)), (33, (16, 16)), (60, (16, 16))])
def test_a_prompt_without_a_middle_sets_the_scale_by_all_of_it(monkeypatch, T, ends):
    """Both caches: over an empty middle the scale would be 0, and every token quantized with it 0."""
    seen = []
    monkeypatch.setattr(kc, "kv_gscale", lambda k, s, r, rot, out: seen.append((s, r)))
    monkeypatch.setattr(kc, "kv_append", lambda *a: None)
    monkeypatch.setattr(kc, "_append_records", lambda *a: None)
    one, many = kc.NVFP4KVCache(1, H, D, capacity=64, device="cpu"), _cache(layers=1)
    one.prefill(torch.ones(1, H, T, D, dtype=BF))
    many.prefill(many.alloc(), _prompt(T, 1), _prompt(T, 1))
    assert seen == [ends] * 3


def test_outputs_that_overlap_themselves_are_told():
    """By brute force over small strided views: accepted only where every element has its own place; everything that
    slicing, transposing and splitting one buffer gives is accepted."""
    import itertools
    buf = torch.arange(400)
    told = 0
    for sizes in itertools.product((1, 2, 3), repeat=3):
        for strides in itertools.product((0, 1, 2, 3, 5, 6, 9), repeat=3):
            t = buf.as_strided(sizes, strides)
            alone = len(set(t.flatten().tolist())) == t.numel()
            try:
                nv._no_shared_elements(t, "out")
                assert alone, (sizes, strides)
            except ValueError:
                told += not alone
    assert told > 1000
    base = torch.zeros(4, 6, 10, 8)
    for t in (base, base.transpose(1, 2), base[:, ::2], base[1:3, :, 2:9:3].permute(2, 0, 1, 3), base.unflatten(1, (2, 3))[:, 1],
              base[:0], base[..., :1], base[:, :, :, 3:5].transpose(0, 2)):
        nv._no_shared_elements(t, "out")
    with pytest.raises(ValueError):                                  # windows that slide by less than their width
        nv._no_shared_elements(torch.zeros(100).as_strided((4, 8), (4, 1)), "out")


def test_views_of_other_dims_are_taken_by_their_span():
    buf = torch.zeros(64)
    a = buf[:32].view(2, 4, 4)
    assert nv._overlap(a, buf[16:48]) and nv._overlap(buf[31:40], a) and not nv._overlap(a, buf[32:]) and nv._overlap(a, buf[8:9])


def test_tables_of_large_pools_stay_within_what_attention_takes(L):
    """A pool of more tokens than one sequence may have: its table has the columns that attention accepts, not one per page."""
    c = kc.NVFP4PagedKVCache(1, 1, 1, 64, 1000, 1 << 20, device="meta")
    assert c.table.shape == (1, 511)
    paged = dict(table=0x80000, lens=0x90000, page_rows=1 << 20, pages=1000, Hkv=1)
    assert L.nvfp4_kv_attention(ctypes.byref(_desc(**paged, table_cols=512)), 1, None, 0, None) == SIZE
    # the table is accepted: what is refused is the missing q
    assert L.nvfp4_kv_attention(ctypes.byref(_desc(**paged, table_cols=511, q=None)), 1, None, 0, None) == ARG
    assert kc.NVFP4PagedKVCache(1, 1, 1, 64, 1000, 64, device="meta").table.shape == (1, 1000)
