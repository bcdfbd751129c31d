"""Host logic of the paged cache without a GPU: which pages sequences own and share, what is quantized where, what is
copied, and the errors raised before anything changes.  Launches are replaced by recorders."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_11_b200.kvcache as kc

H, D, PAGE = 2, 32, 32


@pytest.fixture
def log(monkeypatch):
    out = dict(append=[], copies=[])
    monkeypatch.setattr(kc, "_append_records", lambda recs, lo, hi, dev: out["append"].append(recs.copy()))
    monkeypatch.setattr(kc, "kv_gscale", lambda k, s, r, rot, out: out.fill_(0.5))

    def copy_pages(arrays, src, dst):
        out["copies"].append((list(src), list(dst)))
        for t, dim in arrays:
            t.index_copy_(dim, torch.tensor(dst), t.index_select(dim, torch.tensor(src)))
    monkeypatch.setattr(kc, "copy_pages", copy_pages)
    return out


def _cache(pages=12, slots=4, layers=2, **kw):
    return kc.NVFP4PagedKVCache(layers, slots, H, D, pages, PAGE, device="cpu", **kw)


def _prompt(T, layers=2, v=0.0):
    return [torch.full((H, T, D), v + i, dtype=torch.bfloat16) for i in range(layers)]


def _consistent(c):
    """Reference counts, free list, table and lengths agree with the pages that sequences hold."""
    count = [0] * c.n_pages
    for s, held in enumerate(c._held):
        assert c.table[s].tolist() == (held or []) + [-1] * (c.table.shape[1] - len(held or []))
        assert c.lens[s].tolist() == c._lens[s].tolist()
        if held is not None:
            assert len(held) == -(-int(c._lens[s, 1]) // PAGE) and len(set(held)) == len(held)
            for p in held:
                count[p] += 1
    assert count == c._refs and sorted(c._free) == [p for p, r in enumerate(count) if not r]


def test_prefill_lays_pages_and_records(log):
    c = _cache()
    s = c.alloc()
    c.prefill(s, _prompt(32 + 70), _prompt(32 + 70))
    assert c.lens[s].tolist() == [16, 70, 0, 16] and c.table[s, :4].tolist() == [0, 1, 2, -1] and c.length(s) == 102
    _consistent(c)
    recs = log["append"]
    assert len(recs) == 4 and [r["n"].tolist() for r in recs] == [[32, 32, 6]] * 4
    assert recs[0]["first"].tolist() == [16, 48, 80] and recs[0]["t0"].tolist() == [0, 0, 0]
    assert (recs[3]["codes"] - c.codes[1, 1].data_ptr()).tolist() == [p * H * PAGE * D // 2 for p in (0, 1, 2)]
    assert (recs[2]["scales"] - c.scales[0, 1].data_ptr()).tolist() == [p * H * PAGE * D // 16 for p in (0, 1, 2)]
    assert recs[1]["gscale"].tolist() == [c.gscale.data_ptr() + 4 * (2 * 4 + s)] * 3


def test_steps_flush_full_windows_of_every_layer_and_side(log):
    c = _cache()
    a, b = c.alloc(), c.alloc()
    c.prefill(a, _prompt(32 + 24), _prompt(32 + 24))
    c.prefill(b, _prompt(32), _prompt(32))
    log["append"].clear()
    for i in range(16):
        st = c.step([b, a])
        for layer in range(2):
            x = torch.full((2, H, 1, D), 100.0 + i, dtype=torch.bfloat16)
            c.store(st, layer, x, -x)
    assert not log["append"] and c.lens[:2].tolist() == [[16, 24, 0, 32], [16, 0, 0, 32]]
    assert c.window[1, 1, a, 0, 16:, 0].tolist() == [-100.0 - i for i in range(16)]
    st = c.step([b, a], 3)
    (recs,) = log["append"]
    # sequence b: 16 rows to a new page; a: 8 rows end its first page, 8 begin the next; each for 2 layers x K, V
    assert recs["n"].tolist() == [16, 8, 8] * 4 and recs["t0"].tolist() == [0, 24, 0] * 4 and recs["first"].tolist() == [0, 0, 8] * 4
    assert (recs["k_bf16"].reshape(4, 3)[:, 1] - c.window.data_ptr()).tolist() == [(i * 4 + a) * H * 32 * D * 2 for i in range(4)]
    assert c.lens[:2].tolist() == [[16, 40, 16, 19], [16, 16, 16, 19]] and st.max_mid == 40
    c.store(st, 0, *(torch.full((2, H, 3, D), 7.0, dtype=torch.bfloat16),) * 2)
    assert c.window[0, 0, a, 1, :3, 5].tolist() == [7.0] * 3 and c.window[0, 0, a, 1, 3, 5] != 7.0
    _consistent(c)


def test_fork_shares_full_pages_and_copies_the_rest(log):
    c = _cache()
    a = c.alloc()
    c.prefill(a, _prompt(32 + 70, v=3.0), _prompt(32 + 70, v=9.0))
    c.codes[:, :, 2] = 77
    x, y = c.fork(a, 2)
    assert log["copies"] == [([2, 2], [3, 4]), ([a, a], [x, y])]
    assert c._refs[:5] == [3, 3, 1, 1, 1] and (c.codes[:, :, 3:5] == 77).all()
    assert c.table[x, :4].tolist() == [0, 1, 3, -1] and torch.equal(c.lens[x], c.lens[a])
    assert torch.equal(c.window[:, :, y], c.window[:, :, a]) and torch.equal(c.gscale[:, :, y], c.gscale[:, :, a])
    _consistent(c)
    c.free(a)
    assert c._refs[:5] == [2, 2, 0, 1, 1]
    _consistent(c)
    assert c.alloc() == a                           # a slot that was used starts empty again
    assert c.length(a) == 0
    # a sequence that ends on a page boundary shares everything
    c2 = _cache()
    b = c2.alloc()
    c2.prefill(b, _prompt(32 + 64), _prompt(32 + 64))
    (z,) = c2.fork(b)
    assert c2.table[z, :3].tolist() == [0, 1, -1] and c2.pages_free == 10
    for s in (b, z):
        for _ in range(17):
            c2.step([s])
    assert c2._held[b] == [0, 1, 2] and c2._held[z] == [0, 1, 3]    # each writes its own page
    _consistent(c2)


def test_compact_moves_pages_down(log):
    c = _cache()
    s = [c.alloc() for _ in range(3)]
    for i in s:
        c.prefill(i, _prompt(32 + 96), _prompt(32 + 96))
    (f,) = c.fork(s[2])
    for p in range(9):
        c.codes[:, :, p] = p
    c.free(s[0])
    c.free(s[1])
    assert c.compact() == 3 and c.compact() == 3
    assert log["copies"][-1] == ([6, 7, 8], [0, 1, 2]) and c._held[s[2]] == c._held[f] == [0, 1, 2]
    assert c.codes[0, 0, :3, 0, 0, 0].tolist() == [6, 7, 8] and c._refs[:3] == [2, 2, 2] and c.pages_free == 9
    _consistent(c)


def test_errors_change_nothing(log):
    c = _cache(pages=3)
    a = c.alloc()
    for T, kind in ((31, ValueError), (32 + 97, RuntimeError)):
        with pytest.raises(kind):
            c.prefill(a, _prompt(T), _prompt(T))
    with pytest.raises(ValueError):
        c.prefill(a, _prompt(40, 1), _prompt(40))
    with pytest.raises(ValueError):
        c.prefill(a, _prompt(40), _prompt(41))
    with pytest.raises(RuntimeError):
        c.step([a])                                                  # no prompt yet
    c.prefill(a, _prompt(32 + 80), _prompt(32 + 80))
    with pytest.raises(RuntimeError):
        c.prefill(a, _prompt(40), _prompt(40))
    log["append"].clear()
    for bad in ([a, a], [a, 3], [9]):
        with pytest.raises(ValueError):
            c.step(bad)
    for n in (0, 17):
        with pytest.raises(ValueError):
            c.step([a], n)
    with pytest.raises(RuntimeError):
        c.fork(a)                                                    # no page for its tail
    with pytest.raises(RuntimeError):
        c.fork(a, 9)
    for _ in range(32):
        c.step([a])                                                  # one flush fills the pool
    before = c._lens.copy()
    with pytest.raises(RuntimeError):
        c.step([a])
    assert (c._lens == before).all()
    _consistent(c)
    with pytest.raises(ValueError):
        c.free(2)
    with pytest.raises(IndexError):
        c.stores(2)
    for kw in (dict(page_tokens=24), dict(recent=0), dict(f_lo=-20, f_hi=20)):
        with pytest.raises(ValueError):
            kc.NVFP4PagedKVCache(1, 1, 1, 32, 4, device="cpu", **kw)
    c3 = _cache(max_tokens=40)
    b = c3.alloc()
    with pytest.raises(RuntimeError):
        c3.prefill(b, _prompt(32 + 65), _prompt(32 + 65))            # two columns of 32


def test_attend_refuses_caches_that_differ():
    a, b = (kc.NVFP4KVCache(1, 2, 32, capacity=64, device="cpu") for _ in range(2))
    q = torch.zeros(1, 2, 1, 32, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        kc.attend(q, a, b)
    a.n_window = 5
    with pytest.raises(ValueError):
        kc.attend(q, a, b)


def test_record_layout_matches_the_header():
    f = kc._KvAppendDesc
    assert [(n, kc._APPEND.fields[n][1]) for n in kc._APPEND.names] == [(n, getattr(f, n).offset) for n, _ in f._fields_]
    assert np.dtype(kc._APPEND).itemsize == 96
