"""Argument validation of the decode entry points (attention over the cache, rotary positions, page copies), all decided
on the host before any CUDA work (fake device pointers, no GPU needed), and the host-side sizes."""
import ctypes
import random

import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv
from nvfp4_block_scaled_11_b200 import build as nvbuild

V = ctypes.c_void_p
OK, ARG, SIZE, ALIGN = 0, -1, -2, -3


@pytest.fixture(scope="module")
def L():
    nvbuild.build()
    return nv.lib()


def _desc(**kw):
    """A valid call on fake pointers; B = 0 unless given, so that a valid one returns before any launch."""
    store = dict(sink=0x10000, window=0x20000, codes=0x30000, scales=0x40000, gscale=0x50000, gscale_stride=0, rotate=1,
                 scale_layout=0)
    d = nv._KvAttentionDesc()
    base = dict(q=0x60000, out=0x70000, B=1, Hq=8, Hkv=2, Tq=1, D=128, slots=1, sink_rows=16, window_rows=32, pages=1, page_rows=64,
                table_cols=0, n_sink=16, n_mid=64, head=0, n_window=16, dtype=1, causal=1, scale=0.1)
    sides = {"k": dict(store), "v": dict(store)}
    for name, v in kw.items():
        if name[:2] in ("k_", "v_"):
            sides[name[0]][name[2:]] = v
        else:
            base[name] = v
    for name, v in base.items():
        setattr(d, name, v)
    for name, s in sides.items():
        setattr(d, name, nv._KvStore(*(s[f] for f, _ in nv._KvStore._fields_)))
    return d


def _call(L, splits=1, ws=None, wsb=0, **kw):
    return L.nvfp4_kv_attention(ctypes.byref(_desc(**kw)), splits, ws, wsb, None)


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(nv._KvStore) == 56 and ctypes.sizeof(nv._KvAttentionDesc) == 328
    assert nv._KvAttentionDesc.k.offset == 112 and nv._KvAttentionDesc.slots.offset == 224 and nv._KvAttentionDesc.slot.offset == 272
    assert ctypes.sizeof(nv._RopeTensor) == 72 and ctypes.sizeof(nv._PagesArray) == 40


def test_attention_sizes_and_arguments(L):
    assert L.nvfp4_kv_attention(None, 1, None, 0, None) == ARG
    for n in ("B", "Hq", "Tq"):                                      # nothing to do, whatever else
        assert _call(L, **{n: 0}) == OK
    for kw in (dict(D=96), dict(D=32), dict(B=-1), dict(Hq=7), dict(Hkv=0), dict(Tq=1 << 30), dict(B=2), dict(pages=0),
               dict(page_rows=1 << 30), dict(table=0x80000, table_cols=4, page_rows=24), dict(table=0x80000, table_cols=1 << 60),
               dict(table=0x80000, table_cols=4, page_rows=0), dict(pages=1 << 30, page_rows=64), dict(window_rows=1 << 30)):
        assert _call(L, **kw) == SIZE, kw
    for kw in (dict(dtype=0), dict(dtype=3), dict(causal=2), dict(q=None), dict(out=None), dict(n_sink=17), dict(n_mid=65),
               dict(n_mid=-1), dict(head=32), dict(n_window=33), dict(k_sink=None), dict(v_window=None), dict(k_codes=None),
               dict(v_scales=None), dict(k_gscale=None), dict(k_rotate=2), dict(v_scale_layout=-1), dict(k_gscale_stride=5)):
        assert _call(L, **kw) == ARG, kw
    for kw in (dict(q=0x60001), dict(out=0x70001), dict(lse=0x90002), dict(k_sink=0x10008), dict(v_window=0x20004), dict(k_codes=0x30008),
               dict(k_scales=0x40002), dict(v_gscale=0x50002), dict(table=0x80002, table_cols=1), dict(slot=0x80001), dict(lens=0x80002)):
        assert _call(L, **kw) == ALIGN, kw
    assert _call(L, splits=0) == ARG and _call(L, splits=65536) == ARG
    need = L.nvfp4_kv_attention_workspace_bytes(4, 128, 3)
    assert need == 3 * (2 * 8 * 130 * 4 + 16) and L.nvfp4_kv_attention_workspace_bytes(9, 64, 2) == 2 * (2 * 16 * 66 * 4 + 16)
    assert _call(L, splits=3) == ARG and _call(L, splits=3, ws=V(0xA0000), wsb=need - 1) == SIZE
    assert _call(L, splits=3, ws=V(0xA0008), wsb=need) == ALIGN
    for bad in ((4, 128, 1), (4, 128, 0), (0, 128, 4), (4, 0, 4), (4, 128, 70000)):
        assert L.nvfp4_kv_attention_workspace_bytes(*bad) == 0


def test_attention_splits(L):
    s = ctypes.c_int()
    f = L.nvfp4_kv_attention_splits
    assert f(1, 1, 1, 128, 0, None) == ARG
    for bad in ((-1, 1, 1, 128, 0), (1, 1, 1, 96, 0), (1, 1, 1, 128, -1), (1, 1, 1, 128, 1 << 40)):
        assert f(*bad, ctypes.byref(s)) == SIZE
    for args in ((0, 8, 4, 128, 100), (1, 8, 0, 128, 100)):
        assert f(*args, ctypes.byref(s)) == OK and s.value == 1
    assert f(1, 8, 4, 128, 300, ctypes.byref(s)) == OK and s.value == 8          # short: a part for each job
    assert f(1, 8, 4, 128, 1 << 20, ctypes.byref(s)) == OK and 148 <= s.value <= 65535
    assert f(4096, 64, 4, 128, 1 << 20, ctypes.byref(s)) == OK and s.value <= 1024


def test_rope_arguments(L):
    def call(x=0x10000, out=0x20000, heads=4, strides=(1024, 256, 64, 1024, 256, 64), n=1, B=1, T=4, D=64, rot=64, inter=0, dt=0,
             pos=0x30000, p64=1, freqs=0x40000, inv=0, tensors=True):
        t = (nv._RopeTensor * max(n, 1))(*[nv._RopeTensor(x, out, heads, *strides)] * max(n, 1))
        return L.nvfp4_rope(t if tensors else None, n, B, T, D, rot, inter, dt, pos, p64, 4, 1, freqs, 1.0, inv, None)
    assert call(n=0) == OK and call(heads=0) == OK and call(B=0) == OK and call(T=0) == OK
    for kw in (dict(n=9), dict(n=-1), dict(tensors=False), dict(dt=3), dict(inter=2), dict(p64=2), dict(inv=2), dict(x=None),
               dict(out=None), dict(pos=None), dict(freqs=None), dict(out=0x10000, strides=(1024, 256, 64, 1024, 64, 256))):
        assert call(**kw) == ARG, kw
    for kw in (dict(rot=66), dict(rot=-2), dict(rot=63), dict(D=2048, rot=1026), dict(T=-1), dict(heads=-1), dict(D=65, inter=1),
               dict(heads=1 << 30)):
        assert call(**kw) == SIZE, kw
    for kw in (dict(x=0x10002), dict(out=0x20001), dict(pos=0x30004), dict(freqs=0x40004)):
        assert call(**kw) == ALIGN, kw


def test_copy_pages_arguments(L):
    def call(src=(0,), dst=(1,), n=None, k=1, arr=True, **kw):
        d = dict(base=0x10000, outer=2, stride=800, item=80, pages=10) | kw
        a = (nv._PagesArray * max(k, 1))(*[nv._PagesArray(d["base"], d["outer"], d["stride"], d["item"], d["pages"])] * max(k, 1))
        s, t = ((ctypes.c_int32 * max(len(v), 1))(*v) for v in (src, dst))
        return L.nvfp4_copy_pages(a if arr else None, k, s, t, len(src) if n is None else n, None)
    assert call(n=0) == OK and call(k=0) == OK and call(outer=0) == OK and call(item=0, stride=0) == OK
    for kw in (dict(k=17), dict(k=-1), dict(arr=False), dict(base=None), dict(src=(10,)), dict(dst=(-1,)), dict(src=(3,), dst=(3,)),
               dict(src=(0, 1), dst=(2, 2)), dict(src=(0, 1, 2), dst=(5, 0, 6)), dict(src=tuple(range(5)) * 2, dst=tuple(range(4, 14)))):
        assert call(**kw) == ARG, kw
    for kw in (dict(n=-1), dict(stride=799), dict(item=-1), dict(pages=-1), dict(outer=1 << 40), dict(pages=1 << 40, item=1 << 40)):
        assert call(**kw) == SIZE, kw


def test_frequencies():
    """The stretched frequencies against their formulas at the ends: short wavelengths kept, long ones divided."""
    f0, m = nv.rope_frequencies(64, device="cpu")
    assert m == 1.0 and f0.dtype == torch.float64 and f0[0] == 1 and abs(f0[-1] - 10000.0 ** (-62 / 64)) < 1e-15
    f, _ = nv.rope_frequencies(64, scaling=dict(type="linear", factor=4), device="cpu")
    assert torch.equal(f, f0 / 4)
    f, _ = nv.rope_frequencies(64, scaling=dict(type="ntk", factor=4), device="cpu")
    assert f[0] == 1 and abs(f[-1] * 4 / f0[-1] - 1) < 1e-12
    for kind in ("yarn", "bands"):
        f, m = nv.rope_frequencies(64, scaling=dict(type=kind, factor=8, original=4096), device="cpu")
        assert f[0] == f0[0] and abs(f[-1] * 8 / f0[-1] - 1) < 1e-12 and ((f <= f0) & (f >= f0 / 8 * (1 - 1e-12))).all()
        assert (f[1:] < f[:-1]).all() and (m > 1.2) == (kind == "yarn")
    assert nv.rope_frequencies(0, device="cpu")[0].numel() == 0


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nv.KvStore(z, z, torch.zeros(1, 1, 16, 32, dtype=torch.uint8), torch.zeros(1, 1, 16, 4, dtype=torch.uint8), torch.zeros(1))
    with pytest.raises(TypeError):
        nv.kv_attention(z, None, None, (0, 0, 0, 0))
    with pytest.raises(TypeError):
        nv.rope(z, torch.arange(1), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        nv.copy_pages([(z, 0)], [0], [1])


def test_parts_of_the_work_cover_it():
    """The cut of the units into parts, as the kernel computes it: a partition, and every job's pieces found from the
    first cut inside it (a cut among a job's first units belongs to its beginning)."""
    J = 3

    class Parts:
        def __init__(self, total, most):
            self.n = min(most, max(total // 4, 1))
            self.base, self.rem = divmod(total, self.n)

        def start(self, c):
            return c * self.base + min(c, self.rem)

        def of(self, u):
            return u // (self.base + 1) if u < self.rem * (self.base + 1) else self.rem + (u - self.rem * (self.base + 1)) // self.base

    gen = torch.Generator().manual_seed(0)
    for _ in range(300):
        costs = [J + int(c) for c in torch.randint(1, 40, (int(torch.randint(1, 12, (1,), generator=gen)),), generator=gen)]
        total, most = sum(costs), int(torch.randint(1, 80, (1,), generator=gen))
        p = Parts(total, most)
        assert p.start(0) == 0 and p.start(p.n) == total
        assert all(p.start(p.of(u)) <= u < p.start(p.of(u) + 1) for u in range(total))
        starts, s = [], 0
        for c in costs:
            starts.append(s)
            s += c
        pieces = {j: [] for j in range(len(costs))}       # job -> (part, first, last) units of work
        for c in range(p.n):
            u, end = p.start(c), p.start(c + 1)
            j = max(i for i, st in enumerate(starts) if st <= u)
            while u < end:
                work = starts[j] + J
                if end <= work:
                    break
                units = costs[j] - J
                pieces[j].append((c, max(u - work, 0), min(units, end - work)))
                u, j = work + units, j + 1
        for j, got in pieces.items():
            units = costs[j] - J
            assert got[0][1] == 0 and got[-1][2] == units and all(a[2] == b[1] for a, b in zip(got, got[1:]))
            assert [g[0] for g in got] == list(range(got[0][0], got[0][0] + len(got)))
            if len(got) > 1:                               # the first cut inside the job names all its pieces
                cut = got[1][0]
                work = starts[j] + J
                assert work < p.start(cut) and p.start(cut - 1) <= work
                assert p.of(starts[j] + costs[j] - 1) - cut + 2 == len(got)
            for c, _, _ in got[2:]:
                assert p.start(c - 1) > starts[j] + J      # no later cut claims to be the first


def test_shared_elements_of_views_are_found_exactly():
    """Views of one buffer with the same strides against the sets of their elements."""
    rnd = random.Random(3)
    base = torch.arange(4 * 6 * 10 * 8).view(4, 6, 10, 8)
    seen = set()
    for _ in range(400):
        def view():
            s = [slice(a := rnd.randrange(n), rnd.randrange(a, n) + 1) for n in base.shape]
            return base[tuple(s)]
        a, b = view(), view()
        share = bool(set(a.flatten().tolist()) & set(b.flatten().tolist()))
        assert nv._overlap(a, b) == share and nv._overlap(b, a) == share
        seen.add(share)
    assert seen == {True, False}
    t = base.transpose(1, 2)
    assert nv._overlap(base[:, :2], t[:, :2]) and not nv._overlap(base[:2], t[2:])   # other strides: by their span
