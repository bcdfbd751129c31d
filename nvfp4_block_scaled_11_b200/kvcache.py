"""Attention-sink mixed-precision K/V cache that grows during decode.

"Search your block floating-point scales!" (gist.science summary of arXiv 2605.12464),
ScaleSearchAttention > attention-sink-aware mixed-precision caching: the first and the last block of
the KV cache stay in full precision and the blocks in between are NVFP4.  During decode the last block
moves: every new token enters a BF16 window of recent tokens, and once the window holds two groups of
`recent` tokens the older group is quantized (one `nvfp4_kv_append` launch, Hadamard-rotated along
head_dim when `rotate`) into the NVFP4 middle.  The window therefore always keeps between `recent` and
2 * recent - 1 of the newest tokens in BF16.

The tensor scale is fixed by the prefill (`nvfp4_kv_gscale` over the rotated middle tokens, as in
`nvfp4_kv_mixed`); later tokens use it unchanged, so values beyond 448 * 6 * g saturate.

`attend` reads a K and a V cache where they lie (nvfp4_kv_attention).  NVFP4PagedKVCache holds the K and V
caches of every layer for many sequences of different lengths over one pool of pages, which sequences that
were forked share.

Host-side bookkeeping only: token rows are moved with tensor copies, every quantization, attention and page
copy runs in the library's kernels.  The caches keep values, not gradients: rows that require them are detached, and
attention over a cache returns tensors without.
"""
from __future__ import annotations

import ctypes
import heapq

import numpy as np
import torch

from . import (KV_APPEND_BATCH_MAX, KvAppendBatch, KvStore, _KvAppendDesc, _launch, copy_pages, kv_append, kv_attention,
               kv_gscale, lib, sf_mma_bytes)


def _buffers(c) -> tuple:
    """Where a cache's buffers are: its KvStores are made anew when one has been replaced.  (A KvStore keeps what it reads
    alive, so a replacement never has the old one's address.)"""
    return c.sink.data_ptr(), c.window.data_ptr(), c.codes.data_ptr(), c.scales.data_ptr(), c.gscale.data_ptr(), c.rotate


class NVFP4KVCache:
    """K (or V) cache of B x H heads of dimension D (a multiple of 16; attention over it takes 64, 128 and 256) with room
    for `capacity` NVFP4 middle tokens.

    Attributes (device tensors):
      sink   [B, H, sink, D] bf16      first tokens, verbatim
      window [B, H, 2*recent, D] bf16  ring of the newest tokens; valid slots head .. head + n_window - 1
      codes  [B, H, capacity, D/2]     NVFP4 middle, rows 0 .. n_mid - 1 valid
      scales [B, H, capacity, D/16]    or the tensor-core tile layout of the B*H [capacity, D] matrices
      gscale [1] float32               tensor scale (fixed at prefill)
    """

    def __init__(self, B: int, H: int, D: int, capacity: int, sink: int = 16, recent: int = 16, rotate: bool = True,
                 f_lo: int = -2, f_hi: int = 6, tile_layout: bool = False, device="cuda"):
        if D % 16 or recent <= 0 or sink < 0 or capacity < 0:
            raise ValueError("D must be a multiple of 16; recent > 0; sink, capacity >= 0")
        self.B, self.H, self.D, self.capacity = B, H, D, capacity
        self.n_sink_max, self.recent, self.rotate, self.f_lo, self.f_hi = sink, recent, rotate, f_lo, f_hi
        self.tile_layout = tile_layout
        dev = torch.device(device)
        self.sink = torch.zeros((B, H, sink, D), dtype=torch.bfloat16, device=dev)
        self.window = torch.zeros((B, H, 2 * recent, D), dtype=torch.bfloat16, device=dev)
        self.codes = torch.zeros((B, H, capacity, D // 2), dtype=torch.uint8, device=dev)
        if tile_layout:
            self.scales = torch.zeros(max(sf_mma_bytes(capacity, D, B * H), 1), dtype=torch.uint8, device=dev)
        else:
            self.scales = torch.zeros((B, H, capacity, D // 16), dtype=torch.uint8, device=dev)
        self.gscale = torch.zeros(1, dtype=torch.float32, device=dev)
        self.n_sink = 0
        self.n_mid = 0
        self.head = 0        # first valid window slot: 0 or recent
        self.n_window = 0
        self.prefilled = False
        self._store = self._store_of = None

    def store(self) -> KvStore:
        """The cache as kv_attention reads it, made once for the buffers that the cache has now."""
        of = _buffers(self)
        if self._store_of != of:
            self._store = KvStore(self.sink, self.window, self.codes, self.scales, self.gscale, self.rotate, self.tile_layout)
            self._store_of = of
        return self._store

    @property
    def length(self) -> int:
        return self.n_sink + self.n_mid + self.n_window

    def prefill(self, k: torch.Tensor) -> None:
        """Start the cache from K[B, H, T, D] (BF16), T >= sink + recent: the tensor scale over the rotated
        middle (over the whole prompt when it has none), the middle quantized into rows
        0 .. T - sink - recent - 1, sink and window verbatim."""
        B, H, T, D = k.shape
        if (B, H, D) != (self.B, self.H, self.D) or k.dtype != torch.bfloat16:
            raise ValueError("k must be bfloat16 [B, H, T, D] matching the cache")
        s, r = self.n_sink_max, self.recent
        if T < s + r:
            raise ValueError("prefill needs at least sink + recent tokens")
        k = k.detach().contiguous()
        n_mid = T - s - r
        if n_mid > self.capacity:
            raise ValueError("prefill middle exceeds the cache capacity")
        # a prompt without a middle sets the scale by all of its tokens (0 would quantize every later one to 0)
        kv_gscale(k, s if n_mid else 0, r if n_mid else 0, self.rotate, out=self.gscale)
        if n_mid:
            kv_append(k, s, n_mid, self.gscale, self.codes, self.scales, 0, self.rotate, self.f_lo, self.f_hi,
                      self.tile_layout)
        self.sink.copy_(k[:, :, :s])
        self.window[:, :, :r].copy_(k[:, :, T - r:])
        self.n_sink, self.n_mid, self.head, self.n_window = s, n_mid, 0, r
        self.prefilled = True

    def append(self, k_new: torch.Tensor) -> None:
        """Append tokens K_new[B, H, n, D] (BF16) in order."""
        if not self.prefilled:
            raise RuntimeError("prefill first")
        for i in range(k_new.shape[2]):
            if self._full():
                kv_append(*self._flush_args()[:7], self.rotate, self.f_lo, self.f_hi, self.tile_layout)
                self._flushed()
            self._push(k_new[:, :, i])

    def _full(self) -> bool:
        return self.n_window == 2 * self.recent

    def _flush_args(self):
        """kv_append's arguments for the oldest `recent` window tokens (the contiguous slots head ..
        head + recent - 1) going to rows n_mid .. of the middle, as a kv_append_batch item."""
        r = self.recent
        if self.n_mid + r > self.capacity:
            raise RuntimeError("NVFP4 cache capacity exceeded")
        return (self.window, self.head, r, self.gscale, self.codes, self.scales, self.n_mid, self.rotate,
                self.tile_layout)

    def _flushed(self) -> None:
        r = self.recent
        self.n_mid += r
        self.head = (self.head + r) % (2 * r)
        self.n_window -= r

    def _push(self, token: torch.Tensor) -> None:
        slot = (self.head + self.n_window) % (2 * self.recent)
        self.window[:, :, slot].copy_(token.detach())
        self.n_window += 1

    def recent_tokens(self) -> torch.Tensor:
        """The BF16 window in token order, [B, H, n_window, D]."""
        idx = [(self.head + i) % (2 * self.recent) for i in range(self.n_window)]
        return self.window[:, :, idx]


class NVFP4KVCacheGroup:
    """Caches that advance together, e.g. the K and V caches of every layer of a model: append() steps all
    of them token by token, and whenever windows are full they flush together in one
    nvfp4_kv_append_batch launch per 64 caches, through descriptors prepared once (each flush only sets
    the rows).  The caches must share the ScaleSearch window [f_lo, f_hi] and one device; the result is the same as
    calling append on each cache."""

    def __init__(self, caches):
        self.caches = list(caches)
        if len({(c.f_lo, c.f_hi) for c in self.caches}) > 1:
            raise ValueError("caches in one group must share the offset window")
        if len({c.codes.device for c in self.caches}) > 1:
            raise ValueError("caches in one group must live on one device (each flush is one launch)")
        self._parts = []
        for j in range(0, len(self.caches), KV_APPEND_BATCH_MAX):
            part = self.caches[j:j + KV_APPEND_BATCH_MAX]
            batch = KvAppendBatch([(c.window, c.gscale, c.codes, c.scales, c.rotate, c.tile_layout) for c in part],
                                  part[0].f_lo, part[0].f_hi)
            self._parts.append((part, batch))

    def append(self, ks) -> None:
        """Append ks[i] [B, H, n, D] (BF16) to caches[i], the same n for every cache."""
        ks = list(ks)
        if len(ks) != len(self.caches):
            raise ValueError("one token tensor per cache")
        if not ks:
            return
        for c in self.caches:
            if not c.prefilled:
                raise RuntimeError("prefill first")
        n = ks[0].shape[2]
        if any(k.shape[2] != n for k in ks):
            raise ValueError("every cache receives the same number of tokens")
        for i in range(n):
            for part, batch in self._parts:
                full = [c._full() for c in part]
                if any(full):
                    for c, f in zip(part, full):
                        if f and c.n_mid + c.recent > c.capacity:
                            raise RuntimeError("NVFP4 cache capacity exceeded")
                    # full windows flush their oldest `recent` slots (head ..) into rows n_mid ..; others skip
                    batch([c.head for c in part], [c.recent if f else 0 for c, f in zip(part, full)],
                          [c.n_mid for c in part])
                    for c, f in zip(part, full):
                        if f:
                            c._flushed()
            for c, k in zip(self.caches, ks):
                c._push(k[:, :, i])


def append_many(caches, ks) -> None:
    """Append one decode step's new tokens to several caches at once (a one-off NVFP4KVCacheGroup; keep a
    group for a decode loop, so that its descriptors are prepared once)."""
    NVFP4KVCacheGroup(caches).append(ks)


def attend(q: torch.Tensor, k_cache: NVFP4KVCache, v_cache: NVFP4KVCache, causal: bool = True,
           scale: float | None = None, want_lse: bool = False, out: torch.Tensor | None = None):
    """Attention of the newest Tq tokens (already appended to both caches) over everything the caches hold: q
    [B, Hq, Tq, D] (BF16 or FP16, Hq a multiple of the caches' heads), kv_attention's output(s).  The lengths are the
    caches' at the call: one captured into a CUDA graph keeps them (give kv_attention lengths on the device, or use
    NVFP4PagedKVCache, where they change)."""
    a, b = ((c.n_sink, c.n_mid, c.head, c.n_window) for c in (k_cache, v_cache))
    if a != b:
        raise ValueError("the K and V caches hold different tokens")
    if not k_cache.prefilled or not v_cache.prefilled:
        raise RuntimeError("prefill first")
    if q.shape[0] != k_cache.B:
        raise ValueError("q must have the caches' batch")
    return kv_attention(q, k_cache.store(), v_cache.store(), a, causal=causal, scale=scale, want_lse=want_lse, out=out)


_MAX_MIDDLE = 2 ** 29 - 1      # tokens of a sequence's middle at most (nvfp4_kv_attention)

# nvfp4_kv_append_desc as a numpy record, so that a flush over many layers and sequences is filled column by column
_APPEND = np.dtype([("k_bf16", np.uint64), ("gscale", np.uint64), ("codes", np.uint64), ("scales", np.uint64),
                    *((n, np.int64) for n in ("BH", "T", "first", "n", "D", "cap", "t0")),
                    ("rotate", np.int32), ("scale_layout", np.int32)])
assert _APPEND.itemsize == ctypes.sizeof(_KvAppendDesc)


def _append_records(recs: np.ndarray, f_lo: int, f_hi: int, device: torch.device) -> None:
    """nvfp4_kv_append_batch over `recs` (dtype _APPEND), 64 to a launch."""
    fn = lib().nvfp4_kv_append_batch
    for j in range(0, len(recs), KV_APPEND_BATCH_MAX):
        part = recs[j:j + KV_APPEND_BATCH_MAX]
        _launch(device, fn, part.ctypes.data, len(part), f_lo, f_hi)


class DecodeStep:
    """n new tokens of some sequences of an NVFP4PagedKVCache, as `step` reserved them: `slots` (host), `slot_ids`
    (device int32 [B], not to be written) and where their rows go in the windows."""

    def __init__(self, slots, n, slot_ids, rows, at, max_mid):
        self.slots, self.n, self.slot_ids, self._rows, self._at, self.max_mid = slots, n, slot_ids, rows, at, max_mid


class NVFP4PagedKVCache:
    """K and V caches of `layers` layers for up to `slots` sequences, the NVFP4 middle in pages of `page_tokens`
    tokens from one pool (page p holds the same tokens of every layer, K and V).  A decode step:

        step = cache.step(slots)                     # once: room for the new tokens, windows flushed, lengths advanced
        for layer in range(layers):
            cache.store(step, layer, k, v)           # [B, H, n, D] BF16, rotary positions already applied
            o = cache.attend(step, layer, q)         # [B, Hq, n, D]

    D is a multiple of 16 to be filled, 64, 128 or 256 to be attended over.  Every sequence has its own tensor
    scales, fixed by its prefill and inherited by its forks.  Full pages of a forked sequence are shared (counted),
    its half-filled last page is copied, so a page with two owners is never written.  All calls of one cache belong
    on one stream.

    store and attend may be captured into a CUDA graph, for all layers or some.  A replay serves the captured step's
    sequences, in its order and with its n, as their lengths and pages are then: call step(slots, n) with those before each
    replay (the other calls keep books on the host and cannot be captured).

    Attributes (device tensors):
      codes  [layers, 2, pages, H, page_tokens, D/2]   scales [..., D/16]   (2: K, V)
      sink   [layers, 2, slots, H, sink, D] bf16       window [layers, 2, slots, H, 2*recent, D] bf16 ring
      gscale [layers, 2, slots] float32                table  [slots, cols] int32 (-1: none)
      lens   [slots, 4] int32: n_sink, n_mid, head, n_window
    """

    def __init__(self, layers: int, slots: int, H: int, D: int, pages: int, page_tokens: int = 64,
                 max_tokens: int | None = None, sink: int = 16, recent: int = 16, rotate: bool = True, f_lo: int = -2,
                 f_hi: int = 6, device="cuda"):
        if D % 16 or recent <= 0 or sink < 0 or min(layers, slots, H, pages) <= 0:
            raise ValueError("D must be a multiple of 16; recent, layers, slots, H, pages > 0; sink >= 0")
        if page_tokens <= 0 or page_tokens % 16:
            raise ValueError("page_tokens must be a multiple of 16")
        if f_hi - f_lo + 1 > 32:
            raise ValueError("the offset window holds at most 32 offsets")
        self.layers, self.n_slots, self.H, self.D, self.n_pages, self.page_tokens = layers, slots, H, D, pages, page_tokens
        self.n_sink_max, self.recent, self.rotate, self.f_lo, self.f_hi = sink, recent, rotate, f_lo, f_hi
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        # (attention counts positions in 32 bits: a table of more columns than a sequence can fill is refused there)
        cols = min(pages if max_tokens is None else max(-(-max_tokens // page_tokens), 1), pages, max(_MAX_MIDDLE // page_tokens, 1))
        z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
        self.codes, self.scales = (z(layers, 2, pages, H, page_tokens, D // w) for w in (2, 16))
        self.sink = z(layers, 2, slots, H, sink, D, dt=torch.bfloat16)
        self.window = z(layers, 2, slots, H, 2 * recent, D, dt=torch.bfloat16)
        self.gscale = z(layers, 2, slots, dt=torch.float32)
        self.lens = z(slots, 4, dt=torch.int32)
        self.table = torch.full((slots, cols), -1, dtype=torch.int32, device=dev)
        self._lens = np.zeros((slots, 4), np.int32)       # the host's copies; the device's follow in _publish
        self._table = np.full((slots, cols), -1, np.int32)
        self._held: list[list[int] | None] = [None] * slots   # pages of each sequence, None: the slot is free
        self._refs = [0] * pages
        self._free = list(range(pages))                    # a heap: the lowest page first
        self._stores: dict[int, tuple[KvStore, KvStore]] = {}
        self._stores_of = None
        self._capturing = torch.cuda.is_current_stream_capturing if dev.type == "cuda" else bool   # (bool() is False)
        self._captured: list[torch.Tensor] = []           # slot ids that CUDA graphs read, for the cache's life

    # ---- sequences ----
    @property
    def pages_free(self) -> int:
        return len(self._free)

    def length(self, slot: int) -> int:
        self._owned(slot)
        return int(self._lens[slot, 0] + self._lens[slot, 1] + self._lens[slot, 3])

    def alloc(self) -> int:
        """A free slot, now an empty sequence."""
        for s, held in enumerate(self._held):
            if held is None:
                self._held[s] = []
                return s
        raise RuntimeError("no free slot")

    def free(self, slot: int) -> None:
        """End a sequence: its slot and the pages that no other sequence shares are free again."""
        self._on_host("free")
        self._owned(slot)
        self._release(slot)
        self._held[slot] = None
        self._lens[slot] = 0
        self._publish([slot])

    def prefill(self, slot: int, ks, vs) -> None:
        """Start sequence `slot` (from alloc) from its prompt: ks[l], vs[l] [H, T, D] or [1, H, T, D] BF16, T >= sink +
        recent, rotary positions applied.  Tensor scales over the middle as NVFP4KVCache.prefill, per layer and side."""
        self._on_host("prefill")
        if self._owned(slot) or self._lens[slot].any():
            raise RuntimeError("the sequence has been started")
        sides = [[self._prompt(x) for x in xs] for xs in (ks, vs)]
        T = sides[0][0].shape[2] if sides[0] else 0
        if any(len(xs) != self.layers or any(x.shape[2] != T for x in xs) for xs in sides):
            raise ValueError("one K and one V tensor per layer, all of one length")
        s, r = self.n_sink_max, self.recent
        if T < s + r:
            raise ValueError("prefill needs at least sink + recent tokens")
        mid = T - s - r
        self._grow([(slot, mid)])
        try:
            for side, xs in enumerate(sides):
                for layer, x in enumerate(xs):
                    # a prompt without a middle sets the scale by all of its tokens (0 would quantize every later one to 0)
                    kv_gscale(x, s if mid else 0, r if mid else 0, self.rotate, out=self.gscale[layer, side, slot:slot + 1])
                    self.sink[layer, side, slot].copy_(x[0, :, :s])
                    self.window[layer, side, slot, :, :r].copy_(x[0, :, T - r:])
            P = self.page_tokens
            rows = [(slot, s + i * P, min(P, mid - i * P), p, 0) for i, p in enumerate(self._held[slot])]
            for side, xs in enumerate(sides):
                for layer, x in enumerate(xs):
                    if rows:
                        self._quantize(rows, layer, side, x.data_ptr(), 0, T)
        except BaseException:                      # the sequence stays empty and holds nothing
            self._release(slot)
            raise
        self._lens[slot] = (s, mid, 0, r)
        self._publish([slot])

    def fork(self, slot: int, n: int = 1) -> list[int]:
        """n new sequences that continue `slot`: its full pages are shared, the last page (when half filled) and the
        BF16 ends are copied, in one launch each."""
        self._on_host("fork")
        held = self._owned(slot)
        free = [s for s, h in enumerate(self._held) if h is None]
        if n < 0 or len(free) < n:
            raise RuntimeError("not enough free slots")
        new = free[:n]
        full = int(self._lens[slot, 1]) // self.page_tokens
        tail = held[full:]                                   # at most one page
        if len(tail) * n > len(self._free):
            raise RuntimeError("NVFP4 page pool exhausted")
        src, dst = [], []
        for s in new:
            self._held[s] = list(held[:full])
            for p in held[:full]:
                self._refs[p] += 1
            for p in tail:
                q = self._take()
                self._held[s].append(q)
                src.append(p)
                dst.append(q)
            self._lens[s] = self._lens[slot]
            self._table[s] = -1
            self._table[s, :len(self._held[s])] = self._held[s]
        if src:
            copy_pages([(self.codes, 2), (self.scales, 2)], src, dst)
        if new:
            ends = [(t, 2) for t in (self.sink, self.window, self.gscale) if t.numel()]
            copy_pages(ends, [slot] * n, new)
        self._publish(new)
        return new

    def compact(self) -> int:
        """Moves the pages in use to the front of the pool, in one launch; returns their number (the pages from there
        on hold nothing)."""
        self._on_host("compact")
        used = [p for p, r in enumerate(self._refs) if r]
        n = len(used)
        holes = [p for p in range(n) if not self._refs[p]]
        move = dict(zip((p for p in used if p >= n), holes))
        if move:
            copy_pages([(self.codes, 2), (self.scales, 2)], list(move), list(move.values()))
            for a, b in move.items():
                self._refs[b], self._refs[a] = self._refs[a], 0
            self._free = list(range(n, self.n_pages))
            changed = []
            for s, held in enumerate(self._held):
                if held and any(p in move for p in held):
                    held[:] = [move.get(p, p) for p in held]
                    self._table[s, :len(held)] = held
                    changed.append(s)
            self._publish(changed)
        return n

    # ---- decoding ----
    def step(self, slots, n: int = 1) -> DecodeStep:
        """Reserve n (at most `recent`) new tokens for each of the distinct sequences `slots`: windows without room flush
        their oldest `recent` tokens into pages (64 rows of one layer and side each per launch), and the lengths on the
        device count the new tokens from here on."""
        self._on_host("step")
        slots, r = [int(s) for s in slots], self.recent
        if len(set(slots)) != len(slots):
            raise ValueError("a sequence appears twice")
        if not 0 < n <= r:
            raise ValueError("a step holds 1 to `recent` tokens")
        for s in slots:
            self._owned(s)
            if not self._lens[s].any():
                raise RuntimeError("prefill first")
        full = [s for s in slots if self._lens[s, 3] + n > 2 * r]
        self._grow([(s, int(self._lens[s, 1]) + r) for s in full])
        rows, flushed, P = [], [], self.page_tokens
        for s in full:
            first, mid, left = int(self._lens[s, 2]), int(self._lens[s, 1]), r
            while left:                                      # a group may cross pages
                k = min(left, P - mid % P)
                rows.append((s, first, k, self._held[s][mid // P], mid % P))
                first, mid, left = first + k, mid + k, left - k
            flushed.append((self._lens[s, 0], mid, (self._lens[s, 2] + r) % (2 * r), self._lens[s, 3] - r))
        if rows:
            self._quantize(rows, None, None, self.window.data_ptr(), self.H * 2 * r * self.D * 2, 2 * r)
            self._lens[full] = flushed               # only now: a step that fails can be made again
        head = (self._lens[slots, 2] + self._lens[slots, 3]).astype(np.int64)
        self._lens[slots, 3] += n
        self._publish(slots)
        at = self._upload((head[:, None] + np.arange(n)) % (2 * r))
        ids = self._upload(np.array(slots, np.int32))
        return DecodeStep(slots, n, ids, ids.long()[:, None], at, int(self._lens[slots, 1].max()) if slots else 0)

    def store(self, step: DecodeStep, layer: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """Write the step's K and V rows [B, H, n, D] (BF16) of one layer into the windows (what attention reads of a layer
        is `stores(layer)`)."""
        shape = (len(step.slots), self.H, step.n, self.D)
        if not 0 <= layer < self.layers:
            raise IndexError("no such layer")
        for x in (k, v):                             # both before the first is written
            if x.shape != shape or x.dtype != torch.bfloat16 or x.device != self.device:
                raise ValueError(f"k and v must be bfloat16 {list(shape)} on {self.device}")
        rows, at = self._places(step) if self._capturing() else (step._rows, step._at)
        for side, x in enumerate((k, v)):
            self.window[layer, side][rows, :, at] = x.detach().transpose(1, 2)

    def _places(self, step: DecodeStep) -> tuple[torch.Tensor, torch.Tensor]:
        """Where a step's rows go, from the lengths on the device: a graph's replay follows those of its own step."""
        self._keep(step)
        ids = step.slot_ids.long()
        _, _, head, n_window = self.lens[ids].long()[:, :, None].unbind(1)
        at = (head + n_window - step.n + torch.arange(step.n, device=self.device)) % (2 * self.recent)
        return ids[:, None], at

    def attend(self, step: DecodeStep, layer: int, q: torch.Tensor, scale: float | None = None, causal: bool = True,
               want_lse: bool = False, out: torch.Tensor | None = None):
        """Attention of the step's tokens, q [B, Hq, n, D], over their sequences (kv_attention's output(s))."""
        k, v = self.stores(layer)
        if q.shape[0] != len(step.slots) or q.shape[2] != step.n:
            raise ValueError("q must be [B, Hq, n, D] of the step")
        if self._capturing():
            self._keep(step)
        return kv_attention(q, k, v, self.lens, self.table, step.slot_ids, causal, scale, step.max_mid, want_lse, out)

    def stores(self, layer: int) -> tuple[KvStore, KvStore]:
        """The layer's K and V as kv_attention reads them (with `lens` and `table`)."""
        of = _buffers(self)
        if self._stores_of != of:                    # buffers were replaced (or none was asked for yet)
            self._stores, self._stores_of = {}, of
        if layer not in self._stores:
            if not 0 <= layer < self.layers:
                raise IndexError("no such layer")
            self._stores[layer] = tuple(KvStore(self.sink[layer, i], self.window[layer, i], self.codes[layer, i],
                                                self.scales[layer, i], self.gscale[layer, i], self.rotate) for i in (0, 1))
        return self._stores[layer]

    # ---- bookkeeping ----
    def _keep(self, step: DecodeStep) -> None:
        """A captured step's slot ids outlive the step: the graph reads them at every replay."""
        if not any(t is step.slot_ids for t in self._captured):
            self._captured.append(step.slot_ids)

    def _on_host(self, name: str) -> None:
        if self._capturing():
            raise RuntimeError(f"{name} keeps books on the host: call it outside the capture, before each replay")

    def _owned(self, slot: int) -> list[int]:
        if not 0 <= slot < self.n_slots or self._held[slot] is None:
            raise ValueError(f"slot {slot} holds no sequence")
        return self._held[slot]

    def _prompt(self, x: torch.Tensor) -> torch.Tensor:
        if not isinstance(x, torch.Tensor):
            raise TypeError("prompts must be tensors")
        x = x[None] if x.dim() == 3 else x
        if x.dim() != 4 or x.shape[:2] != (1, self.H) or x.shape[3] != self.D or x.dtype != torch.bfloat16:
            raise ValueError("prompts must be bfloat16 [H, T, D] matching the cache")
        if x.device != self.device:                # its address goes to a kernel on the cache's device
            raise ValueError(f"a prompt is on {x.device}, the cache on {self.device}")
        return x.detach().contiguous()

    def _take(self) -> int:
        p = heapq.heappop(self._free)
        self._refs[p] = 1
        return p

    def _drop(self, p: int) -> None:
        self._refs[p] -= 1
        if not self._refs[p]:
            heapq.heappush(self._free, p)

    def _release(self, slot: int) -> None:
        """The sequence's pages back to the pool (those that no other one shares)."""
        for p in self._held[slot]:
            self._drop(p)
        self._held[slot].clear()
        self._table[slot] = -1

    def _grow(self, wants) -> None:
        """Pages for middles of the given tokens, all or none."""
        need = [(s, -(-mid // self.page_tokens)) for s, mid in wants]
        if any(n > self._table.shape[1] for _, n in need):
            raise RuntimeError("NVFP4 cache capacity exceeded")
        if sum(max(n - len(self._held[s]), 0) for s, n in need) > len(self._free):
            raise RuntimeError("NVFP4 page pool exhausted")
        for s, n in need:
            held = self._held[s]
            while len(held) < n:
                held.append(self._take())
                self._table[s, len(held) - 1] = held[-1]

    def _quantize(self, rows, layer, side, base: int, slot_bytes: int, T: int) -> None:
        """Rows (slot, first, n, page, t0): tokens [first, first + n) of the BF16 [H, T, D] buffer at base + slot *
        slot_bytes go to rows t0 .. of `page`, for one (layer, side), or for all of them (windows, laid out
        [layers, 2, slots, ...]) when layer is None."""
        slot, first, n, page, t0 = np.array(rows, np.int64).T
        pairs = np.arange(self.layers * 2) if layer is None else np.array([2 * layer + side])
        recs = np.zeros((len(pairs), len(rows)), _APPEND)
        lay = pairs[:, None]
        recs["k_bf16"] = base + (lay * self.n_slots + slot) * slot_bytes if layer is None else base
        recs["gscale"] = self.gscale.data_ptr() + 4 * (lay * self.n_slots + slot)
        at = (lay * self.n_pages + page) * self.H * self.page_tokens * self.D
        recs["codes"] = self.codes.data_ptr() + at // 2
        recs["scales"] = self.scales.data_ptr() + at // 16
        recs["BH"], recs["T"], recs["D"], recs["cap"], recs["rotate"] = self.H, T, self.D, self.page_tokens, int(self.rotate)
        recs["first"], recs["n"], recs["t0"] = first, n, t0
        _append_records(recs.reshape(-1), self.f_lo, self.f_hi, self.device)

    def _upload(self, a: np.ndarray) -> torch.Tensor:
        """A host array on the device without waiting for it: a fresh pinned buffer, kept until the copy is done."""
        t = torch.from_numpy(np.array(a))
        return t.pin_memory().to(self.device, non_blocking=True) if self.device.type == "cuda" else t.to(self.device)

    def _publish(self, slots) -> None:
        """The host's lengths and table rows of these sequences to the device."""
        if not slots:
            return
        at = self._upload(np.array(slots, np.int64))
        self.lens.index_copy_(0, at, self._upload(self._lens[slots]))
        self.table.index_copy_(0, at, self._upload(self._table[slots]))
