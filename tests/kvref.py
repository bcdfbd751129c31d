"""A mixed-precision K/V cache with random contents, and attention over it in 64 bits from the definition
(plain torch on the CPU), with a bound on what FP32 sums and the stated roundings may be off by."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E2M1 = torch.cat([E2M1, -E2M1])


def e4m3(b):
    return b.view(torch.float8_e4m3fn).double()


def hadamard16():
    h = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(4):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h / 4


def turn(x, m):
    """x [..., D] times m, block of 16 by block (a NaN stays in its block)."""
    return x if m is None else (x.unflatten(-1, (-1, 16)) @ m).flatten(-2)


def tile_scales(s):
    """[N, rows, C] scale bytes to the tile layout (128 rows x 4 block columns, zero padding)."""
    n, rows, c = s.shape
    out = torch.zeros(n, (rows + 127) // 128, (c + 3) // 4, 512, dtype=torch.uint8)
    r, j = torch.arange(rows)[:, None], torch.arange(c)[None, :]
    out[:, r // 128, j // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4] = s
    return out.flatten()


class Side:
    """K or V: slots x H heads, `pages` pages of `rows` rows (pages = slots for a contiguous cache)."""

    def __init__(self, gen, slots, H, D, sink, window, pages, rows, rotate=True, tile=False, per_slot=False, amp=1.0):
        r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.H, self.D, self.rotate, self.tile = H, D, rotate, tile
        self.sink, self.window = (amp * r(slots, H, sink, D)).bfloat16(), (amp * r(slots, H, window, D)).bfloat16()
        self.codes = torch.randint(0, 256, (pages, H, rows, D // 2), dtype=torch.uint8, generator=gen)
        # scales with the values of blocks whose largest element is a few times the tensor scale's unit
        self.scales = (64 * (1 + torch.rand(pages, H, rows, D // 16, generator=gen) * 2)).to(torch.float8_e4m3fn).view(torch.uint8)
        self.gscale = (amp * (0.5 + torch.rand(slots if per_slot else 1, generator=gen)) / 512).float()

    def store(self, nv, dev="cuda"):
        s = self.scales
        if self.tile:
            s = tile_scales(s.flatten(0, 1))
            if s.numel() == 0:
                s = torch.zeros(1, dtype=torch.uint8)
        return nv.KvStore(self.sink.to(dev), self.window.to(dev), self.codes.to(dev), s.to(dev), self.gscale.to(dev),
                          self.rotate, self.tile)

    def tokens(self, slot, lens, table):
        """(middle as stored [H, n_mid, D], its visibility [n_mid], sink, window in token order) in 64 bits."""
        ns, nm, head, nw = lens
        rows = self.codes.shape[2]
        if table is None:
            codes, scales, there = self.codes[slot, :, :nm], self.scales[slot, :, :nm], torch.ones(nm, dtype=torch.bool)
        else:
            pg = table[slot][torch.arange(nm) // rows].long()
            there = (pg >= 0) & (pg < self.codes.shape[0])
            at, r = pg.clamp(0, self.codes.shape[0] - 1), torch.arange(nm) % rows
            codes, scales = self.codes[at, :, r].transpose(0, 1), self.scales[at, :, r].transpose(0, 1)
        v = torch.stack([E2M1[(codes & 15).long()], E2M1[(codes >> 4).long()]], -1).flatten(2)
        g = self.gscale[slot if self.gscale.numel() > 1 else 0].double()
        mid = v * e4m3(scales.contiguous()).repeat_interleave(16, 2) * g
        w = self.window.shape[2]
        ring = [(head + i) % w for i in range(nw)]
        return mid, there, self.sink[slot, :, :ns].double(), self.window[slot][:, ring].double()


def attention(q, k, v, lens, table=None, slots=None, causal=True, scale=None):
    """(out, lse, out's and lse's error bounds before out's own rounding) for q [B, Hq, Tq, D] on the CPU; lens: a
    list of (n_sink, n_mid, head, n_window) per slot."""
    B, Hq, Tq, D = q.shape
    H = k.H
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    turn_k, turn_v = (hadamard16() if s.rotate else None for s in (k, v))
    abs_v = None if turn_v is None else turn_v.abs()
    out = torch.zeros(B, Hq, Tq, D, dtype=torch.float64)
    err, lerr = torch.zeros_like(out), torch.zeros(B, Hq, Tq, dtype=torch.float64)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64)
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < len(lens):
            continue
        ns, nm, head, nw = lens[s]
        L = ns + nm + nw
        km, there, ks, kw = k.tokens(s, lens[s], table)
        vm, _, vs, vw = v.tokens(s, lens[s], table)
        if L == 0:
            continue
        there = torch.cat([torch.ones(ns, dtype=torch.bool), there, torch.ones(nw, dtype=torch.bool)])
        for hq in range(Hq):
            h = hq // G
            for i in range(Tq):
                seen = there & (torch.arange(L) <= (L - Tq + i if causal else L))
                if not seen.any():
                    continue
                y = q[b, hq, i].double()
                yr = turn(y, turn_k)
                ke, ve = torch.cat([ks[h], kw[h]]), torch.cat([vs[h], vw[h]])
                x = scale * torch.cat([ks[h] @ y, km[h] @ yr, kw[h] @ y])
                x = x.masked_fill(~seen, -math.inf)
                m = torch.where(torch.isnan(x), -math.inf, x).max()
                p = torch.exp(x - m)
                l = p.sum()
                sel = seen
                pe, pm = torch.cat([p[:ns], p[ns + nm:]]), p[ns:ns + nm]
                se, sm = torch.cat([sel[:ns], sel[ns + nm:]]), sel[ns:ns + nm]
                o = (pe[se] @ ve[se] + turn(pm[sm] @ vm[h][sm], turn_v)) / l
                out[b, hq, i], lse[b, hq, i] = o, m + torch.log(l)
                # scores: D products summed in FP32 (the tensor cores may truncate: 2^-23 a step), the rotated query
                # within 2^-21 of its row's largest (two FP16 terms, FP32 butterflies), the factors' roundings
                mags = torch.cat([(ks[h].abs() @ y.abs()), km[h].abs() @ yr.abs() + 2 * yr.abs().max() * km[h].abs().sum(1),
                                  kw[h].abs() @ y.abs()])
                mags = torch.where(seen & torch.isfinite(mags), mags, 0.0)
                ds = float(abs(scale) * ((D / 16 + 8) * 2.0 ** -22 + 2.0 ** -16 * (q.dtype == torch.float32)) * mags.max()
                           + 2.0 ** -21 * x[seen].abs().max().nan_to_num(0, 0, 0)) + 2.0 ** -21
                sums = (L / 16 + 64) * 2.0 ** -22     # FP32 accumulation over the tokens and the joins
                mag_m = turn(pm[sm] @ vm[h][sm].abs(), abs_v) / l
                mag_e = pe[se] @ ve[se].abs() / l
                err[b, hq, i] = (mag_m + mag_e) * (2 * ds + sums) + mag_m * (2.0 ** -12 + 2.0 ** -20) + mag_e * 2.0 ** -16
                lerr[b, hq, i] = ds + sums + 2.0 ** -22 * abs(float(m))
    return out, lse, err, lerr


HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative to the value


def check(got, lse, ref):
    """out and lse of the kernel against attention()'s answer."""
    out, l, err, lerr = ref
    g = got.cpu().double()
    nan = torch.isnan(out)
    assert torch.equal(torch.isnan(g), nan), "NaN in other places"
    tol = err * 1.01 + HALF[got.dtype] * (out.abs() + err) + 2.0 ** -25   # FP16 below its normal range
    bad = ((g - out).abs() > tol) & ~nan
    assert not bad.any(), (int(bad.sum()), float(((g - out).abs() / tol)[~nan].max()), bad.nonzero()[:4].tolist())
    if lse is not None:
        s = lse.cpu().double()
        same = torch.isneginf(l) == torch.isneginf(s)
        assert same.all(), "rows without tokens differ"
        ok = torch.isneginf(l) | torch.isnan(l) | ((s - l).abs() <= lerr + 2.0 ** -23 * l.abs())
        assert ok.all(), float(((s - l).abs() / lerr)[~torch.isneginf(l)].max())
        assert torch.equal(torch.isnan(s), torch.isnan(l))
