"""The decode path's operators as a program uses them, for timing and comparison: attention over the NVFP4
K/V cache, copies of cache pages, and rotary positions.

``run`` computes an operator in plain torch (``own`` false) or calls this library's entry points (``own`` true).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SINK, RECENT = 16, 16                 # the cache's defaults: first tokens and a window of up to 2 * RECENT newest in BF16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # -- attention over the 4-bit cache --
        # the first tokens after a short prompt: one sequence, an odd length; latency
        dict(name="attend short", op="attend", B=1, H=8, G=4, Tq=1, D=128, tokens=301, ragged=False, page=0, tile=False,
             rotate=True, dtype="bf16"),
        # one user at the length of the K/V workload, a contiguous cache with the product's scale tiles
        dict(name="attend long single", op="attend", B=1, H=8, G=8, Tq=1, D=128, tokens=32768, ragged=False, page=0,
             tile=True, rotate=True, dtype="bf16"),
        # a serving batch: sequences of very different lengths over a shared pool of pages
        dict(name="attend ragged batch", op="attend", B=48, H=8, G=4, Tq=1, D=128, tokens=8191, ragged=True, page=64,
             tile=False, rotate=True, dtype="bf16"),
        # four draft tokens verified at once (causal among themselves), narrower heads, FP16
        dict(name="attend draft tokens", op="attend", B=8, H=4, G=4, Tq=4, D=64, tokens=4099, ragged=True, page=32,
             tile=False, rotate=True, dtype="f16"),
        # wide heads, all query heads on one K/V head
        dict(name="attend wide shared head", op="attend", B=16, H=1, G=16, Tq=1, D=256, tokens=12345, ragged=False, page=128,
             tile=False, rotate=False, dtype="bf16"),
        # a full batch of long conversations
        dict(name="attend large", op="attend", B=16, H=8, G=8, Tq=1, D=128, tokens=32768, ragged=False, page=64, tile=False,
             rotate=True, dtype="bf16"),
        # -- rotary positions --
        # one decode step's q and k of a batch
        dict(name="rope decode step", op="rope", B=48, T=1, Hq=32, Hk=8, D=128, rot=128, interleaved=False, dtype="bf16",
             far=8000, scaled=False, inverse=False, token_major=True),
        # a prompt of 8192 tokens at far positions with stretched frequencies, straight from the projection
        dict(name="rope prompt", op="rope", B=1, T=8192, Hq=32, Hk=8, D=128, rot=128, interleaved=False, dtype="bf16",
             far=120000, scaled=True, inverse=False, token_major=True),
        # the gradient's pass, neighbouring pairs in part of the head, an odd length, FP32
        dict(name="rope gradient", op="rope", B=2, T=2047, Hq=16, Hk=16, D=64, rot=32, interleaved=True, dtype="f32",
             far=0, scaled=False, inverse=True, token_major=False),
        # -- pages of the cache --
        # forking eight conversations: the half-filled last page of each, all layers, K and V
        dict(name="pages fork", op="pages", layers=8, H=8, D=128, page=64, pages=64, moves=8),
        # compaction: a third of a pool moves down
        dict(name="pages compact", op="pages", layers=16, H=8, D=128, page=64, pages=384, moves=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "rope", "pages"])
    if kind == "attend":
        D, H, G = rng.choice([64, 128, 256]), _log_int(rng, 1, 16), _log_int(rng, 1, 16)
        B, Tq = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
        most = 16 * 8 * 32768 * 128 // (D * B * H * (1 if G * Tq <= 8 else 2 * ((G * Tq + 15) // 16)))
        page = rng.choice([0, 16, 32, 64, 128])
        return dict(op="attend", B=B, H=H, G=G, Tq=Tq, D=D, tokens=_log_int(rng, Tq, max(Tq, min(32768, most))),
                    ragged=page > 0 and rng.random() < 0.7, page=page, tile=page == 0 and rng.random() < 0.5,
                    rotate=rng.random() < 0.7, dtype=rng.choice(["bf16", "f16"]))
    if kind == "rope":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([D, D, D // 2, D // 4 * 2])
        B, Hq, Hk = _log_int(rng, 1, 64), _log_int(rng, 1, 64), _log_int(rng, 1, 16)
        T = _log_int(rng, 1, max(1, min(16384, 8192 * 40 * 128 // (B * (Hq + Hk) * D))))
        dt = rng.choice(["bf16", "f16", "f32"])
        return dict(op="rope", B=B, T=T if dt != "f32" else max(1, T // 2), Hq=Hq, Hk=Hk, D=D, rot=rot,
                    interleaved=rng.random() < 0.5, dtype=dt, far=rng.choice([0, 1000, 120000, 1000000]),
                    scaled=rng.random() < 0.5, inverse=rng.random() < 0.3, token_major=rng.random() < 0.5)
    layers, H, D, page = _log_int(rng, 1, 16), _log_int(rng, 1, 8), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    item = layers * 2 * H * page * D * 9 // 16
    pages = _log_int(rng, 4, max(4, min(1000, 384 * 16 * 2 * 8 * 64 * 72 // item)))
    return dict(op="pages", layers=layers, H=H, D=D, page=page, pages=pages, moves=_log_int(rng, 1, max(1, pages // 3)))


# ---- what the cases say, in numbers ----
def _lengths(case):
    """(n_sink, n_mid, head, n_window) of every sequence: a cache of that many tokens after some decode steps."""
    rng, rows = random.Random(case["tokens"] * 64 + case["B"]), []
    for b in range(case["B"]):
        n = case["tokens"]
        if case["ragged"] and b:
            n = _log_int(rng, max(case["Tq"], n // 64, 1), n)
        sink = min(n, SINK)
        win = n - sink if n <= SINK + 2 * RECENT else RECENT + n % RECENT
        mid = n - sink - win
        rows.append((sink, mid, RECENT * (mid // RECENT % 2), win))
    return rows


def work(case):
    if case["op"] == "attend":
        D, H, rows = case["D"], case["H"], _lengths(case)
        es = 2
        mid, edge = sum(r[1] for r in rows), sum(r[0] + r[3] for r in rows)
        heads = case["B"] * H * case["G"] * case["Tq"]
        return {"bytes": H * (mid * 2 * (D // 2 + D // 16) + edge * 2 * 2 * D) + heads * (2 * D * es + 4),
                "flops": 4 * D * H * case["G"] * case["Tq"] * (mid + edge)}
    if case["op"] == "rope":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        es = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * case["D"] * es + 8 * case["B"] * case["T"], "flops": 3 * n * case["rot"]}
    item = case["layers"] * 2 * case["H"] * case["page"] * case["D"] * 9 // 16
    return {"bytes": 2 * item * case["moves"], "flops": 0}


# ---- inputs ----
def _hadamard():
    """H16 / 4: entry (i, j) has the sign of the parity of the bits that i and j share."""
    i = torch.arange(16, device=DEV)
    x = i[:, None] & i
    x = x ^ x >> 2
    return (1 - 2 * ((x ^ x >> 1) & 1)).float() / 4


def _to_nvfp4(x, g):
    """x [..., D] float32, g broadcast over the blocks: packed codes [..., D/2] and E4M3 scale bytes [..., D/16]."""
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / (6 * g)).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    y = b / (s.float() * g)[..., None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    c = torch.bucketize(y.abs(), mid).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
    c = c.flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], s.view(torch.uint8)


def _to_tiles(s, rows):
    """Scale bytes [N, rows, C] (C % 4 == 0) in tiles of 128 rows x 4 columns, rows padded with zero bytes."""
    n, _, c = s.shape
    s = torch.cat([s, s.new_zeros(n, -rows % 128, c)], 1)
    return s.view(n, -1, 4, 32, c // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1).contiguous()


def _cache(case, gen, rows):
    """One side (K or V) of a cache in the state its sequences have: BF16 ends, 4-bit middle, tensor scales."""
    B, H, D, page = case["B"], case["H"], case["D"], case["page"]
    most = max(r[1] for r in rows)
    bias = torch.randn(D, generator=gen, device=DEV) * (torch.arange(D, device=DEV) % 37 == 5)
    g = torch.rand(B, generator=gen, device=DEV) * 0.3e-3 + 1.8e-3                       # amax / 2688 of such tokens
    if not page:
        g = g[:1].expand(B).contiguous()                                                  # one scale for a contiguous cache
    ends = [(torch.randn(B, H, n, D, generator=gen, device=DEV) + bias).bfloat16() for n in (SINK, 2 * RECENT)]
    turn = _hadamard()
    per, n = (page, sum(-(-r[1] // page) for r in rows) + 3) if page else (most, B)
    table = None
    owner = torch.arange(n, device=DEV)
    if page:
        cols = max(-(-most // page), 1)
        order = torch.randperm(n, generator=gen, device=DEV)
        first = torch.tensor([0] + [-(-r[1] // page) for r in rows], device=DEV).cumsum(0)
        at = first[:-1, None] + torch.arange(cols, device=DEV)
        used = at < first[1:, None]
        table = torch.where(used, order[at.clamp(max=n - 1)], -1).to(torch.int32)
        owner = torch.zeros(n, dtype=torch.long, device=DEV)
        owner[table[used].long()] = torch.arange(B, device=DEV)[:, None].expand(-1, cols)[used]
    codes = torch.empty(n, H, per, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(n, H, per, D // 16, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // max(1, H * per * D))
    for i in range(0, n, step):
        x = torch.randn(codes[i:i + step].shape[:3] + (D,), generator=gen, device=DEV) + bias
        if case["rotate"]:
            x = (x.unflatten(-1, (-1, 16)) @ turn).flatten(-2)
        codes[i:i + step], scales[i:i + step] = _to_nvfp4(x, g[owner[i:i + step]][:, None, None, None])
    if case["tile"]:
        scales = _to_tiles(scales.view(n * H, per, D // 16), per)
    return dict(sink=ends[0], window=ends[1], codes=codes, scales=scales, gscale=g), table


def _frequencies(case):
    """Radians per position of each pair, in 64 bits; `scaled`: long wavelengths divided by 8, short ones kept, a ramp between."""
    half = case["rot"] // 2
    f = 10000.0 ** -(torch.arange(half, dtype=torch.float64, device=DEV) / half)
    if case["scaled"]:
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        f = f * (keep + (1 - keep) / 8)
    return f, (0.1 * math.log(8) + 1 if case["scaled"] else 1.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "attend":
        rows = _lengths(case)
        k, table = _cache(case, gen, rows)
        v, table_v = _cache(case, gen, rows)
        if table is not None:   # one page table for K and V: V's pages are put in K's places
            used = table >= 0
            for name in ("codes", "scales"):
                kept = v[name][table_v[used].long()]
                v[name][table[used].long()] = kept
        q = torch.randn(case["B"], case["Tq"], case["H"] * case["G"], case["D"], generator=gen, device=DEV)
        q = (1.5 * q).to(TYPES[case["dtype"]]).transpose(1, 2)                          # as a projection leaves it
        lens = torch.tensor(rows, dtype=torch.int32, device=DEV)
        return dict(case=case, q=q, k=k, v=v, table=table, lens=lens, host=rows[0], max_mid=max(r[1] for r in rows))
    if case["op"] == "rope":
        B, T, D, dt = case["B"], case["T"], case["D"], TYPES[case["dtype"]]
        xs = []
        for H in (case["Hq"], case["Hk"]):
            if case["token_major"]:
                xs.append(torch.randn(B, T, H, D, generator=gen, device=DEV).to(dt).transpose(1, 2))
            else:
                xs.append(torch.randn(B, H, T, D, generator=gen, device=DEV).to(dt))
        at = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=DEV) + torch.arange(T, device=DEV)
        f, m = _frequencies(case)
        return dict(case=case, xs=xs, at=at, freqs=f, mscale=m)
    L, H, D, page, n = (case[k] for k in ("layers", "H", "D", "page", "pages"))
    pool = [torch.randint(0, 256, (L, 2, n, H, page, D // w), dtype=torch.uint8, generator=gen, device=DEV) for w in (2, 16)]
    order = torch.randperm(n, generator=gen, device=DEV).tolist()
    m = case["moves"]
    return dict(case=case, pool=pool, src=order[:m], dst=order[m:2 * m])


# ---- the operators in plain torch ----
def _nvfp4(codes, scales, tile, g, rotate):
    """Values [N, H, rows, D] of packed codes and scale bytes, the rotation along D undone; g [N]."""
    n, H, rows, half = codes.shape
    if tile:
        c = half // 8
        scales = scales.view(n * H, -1, c // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n * H, -1, c)[:, :rows].reshape(n, H, rows, c)
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 16))
    x = x * (scales.view(torch.float8_e4m3fn).float() * g[:, None, None, None])[..., None]
    return (x @ _hadamard() if rotate else x).flatten(-2)


def _tokens(c, case, table, lens):
    """A cache side as [B, H, all rows, D] in the order sink | middle | window."""
    w = c["window"].shape[2]
    ring = (lens[:, 2:3] + torch.arange(w, device=lens.device)) % w
    window = c["window"].gather(2, ring[:, None, :, None].long().expand(-1, c["window"].shape[1], -1, case["D"]))
    codes, scales = c["codes"], c["scales"]
    if table is not None:
        at = table.clamp(min=0).long()
        codes = codes[at].transpose(1, 2).flatten(2, 3)
        scales = scales[at].transpose(1, 2).flatten(2, 3)
    mid = _nvfp4(codes, scales, case["tile"], c["gscale"], case["rotate"])
    return torch.cat([c["sink"].float(), mid, window.float()], 2)


def _attend(s):
    case, lens, q = s["case"], s["lens"], s["q"]
    k, v = (_tokens(s[n], case, s["table"], lens) for n in "kv")
    B, H, rows, D = k.shape
    i = torch.arange(rows, device=q.device)
    w = s["k"]["window"].shape[2]
    mid = rows - SINK - w
    part = torch.stack([(i < SINK), (i >= SINK) & (i < SINK + mid), i >= SINK + mid])
    local = torch.where(part[0], i, torch.where(part[1], i - SINK, i - SINK - mid))
    have, before = lens[:, [0, 1, 3]], torch.stack([lens[:, 0] * 0, lens[:, 0], lens[:, 0] + lens[:, 1]], 1)
    which = part.int().argmax(0)
    pos = before[:, which] + local
    there = local < have[:, which]
    last = have.sum(1)[:, None] - case["Tq"] + torch.arange(case["Tq"], device=q.device)
    seen = there[:, None, :] & (pos[:, None, :] <= last[:, :, None])                   # [B, Tq, rows]
    q = q.float().unflatten(1, (H, case["G"])).flatten(2, 3)                           # [B, H, G * Tq, D]
    x = (q @ k.transpose(2, 3)).unflatten(2, (case["G"], case["Tq"])) * D ** -0.5
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = ((p / total).flatten(2, 3) @ v).unflatten(2, (case["G"], case["Tq"])).flatten(1, 2)
    return out.to(s["q"].dtype), (top + torch.log(total))[..., 0].flatten(1, 2)


def _rope(s):
    case, out = s["case"], []
    angle = s["at"].double()[..., None] * s["freqs"]
    if case["inverse"]:
        angle = -angle
    c, n = ((f(angle) * s["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))  # [B, 1, T, rot / 2]

    def turn(x):
        y, rest = x[..., :case["rot"]].float(), x[..., case["rot"]:]
        a, b = (y[..., 0::2], y[..., 1::2]) if case["interleaved"] else y.chunk(2, -1)
        a, b = a * c - b * n, a * n + b * c
        y = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([y.to(x.dtype), rest], -1)

    return [turn(x) for x in s["xs"]]


def _pages(s):
    src, dst = (torch.tensor(s[n], device=DEV) for n in ("src", "dst"))

    def move(pool):
        pool[:, :, dst] = pool[:, :, src]
        return pool

    return [move(s["pool"][0]), move(s["pool"][1])]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attend": _attend, "rope": _rope, "pages": _pages}[op](s)
    import nvfp4_block_scaled_11_b200 as nv
    if op == "attend":
        if "stores" not in s:   # the cache's own views of its buffers, which a program keeps for the cache's life
            s["stores"] = [nv.KvStore(c["sink"], c["window"], c["codes"], c["scales"], c["gscale"], s["case"]["rotate"],
                                      s["case"]["tile"]) for c in (s["k"], s["v"])]
        k, v = s["stores"]
        if s["table"] is None:
            return nv.kv_attention(s["q"], k, v, s["host"], want_lse=True)
        return nv.kv_attention(s["q"], k, v, s["lens"], s["table"], max_mid=s["max_mid"], want_lse=True)
    if op == "rope":
        return nv.rope(s["xs"], s["at"], s["freqs"], interleaved=s["case"]["interleaved"], mscale=s["mscale"],
                       inverse=s["case"]["inverse"])
    nv.copy_pages([(s["pool"][0], 2), (s["pool"][1], 2)], s["src"], s["dst"])
    return s["pool"]


# ---- the operators from their definitions in 64 bits ----
def _exact_attend(case, s):
    """Sequence by sequence: the keys as stored, the query turned instead of the keys, the output turned back."""
    D, G, H, Tq = case["D"], case["G"], case["H"], case["Tq"]
    turn = torch.block_diag(*[_hadamard().double()] * (D // 16)) if case["rotate"] else torch.eye(D, device=DEV, dtype=torch.float64)
    e4m3 = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    outs, lses = [], []
    for b, (ns, nm, head, nw) in enumerate(_lengths(case)):
        ks, vs = [], []
        for c, into in ((s["k"], ks), (s["v"], vs)):
            if s["table"] is None:
                codes, sc, rows = c["codes"][b, :, :nm], c["scales"], torch.arange(nm, device=DEV)
                if case["tile"]:
                    cols, per = D // 16, c["codes"].shape[2]
                    tiles = -(-per // 128)
                    h, cc = torch.arange(H, device=DEV)[:, None, None], torch.arange(cols, device=DEV)
                    r = rows[None, :, None]
                    at = (((b * H + h) * tiles + r // 128) * (cols // 4) + cc // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + cc % 4
                    sc = sc[at]
                else:
                    sc = sc[b, :, :nm]
            else:
                p = s["table"][b, :-(-nm // case["page"])].long()
                codes, sc = (c[n][p].permute(1, 0, 2, 3).flatten(1, 2)[:, :nm] for n in ("codes", "scales"))
            nib = torch.stack([codes & 15, codes >> 4], -1).flatten(2).long()
            val = torch.where(nib >= 8, -e2m1[nib & 7], e2m1[nib & 7])
            into.append(val * e4m3[sc.long()].repeat_interleave(16, 2) * c["gscale"][b].double())
            w = c["window"].shape[2]
            ring = [(head + i) % w for i in range(nw)]
            into.append(torch.cat([c["sink"][b, :, :ns], c["window"][b][:, ring]], 1).double())
        q = s["q"][b].double().unflatten(0, (H, G)) * D ** -0.5                              # [H, G, Tq, D]
        place = [torch.arange(nm, device=DEV) + ns,
                 torch.cat([torch.arange(ns, device=DEV), torch.arange(nw, device=DEV) + ns + nm])]
        last = ns + nm + nw - Tq + torch.arange(Tq, device=DEV)
        x = torch.cat([torch.einsum("hgtd,hnd->hgtn", y, kk).masked_fill(pl > last[:, None], -math.inf)
                       for y, kk, pl in ((q @ turn, ks[0], place[0]), (q, ks[1], place[1]))], -1)
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[..., None])
        o = torch.einsum("hgtn,hnd->hgtd", p[..., :nm], vs[0]) @ turn + torch.einsum("hgtn,hnd->hgtd", p[..., nm:], vs[1])
        outs.append(o.flatten(0, 1))
        lses.append(lse.flatten(0, 1))
    return torch.stack(outs), torch.stack(lses)


def _exact_rope(case, s):
    """Each pair as a complex number, turned by exp(i angle) in 64 bits."""
    angle = s["at"][..., None] * s["freqs"]
    z = torch.polar(torch.full_like(angle, s["mscale"]), -angle if case["inverse"] else angle)[:, None]
    out, half = [], case["rot"] // 2
    for x in s["xs"]:
        y = x.double().clone()
        at = torch.arange(half, device=DEV)
        ia, ib = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
        w = torch.complex(y[..., ia], y[..., ib]) * z
        y[..., ia], y[..., ib] = w.real, w.imag
        out.append(y)
    return out


def exact(case, seed):
    if case["op"] == "pages":
        return None     # bytes are moved, nothing is computed
    s = prepare(case, seed)
    return _exact_attend(case, s) if case["op"] == "attend" else _exact_rope(case, s)
