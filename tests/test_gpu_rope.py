"""Rotary positions against the definition in 64 bits (each pair as a complex number), for both pair layouts, parts of
the head, strides, types, far positions, in place, and the inverse as the gradient."""
import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _ref(x, pos, freqs, inter, mscale=1.0, inverse=False):
    """(values, magnitude of each one's two terms) in 64 bits."""
    x = x.cpu().double()
    rot = 2 * freqs.numel()
    a = pos.cpu().double()[..., None] * freqs.cpu()
    if a.dim() == 3:
        a = a[:, None]
    z = torch.polar(torch.full_like(a, mscale), -a if inverse else a)
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    w = torch.complex(x[..., ia], x[..., ib]) * z
    y, mag = x.clone(), x.abs()
    y[..., ia], y[..., ib] = w.real, w.imag
    mag[..., ia] = mag[..., ib] = mscale * (x[..., ia].abs() + x[..., ib].abs())
    return y, mag


def _check(got, x, pos, freqs, inter, mscale=1.0, inverse=False):
    y, mag = _ref(x, pos, freqs, inter, mscale, inverse)
    # the angle's fraction of a turn is rounded to FP32 (2^-24 half turns and the FP64 product of far positions,
    # 2^-52 |angle|), sine and cosine are within 2 ulp, times mscale, two products, one sum; then the type's rounding
    far = float((pos.cpu().double().abs().max() * freqs.abs().max()) if freqs.numel() and pos.numel() else 0.0)
    tol = mag * (2.0 ** -22 + 2.0 ** -22 + 3 * 2.0 ** -24 + far * 2.0 ** -51) + HALF[x.dtype] * (y.abs() + mag * 2.0 ** -20) + 2.0 ** -26
    err = (got.cpu().double() - y).abs()
    assert (err <= tol).all(), float((err / tol).max())
    rot = 2 * freqs.numel()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,H,T,D,rot", [(1, 1, 1, 64, 64), (2, 3, 5, 128, 128), (1, 8, 129, 80, 40), (3, 5, 7, 96, 0),
                                         (2, 2, 33, 18, 6), (1, 40, 300, 256, 64), (1, 1, 2, 2050, 1024), (1, 2, 3, 2, 2)])
def test_layouts_types_and_sizes(dt, inter, B, H, T, D, rot):
    g = torch.Generator().manual_seed(D + rot + T)
    x = (3 * torch.randn(B, H, T, D, generator=g)).to(dt).cuda()
    pos = torch.randint(0, 5000, (B, T), generator=g).cuda()
    f, _ = nv.rope_frequencies(rot)
    _check(nv.rope(x, pos, f, inter), x, pos, f, inter)
    _check(nv.rope(x, pos.int(), f, inter, mscale=1.25, inverse=True), x, pos, f, inter, 1.25, True)


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions_and_scaled_frequencies(inter):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 2, 64, 128, generator=g).cuda()
    pos = torch.cat([torch.randint(0, 1 << 31, (62,), generator=g), torch.tensor([(1 << 31) - 1, -12345])])
    for s in (None, dict(type="linear", factor=8), dict(type="ntk", factor=8), dict(type="yarn", factor=16, original=4096),
              dict(type="bands", factor=8, original=8192)):
        f, m = nv.rope_frequencies(128, 500000.0, s)
        _check(nv.rope(x, pos.cuda(), f, inter, mscale=m), x, pos, f, inter, m)


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("inter", [False, True])
def test_slices_of_a_projection_in_place_and_together(pad, inter):
    """q and k as token-major slices of one buffer: into new tensors, and in place (v and the padding untouched)."""
    g = torch.Generator().manual_seed(2)
    B, T, Hq, Hk, D = 2, 19, 6, 2, 64
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * D + pad, generator=g).bfloat16().cuda()
    pos = (torch.arange(T) + 100).cuda()
    f, _ = nv.rope_frequencies(32)
    view = lambda t, a, n: t[..., a * D:(a + n) * D].unflatten(-1, (n, D)).transpose(1, 2)  # noqa: E731
    q, k = view(qkv, 0, Hq), view(qkv, Hq, Hk)
    rq, rk = nv.rope([q, k], pos, f, inter)
    _check(rq, q, pos, f, inter)
    _check(rk, k, pos, f, inter)
    assert rq.is_contiguous() and rk.shape == (B, Hk, T, D)
    other = qkv.clone()
    oq, ok = view(other, 0, Hq), view(other, Hq, Hk)
    nv.rope([oq, ok], pos, f, inter, out=[oq, ok])
    assert torch.equal(oq, rq) and torch.equal(ok, rk)
    assert torch.equal(other[..., (Hq + Hk) * D:], qkv[..., (Hq + Hk) * D:])


def test_inverse_is_the_gradient():
    """d/dx of <w, rope(x)> is rope(w, inverse): against the formula's own differences in 64 bits, and back and forth."""
    g = torch.Generator().manual_seed(3)
    f, m = nv.rope_frequencies(24, scaling=dict(type="yarn", factor=4, original=64))
    pos = torch.tensor([3, 77, 1000])
    x, w = torch.randn(1, 2, 3, 32, generator=g), torch.randn(1, 2, 3, 32, generator=g)
    for inter in (False, True):
        grad = nv.rope(w.cuda(), pos.cuda(), f, inter, mscale=m, inverse=True).cpu().double()
        ref = lambda t: float((_ref(t, pos, f, inter, m)[0] * w.double()).sum())  # noqa: E731
        for i in range(0, x.numel(), 7):
            e = torch.zeros(x.numel(), dtype=torch.float64)
            e[i] = 0.5                                # the map is linear: the central difference is exact
            e = e.view(x.shape)
            d = ref(x.double() + e) - ref(x.double() - e)
            assert abs(d - float(grad.flatten()[i])) < 1e-5
        y = nv.rope(nv.rope(x.cuda(), pos.cuda(), f, inter), pos.cuda(), f, inter, inverse=True)
        assert (y.cpu() - x).abs().max() < 1e-5


def test_three_dims_empty_calls_and_one_position_row():
    g = torch.Generator().manual_seed(4)
    f, _ = nv.rope_frequencies(16)
    x = torch.randn(4, 6, 16, generator=g).cuda()
    pos = torch.arange(6).cuda()
    assert torch.equal(nv.rope(x, pos, f), nv.rope(x[None], pos[None], f)[0])
    assert torch.equal(nv.rope(x, pos[None], f), nv.rope(x, pos, f))
    assert nv.rope(x[:, :0], pos[:0], f).shape == (4, 0, 16)
    assert nv.rope(x[:0], pos, f).shape == (0, 6, 16)
    a = torch.randn(1, 1, 6, 16, generator=g).cuda().expand(3, 4, 6, 16)     # broadcast input, own outputs
    assert torch.equal(nv.rope(a, pos, f), nv.rope(a.contiguous(), pos, f))


def test_many_heads_and_rows_cover_the_grid():
    g = torch.Generator().manual_seed(5)
    f, _ = nv.rope_frequencies(64)
    for B, H, T in ((1, 333, 3), (7, 2, 1000), (1, 1, 5000), (64, 33, 1)):
        x = torch.randn(B, H, T, 64, generator=g).bfloat16().cuda()
        pos = torch.randint(0, 9999, (B, T), generator=g).cuda()
        _check(nv.rope(x, pos, f), x, pos, f, False)


def test_captured_and_on_two_streams():
    f, _ = nv.rope_frequencies(64)
    x = torch.randn(2, 4, 8, 64, device="cuda")
    pos = torch.arange(8, device="cuda")
    out, s = torch.empty_like(x), torch.cuda.Stream()
    nv.rope(x, pos, f, out=out)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        nv.rope(x, pos, f, out=out)
    pos += 5
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        gr.replay()
        b = nv.rope(x, pos, f)
    c = nv.rope(x, pos, f)
    torch.cuda.synchronize()
    assert torch.equal(out, c) and torch.equal(b, c)


def test_refusals():
    f, _ = nv.rope_frequencies(16)
    x = torch.randn(2, 4, 8, 16, device="cuda")
    pos = torch.arange(8, device="cuda")
    for bad, kind in ((dict(x=x.cpu()), TypeError), (dict(x=x.double()), TypeError), (dict(pos=pos.float()), TypeError),
                      (dict(pos=pos[:7]), ValueError), (dict(f=f.float()), TypeError), (dict(x=x[..., :8]), ValueError),
                      (dict(x=x.transpose(2, 3)), ValueError), (dict(x=[x, x[:, :, :4]]), ValueError),
                      (dict(x=[x, x.bfloat16()]), ValueError), (dict(x=[]), ValueError), (dict(x=[x] * 9), ValueError),
                      (dict(x=x, out=x[:1].expand(2, 4, 8, 16)), ValueError), (dict(x=x, out=x[..., :8]), ValueError),
                      (dict(x=[x, x], out=[x, x]), ValueError), (dict(x=x[0, 0]), ValueError)):
        a = dict(x=x, pos=pos, f=f, out=None) | bad
        with pytest.raises(kind):
            nv.rope(a["x"], a["pos"], a["f"], out=a["out"])
    buf = torch.randn(2 * 4 * 8 * 16 + 16, device="cuda")
    n = x.numel()
    with pytest.raises(ValueError):                                  # shifted by one row
        nv.rope(buf[:n].view_as(x), pos, f, out=buf[16:].view_as(x))
    with pytest.raises(nv.NVFP4Error):
        nv.rope(torch.randn(1, 1, 8, 17, device="cuda"), pos, f, interleaved=True)   # one channel left over
    with pytest.raises(ValueError):
        nv.rope_frequencies(7)
    with pytest.raises(ValueError):
        nv.rope_frequencies(8, scaling=dict(type="other", factor=2))
    with pytest.raises(ValueError):
        nv.rope_frequencies(8, scaling=dict(type="yarn", factor=2))


def test_outputs_beside_their_inputs_and_shared_ones():
    """Rows of one buffer that lie side by side are told apart; a tensor written while another reads it is refused."""
    f, _ = nv.rope_frequencies(16)
    pos = torch.arange(8, device="cuda")
    buf = torch.randn(2, 8, 3 * 4 * 16, device="cuda").view(2, 8, 12, 16).transpose(1, 2)
    q, k, o = buf[:, :4], buf[:, 4:8], buf[:, 8:]
    want = nv.rope([q.clone(), k.clone()], pos, f)
    nv.rope(q, pos, f, out=o)
    assert torch.equal(o, want[0])
    nv.rope([q, k], pos, f, out=[q, k])
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    new = torch.empty(2, 4, 8, 16, device="cuda")
    for xs, outs in (([q, q], [q, new]), ([q, buf[:, 3:7]], [q, new]), ([q, k], [o, buf[:, 7:11]]), ([q, k], [new, new])):
        with pytest.raises(ValueError):
            nv.rope(xs, pos, f, out=outs)
