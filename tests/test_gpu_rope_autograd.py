"""Gradients of rotary positions through autograd, against differences of the formula in 64 bits (the map is linear, so a
central difference is exact) and against the inverse call."""
import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv
from tests.test_gpu_rope import HALF, _ref

pytestmark = pytest.mark.gpu


def _freqs(rot=24):
    return nv.rope_frequencies(rot, scaling=dict(type="yarn", factor=4, original=64))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradient_against_differences(inter, inverse):
    g = torch.Generator().manual_seed(1)
    f, m = _freqs()
    pos = torch.tensor([3, 77, 1000])
    x, w = torch.randn(1, 2, 3, 32, generator=g), torch.randn(1, 2, 3, 32, generator=g)
    y = x.cuda().requires_grad_()
    out = nv.rope(y, pos.cuda(), f, inter, mscale=m, inverse=inverse)
    assert torch.equal(out.detach(), nv.rope(y.detach(), pos.cuda(), f, inter, mscale=m, inverse=inverse))
    (grad,) = torch.autograd.grad((out * w.cuda()).sum(), y)
    ref = lambda t: float((_ref(t, pos, f, inter, m, inverse)[0] * w.double()).sum())  # noqa: E731
    for i in range(0, x.numel(), 5):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[i] = 0.5
        d = ref(x.double() + e.view(x.shape)) - ref(x.double() - e.view(x.shape))
        # two products of FP32 sines (a few 2^-23 of mscale |w|, |w| < 4)
        assert abs(d - float(grad.flatten()[i])) <= 2.0 ** -19 * m * 8


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_several_tensors_of_one_projection(dt):
    """q and k as slices of one buffer that trains, v beside them: one gradient for the whole buffer."""
    g = torch.Generator().manual_seed(2)
    B, T, Hq, Hk, D = 2, 19, 6, 2, 64
    f, m = _freqs(32)
    pos = (torch.arange(T) + 100).cuda()
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * D, generator=g).to(dt).cuda().requires_grad_()
    view = lambda t, a, n: t[..., a * D:(a + n) * D].unflatten(-1, (n, D)).transpose(1, 2)  # noqa: E731
    wq, wk, wv = (torch.randn(B, n, T, D, generator=g).to(dt).cuda() for n in (Hq, Hk, Hk))
    q, k = nv.rope([view(qkv, 0, Hq), view(qkv, Hq, Hk)], pos, f, mscale=m)
    torch.autograd.backward([q, k, view(qkv, Hq + Hk, Hk)], [wq, wk, wv])
    got = qkv.grad
    for w, a, n in ((wq, 0, Hq), (wk, Hq, Hk)):
        y, mag = _ref(w, pos, f, False, m, True)
        # (below FP16's normal range a step is 2^-24: half of it is off whatever the value)
        assert ((view(got, a, n).cpu().double() - y).abs() <= mag * 2.0 ** -20 + HALF[dt] * (y.abs() + mag * 2.0 ** -20) + 2.0 ** -25).all()
    assert torch.equal(view(got, Hq + Hk, Hk), wv)


def test_gradients_that_autograd_hands_over():
    """Expanded ones (of a sum), ones along other strides, none for an output that is not used, inputs that need none,
    broadcast inputs, and the gradient's gradient."""
    g = torch.Generator().manual_seed(3)
    f, m = _freqs(16)
    pos = torch.arange(5).cuda() * 9
    inv = lambda t: nv.rope(t.contiguous(), pos, f, mscale=m, inverse=True)  # noqa: E731
    x, y = (torch.randn(2, 3, 5, 16, generator=g).cuda().requires_grad_() for _ in range(2))
    ones = torch.ones(2, 3, 5, 16, device="cuda")
    nv.rope(x, pos, f, mscale=m).sum().backward()
    assert torch.equal(x.grad, inv(ones))
    w = torch.randn(2, 3, 16, 5, generator=g).cuda()
    (got,) = torch.autograd.grad(nv.rope(x, pos, f, mscale=m).transpose(2, 3), x, w)
    assert torch.equal(got, inv(w.transpose(2, 3)))
    a, b = nv.rope([x, y], pos, f, mscale=m)
    gx, gy = torch.autograd.grad(a, [x, y], ones, allow_unused=True)
    assert torch.equal(gx, inv(ones)) and gy is None
    a, b = nv.rope([x.detach(), y], pos, f, mscale=m)
    (gy,) = torch.autograd.grad((a + b).sum(), y)
    assert torch.equal(gy, inv(ones))
    s = torch.randn(1, 1, 5, 16, generator=g).cuda().requires_grad_()
    nv.rope(s.expand(2, 3, 5, 16), pos, f, mscale=m).backward(ones)
    assert (s.grad - inv(ones).sum((0, 1), keepdim=True)).abs().max() <= 6 * 2.0 ** -22 * 3
    (gx,) = torch.autograd.grad((nv.rope(x, pos, f, mscale=m) ** 2).sum(), x, create_graph=True)
    (ggx,) = torch.autograd.grad(gx, x, ones)                         # d/dx of 2 R'R x is 2 R'R = 2 mscale^2 in the turned part
    want = torch.full((16,), 2 * m * m, device="cuda")
    assert (ggx - want).abs().max() <= 2.0 ** -18
    with torch.no_grad():
        assert not nv.rope(x, pos, f).requires_grad
    assert not nv.rope(x.detach(), pos, f).requires_grad


def test_gradients_that_would_be_lost_are_refused():
    f, _ = _freqs(16)
    pos, x = torch.arange(5).cuda(), torch.randn(2, 3, 5, 16, device="cuda", requires_grad=True)
    before = x.detach().clone()
    for kw in (dict(out=torch.empty(2, 3, 5, 16, device="cuda")), dict(out=x)):
        with pytest.raises(ValueError, match="gradient"):
            nv.rope(x, pos, f, **kw)
    with pytest.raises(ValueError, match="gradient"):
        nv.rope(before, pos, f, out=x)
    with pytest.raises(ValueError, match="gradient"):
        nv.rope(before, pos, f.clone().requires_grad_())
    assert torch.equal(x.detach(), before)
    with torch.no_grad():
        nv.rope(x, pos, f, out=x)
    assert torch.equal(x.detach(), nv.rope(before, pos, f))
    pos2 = pos.clone()
    out = nv.rope(x, pos2, f)
    pos2 += 1
    with pytest.raises(RuntimeError):                                 # positions changed before the gradient's pass
        out.sum().backward()
