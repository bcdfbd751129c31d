"""Copies of cache pages, byte for byte: several arrays, odd item sizes and addresses, long lists, refusals."""
import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv

pytestmark = pytest.mark.gpu


def _fill(shape, dt, gen):
    return torch.randint(0, 120, shape, generator=gen).to(dt).cuda()


@pytest.mark.parametrize("shape,dim,dt", [((2, 2, 40, 3, 16, 64), 2, torch.uint8), ((40, 8, 64, 72), 0, torch.uint8),
                                          ((3, 40, 7), 1, torch.uint8), ((3, 40), 1, torch.float32), ((40,), 0, torch.uint8),
                                          ((2, 40, 5, 3), 1, torch.bfloat16), ((2, 40, 24), 1, torch.uint8),
                                          ((1, 40, 70001), 1, torch.uint8), ((5, 40, 16384 + 16), 1, torch.uint8)])
def test_pages_move_and_the_rest_stays(shape, dim, dt):
    gen = torch.Generator().manual_seed(len(shape) + shape[-1])
    a = _fill(shape, dt, gen)
    order = torch.randperm(40, generator=gen).tolist()
    src, dst = order[:13] + order[:1], order[13:27]                  # a source may go to two pages
    ref = a.clone()
    ref.index_copy_(dim, torch.tensor(dst, device="cuda"), a.index_select(dim, torch.tensor(src, device="cuda")))
    nv.copy_pages([(a, dim)], src, dst)
    assert torch.equal(a, ref)


def test_several_arrays_at_once_and_unaligned_bases():
    gen = torch.Generator().manual_seed(1)
    raw = _fill((4 * 10 * 48 + 64,), torch.uint8, gen)
    arrays = [(_fill((2, 10, 33), torch.uint8, gen), 1), (_fill((10, 2, 1000), torch.float32, gen), 0),
              (raw[16:16 + 1920].view(4, 10, 48), 1), (_fill((3, 10), torch.float32, gen), -1),
              (_fill((2, 10, 4096), torch.uint8, gen)[1:], 1), (_fill((0, 10, 8), torch.uint8, gen), 1)]
    refs = [t.clone() for t, _ in arrays]
    for r, (_, d) in zip(refs, arrays):
        r.index_copy_(d, torch.tensor([1, 9], device="cuda"), r.index_select(d, torch.tensor([4, 0], device="cuda")))
    before = raw.clone()
    nv.copy_pages(arrays, (4, 0), (1, 9))
    assert all(torch.equal(t, r) for (t, _), r in zip(arrays, refs))
    assert torch.equal(raw[:16], before[:16]) and torch.equal(raw[16 + 1920:], before[16 + 1920:])
    for shift in (1, 4, 16):
        r2 = raw.clone()
        v = raw[shift:shift + 1920].view(4, 10, 48)
        want = r2[shift:shift + 1920].view(4, 10, 48)
        want[:, 3] = want[:, 7].clone()
        nv.copy_pages([(v, 1)], [7], [3])
        assert torch.equal(raw, r2)


def test_more_pairs_than_one_launch():
    gen = torch.Generator().manual_seed(2)
    a, b = _fill((5000, 40), torch.uint8, gen), _fill((2, 5000, 16), torch.uint8, gen)
    order = torch.randperm(5000, generator=gen)
    src, dst = order[:2500], order[2500:]
    ra, rb = a.clone(), b.clone()
    ra[dst.cuda()] = a[src.cuda()]
    rb[:, dst.cuda()] = b[:, src.cuda()]
    nv.copy_pages([(a, 0), (b, 1)], src.tolist(), dst.tolist())
    assert torch.equal(a, ra) and torch.equal(b, rb)


def test_offsets_past_32_bits():
    a = torch.zeros(2, 70, 1 << 25, dtype=torch.uint8, device="cuda")   # 4.7 GB
    a[1, 69] = 7
    a[0, 69] = 5
    nv.copy_pages([(a, 1)], [69], [1])
    assert (a[0, 1] == 5).all() and (a[1, 1] == 7).all() and not a[:, 2:69].any() and not a[:, 0].any()


def test_captured_copy():
    a = torch.arange(64, device="cuda", dtype=torch.uint8).view(16, 4)
    nv.copy_pages([(a, 0)], [1], [2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.copy_pages([(a, 0)], [3, 4], [5, 6])
    a[3], a[4] = 101, 102
    g.replay()
    torch.cuda.synchronize()
    assert (a[5] == 101).all() and (a[6] == 102).all() and a[2].tolist() == a[1].tolist()


def test_refusals_move_nothing():
    a = torch.arange(80, device="cuda", dtype=torch.uint8).view(10, 8)
    ref = a.clone()
    for src, dst in (([0], [10]), ([10], [0]), ([-1], [0]), ([0, 1], [2, 2]), ([0, 1], [1, 2]), ([3], [3])):
        with pytest.raises(nv.NVFP4Error):
            nv.copy_pages([(a, 0)], src, dst)
    for arrays, src, dst, kind in (([(a, 0)], [0], [1, 2], ValueError), ([(a, 2)], [0], [1], ValueError),
                                   ([(a.cpu(), 0)], [0], [1], TypeError), ([(a.t(), 0)], [0], [1], ValueError),
                                   ([(a, 0), (a, 0)], [0], [1], ValueError), ([(a, 0)] * 17, [0], [1], ValueError)):
        with pytest.raises(kind):
            nv.copy_pages(arrays, src, dst)
    nv.copy_pages([], [0], [1])
    nv.copy_pages([(a, 0)], [], [])
    assert torch.equal(a, ref)
