"""Edges of attention over the cache and of the calls around it: pools and batches without entries, the far end of a long
cache, layouts in combination, large batches, many query rows."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv
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
