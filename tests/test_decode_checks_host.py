"""Decode cache and its calls without a GPU: tensors on other devices, refused calls that change nothing.  Launches are
replaced by recorders; a `meta` tensor stands for one on another device."""
import pytest
import torch

import nvfp4_block_scaled_11_b200 as nv

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
