"""Arguments of the chunk and top-k calls that are refused on the host (CPU): buffers that overlap
what a call still reads, and buffers on another device."""
import ctypes

import pytest
import torch

from sampled_sparse_decode_gb300 import binding
from sampled_sparse_decode_gb300.binding import DecodeBuffers, SantaError


class _OnDevice(torch.Tensor):
    """A CPU tensor that claims to live on a CUDA device: what the checks look at."""
    index = 0
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index)


def on(t, index=0):
    t = t.as_subclass(_OnDevice)
    t.index = index
    return t


TOPK_FIELDS = ["out", "sel_ids", "sel_count", "pi", "workspace", "device_status"]


@pytest.mark.parametrize("field", TOPK_FIELDS)
def test_topk_buffers_of_another_device_are_refused(field, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    B, hq, hkv, d, T, k, P = 1, 4, 2, 64, 64, 3, 8
    i32 = torch.int32
    bufs = DecodeBuffers(
        out=on(torch.zeros(B, hq, d)), draw_ids=on(torch.zeros(B, hkv, k, dtype=i32)),
        sel_ids=on(torch.zeros(B, hkv, k, dtype=i32)), sel_count=on(torch.zeros(B, hkv, dtype=i32)),
        pi=on(torch.zeros(B, hkv, k)), team_probs=None,
        workspace=on(torch.zeros(256, dtype=torch.uint8)), device_status=on(torch.zeros(1, dtype=i32)))
    pool = on(torch.zeros(P, hkv, T, d))
    args = [on(torch.zeros(B, hq, d)), pool, pool, on(torch.zeros(P, hkv, d)),
            on(torch.zeros(B, P, dtype=i32)), on(torch.ones(B, dtype=i32)), k, bufs, None]
    setattr(bufs, field, on(getattr(bufs, field), 1))
    with pytest.raises(SantaError, match=field):
        binding._topk("santa_topk_decode", *args)
