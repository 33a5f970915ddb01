"""The attention bindings' own checks and caches, without a GPU."""
import pytest
import torch

import trellis_quantized_gb300 as tq


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int32, torch.int8])
def test_norm_weights_and_caches_are_fp16(dtype):
    """bfloat16 has fp16's width and other values: its bits must not be read as fp16."""
    w, ok = torch.ones(128, dtype=dtype), torch.zeros(2, 16, 8, 128, dtype=torch.float16)
    for kw in (dict(q_norm=w), dict(k_norm=w)):
        with pytest.raises(TypeError, match="_norm must be torch.float16"):
            tq.head_transform(**kw)
    bad = ok.to(dtype)
    with pytest.raises(TypeError, match="k must be torch.float16"):
        tq.kv_cache(bad, bad)


@pytest.mark.gpu
def test_cache_of_two_types_is_refused():
    k = torch.zeros(2, 16, 8, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError, match="v must be torch.float16"):
        tq.kv_cache(k, k.bfloat16())
    with pytest.raises(TypeError, match="q_norm must be torch.float16"):
        tq.head_transform(q_norm=torch.ones(128, dtype=torch.bfloat16, device="cuda"))
    tq.kv_cache(k.view(torch.int16), k.view(torch.int16))
    tq.head_transform(q_norm=torch.ones(128, dtype=torch.float16, device="cuda").view(torch.int16))


def test_workspace_sizes_are_kept_by_device(monkeypatch):
    """The size of a call's workspace goes by the device's number of SMs."""
    sms = {0: 152, 1: 76}
    current = [0]
    monkeypatch.setattr(tq, "exl3_paged_attention_workspace_size", lambda *shape: sms[current[0]] * 1024)
    tq._attention_workspace.cache_clear()
    try:
        for device in (0, 1, 0, 1):
            current[0] = device
            assert tq._attention_workspace(device, 1, 40, 8, 128, 1) == sms[device] * 1024
    finally:
        tq._attention_workspace.cache_clear()
