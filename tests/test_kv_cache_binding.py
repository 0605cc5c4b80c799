"""The binding of the 8-bit cache without a GPU."""
import pytest
import torch

import attention_backward_gb300 as ab


@pytest.mark.parametrize("device,want", [(None, torch.device("cuda")), (0, torch.device("cuda", 0)),
                                         (1, torch.device("cuda", 1)), ("cuda:0", torch.device("cuda", 0)),
                                         (torch.device("cuda", 0), torch.device("cuda", 0))])
def test_new_kv_cache_goes_to_the_device_asked_for(monkeypatch, device, want):
    """Device 0 by its number is not the current device."""
    zeros, asked = torch.zeros, []

    def on_the_host(*size, device, **kw):
        asked.append(torch.device(device))
        return zeros(*size, **kw)

    monkeypatch.setattr(torch, "zeros", on_the_host)
    k, v, ks, vs = ab.new_kv_cache(3, 16, 2, 64, device=device)
    assert asked == [want] * 4
    assert k.shape == v.shape == (3, 16, 2, 64) and k.stride(3) == 1 and ks.shape == vs.shape == (3, 2)
