"""The device argument of Boundary and Sublayer, without a GPU."""
import pytest
import torch

from mhc_residual_boundary_gb300 import boundary, sublayer


@pytest.fixture
def made(monkeypatch):
    """Device indices that handles were created on."""
    got = []

    def create(config, device):
        got.append(device)
        return None

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(boundary.capi, "mhc_boundary_create", create)
    monkeypatch.setattr(sublayer.capi, "mhc_sublayer_create", create)
    monkeypatch.setattr(sublayer.capi, "sublayer_calls",
                        lambda: dict.fromkeys(("add_rms_norm", "quantize", "swiglu", "matmul", "moe")))
    return got


MAKE = [lambda **kw: boundary.Boundary(hidden=64, tp=1, max_num_tokens=1, **kw), sublayer.Sublayer]


@pytest.mark.parametrize("make", MAKE)
@pytest.mark.parametrize("device,index", [(None, 3), ("cuda", 3), (torch.device("cuda"), 3), (0, 0), (2, 2),
                                          ("cuda:1", 1), (torch.device("cuda", 2), 2), (torch.device("cuda:0"), 0)])
def test_device(made, make, device, index):
    handle = make(device=device)
    assert made == [index] and handle.device == torch.device("cuda", index)
    assert make().device == torch.device("cuda", 3)


@pytest.mark.parametrize("make", MAKE)
@pytest.mark.parametrize("device,error", [("cpu", ValueError), (torch.device("cpu"), ValueError), ("meta", ValueError),
                                          (1.5, TypeError)])
def test_other_devices_are_refused(made, make, device, error):
    with pytest.raises(error):
        make(device=device)
    assert made == []
