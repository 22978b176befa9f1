"""The binding's own rules around the adapter and block-norm calls, on the host: what is checked before anything
is queued.  Stand-ins take the place of device tensors; nothing is launched."""
import types

import pytest
import torch


@pytest.fixture(scope="module")
def nq():
    from rank_binary_factorized_b200 import nq as mod
    return mod


def _adapters(nq, n=2, rank=8, d_in=64, d_out=96):
    """Adapters as the binding keeps them, without tensors behind the addresses."""
    ad = object.__new__(nq.Adapters)
    ad.n, ad.rank, ad.d_in, ad.d_out = n, rank, d_in, d_out
    ad.device = torch.device("cuda", 0)
    ad.struct = nq.nq_adapters(n, rank, d_in, d_out, 0x10000, d_in, 0x20000, rank, 0)
    ad._ref = nq.ctypes.byref(ad.struct)
    ad._ws = None
    return ad


def _groups(nq, M, n=2, device="cuda:0", rows=0x40000):
    g = object.__new__(nq.AdapterRows)
    g.rows = types.SimpleNamespace(device=torch.device(device))
    g.M, g.n, g._rows_ptr, g._offsets_ptr = M, n, rows, 0x50000
    return g


class Fake:
    """A device tensor's face: type, shape, device, address."""

    def __init__(self, shape, dtype=torch.bfloat16, at=0x60000, device=0):
        self.shape, self.dtype, self.at, self.device_index = torch.Size(shape), dtype, at, device

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def test_adapted_layer_checks_everything_before_the_projection_runs(nq, monkeypatch):
    ran = []
    monkeypatch.setattr(nq, "_forward", lambda *a, **k: ran.append("projection") or Fake((4, 96)))
    monkeypatch.setattr(nq, "adapter_forward", lambda *a, **k: ran.append("adapters"))
    monkeypatch.setattr(nq.Adapters, "workspace_bytes",
                        lambda self, M: nq.raw_lib().nq_adapter_workspace_bytes(self._ref, M))  # no device here
    layer = types.SimpleNamespace(d_in=64, d_out=96)
    ad, x = _adapters(nq), Fake((4, 64))
    nq.layer_forward(layer, x, adapters=ad, groups=_groups(nq, 4), t=Fake((4, 8), torch.float32))
    assert ran == ["projection", "adapters"]
    ran.clear()
    bad = [dict(groups=_groups(nq, 5)), dict(groups=_groups(nq, 4, n=3)), dict(groups=_groups(nq, 4, device="cuda:1")),
           dict(groups=_groups(nq, 4), t=Fake((4, 9), torch.float32)), dict(groups=_groups(nq, 4), t=Fake((4, 8))),
           dict(groups=_groups(nq, 4), t=Fake((4, 8), torch.float32, at=0x60004)),
           dict(groups=_groups(nq, 4, rows=0x40004)), dict(groups=_groups(nq, 4), y=Fake((5, 96))),
           dict(groups=_groups(nq, 4), y=Fake((4, 96), device=1)), dict(groups=_groups(nq, 4), adapters=_adapters(nq, rank=129)),
           dict(groups=_groups(nq, 4, n=16385), adapters=_adapters(nq, n=16385)), dict(groups=None)]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, nq.NQError)):
            nq.layer_forward(layer, x, **{"adapters": ad, **kw})
        assert not ran, kw


def test_workspace_sizes_are_those_of_the_tensors_device(nq, monkeypatch):
    """The size of a workspace goes by its device's multiprocessors, so the device of the tensors, not the
    current one, is asked."""
    current = [1]

    class on:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", on)
    asked = types.SimpleNamespace(nq_adapter_workspace_bytes=lambda S, M: 100 + current[0],
                                  nq_block_norm_workspace_bytes=lambda N, M: 200 + current[0])
    monkeypatch.setattr(nq, "_lib", asked)
    norm = nq.BlockNorm(64)
    assert norm.workspace_bytes(3) == 201  # no vectors: the current device
    norm.device = torch.device("cuda", 0)
    assert norm.workspace_bytes(3) == 200 and _adapters(nq).workspace_bytes(3) == 100
    assert current == [1]
    current[0] = 0
    assert norm.workspace_bytes(3) == 200 and _adapters(nq).workspace_bytes(3) == 100
