"""What the binding of linear attention and the pages refuses besides the operands' shapes and types: it runs
no launch here."""

import pytest
import torch

from selective_state_space_53_b200 import m3


class Fake:
    """The attributes the binding's checks read, without memory behind them."""

    def __init__(self, *shape, dtype=torch.bfloat16, device="cuda:0", contiguous=True):
        self.shape, self.dtype, self.device, self._c = torch.Size(shape), dtype, torch.device(device), contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return 1 << 24


F32, I32 = dict(dtype=torch.float32), dict(dtype=torch.int32)
B, T, H, G, N, P = 2, 5, 4, 2, 16, 8


@pytest.fixture
def closed(monkeypatch):
    """A library that no call may reach."""
    monkeypatch.setattr(m3, "lib", lambda: pytest.fail("a refused call reached the library"))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)


def _prompt():
    return dict(q=Fake(B, T, G, N), k=Fake(B, T, G, N), v=Fake(B, T, H, P), log_decay=Fake(H, **F32),
                state=Fake(B, H, N, P, **F32), y=Fake(B, T, H, P))


@pytest.mark.parametrize("workspace", [
    Fake(1 << 20, dtype=torch.uint8, device="cpu"), Fake(1 << 20, dtype=torch.uint8, device="cuda:1"),
    Fake(1 << 20, dtype=torch.uint8, contiguous=False)], ids=["host", "other device", "expanded"])
def test_workspace_refused(closed, workspace):
    with pytest.raises(m3.M3Error) as e:
        m3.linattn(**_prompt(), workspace=workspace)
    assert e.value.code == -1 and "workspace" in str(e.value)
