"""What the tensor functions of the operators around the recurrence see to on the host: checks before any GPU work,
the device of a call, and the library's loading (CPU only)."""

import pytest
import torch

from hybrid_linear_attention_prefill_gb300 import build as B
from hybrid_linear_attention_prefill_gb300 import gdn


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return gdn.load()


class Entries:
    """Stands in for the library: notes the calls of its entries and returns 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append(name)
            return 0
        return entry


@pytest.fixture
def entries(monkeypatch):
    e = Entries()
    monkeypatch.setattr(gdn, "load", lambda *a: e)
    monkeypatch.setattr(gdn, "_fast", None)
    monkeypatch.setattr(gdn, "_raw_stream", lambda *a: 0)
    return e


def scan_operands(n=8):
    z, bf = torch.zeros, torch.bfloat16
    return dict(x=z(n, 4, 64, dtype=bf), dt=z(n, 4), A=z(4), Bm=z(n, 2, 32, dtype=bf), Cm=z(n, 2, 32, dtype=bf))


@pytest.mark.parametrize("workspace", [
    torch.zeros(4096, dtype=torch.uint8)[::2],          # strided: its bytes are not in one piece
    torch.zeros(64, 64, dtype=torch.uint8).t(),
    torch.zeros(4096, dtype=torch.uint8, device="meta")])  # on another device than x
def test_scan_refuses_a_workspace_that_is_not_one_piece_beside_x(entries, workspace):
    with pytest.raises(ValueError, match="workspace"):
        gdn.ssm_scan(**scan_operands(), workspace=workspace)
    assert entries.calls == []
    gdn.ssm_scan(**scan_operands(), workspace=torch.zeros(4096, dtype=torch.uint8))
    assert entries.calls == ["gdn_ssm_scan"]
