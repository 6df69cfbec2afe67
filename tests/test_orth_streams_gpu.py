"""gemm_orthogonalize's own workspace is allocated on the stream the call runs
on, whichever way the stream is given."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["none", "default", "null handle", "stream", "handle"])
def test_workspace_is_allocated_on_the_calls_stream(how, monkeypatch):
    """Memory of another stream could be handed to that stream's next
    allocation while this call still works in it."""
    side = torch.cuda.Stream()
    stream, handle = {"none": (None, torch.cuda.current_stream().cuda_stream),
                      "default": (torch.cuda.default_stream(), 0), "null handle": (0, 0),
                      "stream": (side, side.cuda_stream), "handle": (side.cuda_stream, side.cuda_stream)}[how]
    M = 300
    G = torch.randn(M, M, device="cuda")
    want, O = (torch.empty(M, M, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dgt.check(dgt.orthogonalize(G, want))
    torch.cuda.synchronize()
    at = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty",
                        lambda *a, **k: (at.append(torch.cuda.current_stream().cuda_stream), empty(*a, **k))[1])
    dgt.check(dgt.orthogonalize(G, O, stream=stream))
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert at == [handle]
    assert torch.equal(O, want)
