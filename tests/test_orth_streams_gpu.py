"""gemm_orthogonalize's own workspace lives on the stream the call runs on,
whichever way the stream is given."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt

pytestmark = pytest.mark.gpu


def segments(nbytes):
    return {s["address"]: s["stream"] for s in torch.cuda.memory_snapshot() if s["total_size"] >= nbytes}


@pytest.mark.parametrize("how", ["none", "default", "null handle", "stream", "handle"])
def test_workspace_is_allocated_on_the_calls_stream(how):
    """Memory of another stream could be handed to that stream's next
    allocation while this call still works in it."""
    side = torch.cuda.Stream()
    stream, handle = {"none": (None, torch.cuda.current_stream().cuda_stream),
                      "default": (torch.cuda.default_stream(), 0), "null handle": (0, 0),
                      "stream": (side, side.cuda_stream), "handle": (side.cuda_stream, side.cuda_stream)}[how]
    M = 3000  # a segment of its own
    need = dgt.gemm_orthogonalize_workspace_size(M, M, 1)
    G = torch.randn(M, M, device="cuda")
    want, O = (torch.empty(M, M, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dgt.check(dgt.orthogonalize(G, want))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = segments(need)
    dgt.check(dgt.orthogonalize(G, O, stream=stream))
    new = {a: s for a, s in segments(need).items() if a not in before}
    torch.cuda.synchronize()
    assert list(new.values()) == [handle]
    assert torch.equal(O, want)
