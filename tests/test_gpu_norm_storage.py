"""What a norm that a program keeps holds in memory."""
import io

import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("count", [1, 300])
def test_a_norm_is_four_bytes(count):
    gq = gq_module()
    t = [torch.ones(1000, device="cuda") for _ in range(count)]
    norm = gq.gq_tensors_norm(t)
    assert norm.untyped_storage().nbytes() == 4
    few, f = io.BytesIO(), io.BytesIO()
    torch.save(torch.ones(1), few)
    torch.save(norm.cpu(), f)
    assert len(f.getvalue()) <= len(few.getvalue()) + 64


def test_norms_that_are_kept(monkeypatch):
    """A thousand of them: 512 bytes of the allocator's each, and what they hold stays what it was while others
    are computed, on two streams and in graphs."""
    gq = gq_module()
    t = [torch.full((100000,), 0.5, device="cuda"), torch.ones(7, device="cuda")]
    want = gq.gq_tensors_norm(t).item()
    before = torch.cuda.memory_allocated()
    kept = [gq.gq_tensors_norm(t) for _ in range(1000)]
    assert torch.cuda.memory_allocated() - before <= 1000 * 512
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    kept += [gq.gq_tensors_norm(t, stream=streams[k % 2]) for k in range(400)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept += [gq.gq_tensors_norm(t) for _ in range(5)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(n.item() == want for n in kept)
