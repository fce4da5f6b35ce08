"""Library calls that take scratch from the pool, captured into a CUDA graph."""
import pytest
import torch

from graph_transformer_sparse_kmip_b200 import binding
from graph_transformer_sparse_kmip_b200 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    yield torch.device("cuda:0")
    torch.cuda.synchronize()
    binding.kmip_scratch_trim()  # other tests measure what the pool holds


def test_attention_calls_can_be_captured(dev):
    """The library's scratch pool inside a capture (here through k-MIP
    attention, forward and both backwards)."""
    inp = wl.random_case([300, 45, 517], H=2, d=32, dtype="bf16", seed=12)
    g = {n: t.to(dev) for n, t in inp.items()}
    out, idx, lse = binding.attn_fwd(g["Q"], g["K"], g["V"], 15, 0.2, g["offsets"])
    want = binding.attn_bwd(g["dO"], g["Q"], g["K"], g["V"], idx, lse, 0.2, deterministic=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, i2, l2 = binding.attn_fwd(g["Q"], g["K"], g["V"], 15, 0.2, g["offsets"])
        got = binding.attn_bwd(g["dO"], g["Q"], g["K"], g["V"], i2, l2, 0.2, deterministic=True)
    graph.replay()
    torch.cuda.synchronize()
    binding.check_status()
    assert torch.equal(o2, out) and torch.equal(i2, idx)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
