"""Calls on a stream that is given (stream=): their results come from that
stream's memory, because the stream writes them without waiting for the
caller's, whose freed memory may still be in use there; and they are those of
the same call on the current stream."""
import pytest
import torch

from graph_transformer_sparse_kmip_b200 import binding
from graph_transformer_sparse_kmip_b200 import workloads as wl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    yield torch.device("cuda:0")
    torch.cuda.synchronize()
    binding.kmip_scratch_trim()  # other tests measure what the pool holds


def _owner(t):
    """The stream whose memory t lies in."""
    for segment in torch.cuda.memory_snapshot():
        if 0 <= t.data_ptr() - segment["address"] < segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not from torch's allocator")


def _calls(name, dev):
    """(call with a stream or None) -> results."""
    g = torch.Generator(device=dev).manual_seed(3)

    def n(*shape, dtype=BF):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    if name == "rotary":
        x, pos = n(600, 4, 32), n(600, 2, dtype=F32)
        freq = torch.ones(16, dtype=torch.float64, device=dev)
        axis = torch.arange(16, dtype=torch.int32, device=dev) % 2
        return lambda s: binding.rotary(x, pos, freq, axis, stream=s)
    if name.startswith("norm"):
        N = 70000 if name.endswith("large") else 600
        x, dy, w, b = n(N, 128), n(N, 128), n(128), n(128)
        stats = torch.zeros(1, 8, device=dev)
        if "fwd" in name:
            return lambda s: binding.group_norm_fwd(x, w, b, 8, act="silu", stream=s)
        return lambda s: binding.group_norm_bwd(dy, x, w, b, stats, stats + 1, 8, act="silu",
                                                stream=s)
    if name.startswith("ffn"):
        N = 5 if name.endswith("rows") else 600
        dtype = F32 if name.endswith("f32") else BF
        x, dy = n(N, 128, dtype=dtype), n(N, 128, dtype=dtype)
        wg, wu, wd = n(344, 128, dtype=dtype), n(344, 128, dtype=dtype), n(128, 344, dtype=dtype)
        if "fwd" in name:
            return lambda s: binding.ffn_fwd(x, wg, wu, wd, stream=s)
        return lambda s: binding.ffn_bwd(dy, x, wg, wu, wd, stream=s)
    q, k, v, do = (n(300, 2, 32) for _ in range(4))
    out, idx, lse = binding.attn_fwd(q, k, v, 5, 0.2)
    return {"attn_fwd": lambda s: binding.attn_fwd(q, k, v, 5, 0.2, stream=s),
            "attn_fwd_diag": lambda s: binding.attn_fwd_diag(q, k, v, 5, 0.2, stream=s),
            "attn_gather": lambda s: binding.attn_gather(q, k, v, idx, 0.2, stream=s),
            "attn_bwd": lambda s: binding.attn_bwd(do, q, k, v, idx, lse, 0.2, stream=s,
                                                   deterministic=True)}[name]


def _check(dev, call):
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        spare = torch.empty(1 << 24, device=dev)  # memory of this stream that a call could take
        del spare
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        side.synchronize()
        for a, c in zip(*(t if isinstance(t, tuple) else (t,) for t in (got, want))):
            assert _owner(a) == side.cuda_stream
            assert torch.equal(a, c)
        assert torch.cuda.current_stream() != side
    binding.check_status()


@pytest.mark.parametrize("name", ["rotary", "norm_fwd", "norm_bwd", "norm_fwd_large",
                                  "norm_bwd_large", "ffn_fwd", "ffn_fwd_rows", "ffn_fwd_f32",
                                  "ffn_bwd", "ffn_bwd_f32", "attn_fwd", "attn_fwd_diag",
                                  "attn_gather", "attn_bwd"])
def test_results_belong_to_the_stream_that_writes_them(dev, name):
    _check(dev, _calls(name, dev))


def test_a_given_out_and_a_refused_call_leave_the_current_stream(dev):
    x, pos = torch.randn((50, 2, 32), device=dev), torch.rand((50, 1), device=dev)
    freq = torch.ones(16, dtype=torch.float64, device=dev)
    axis = torch.zeros(16, dtype=torch.int32, device=dev)
    want = binding.rotary(x, pos, freq, axis)
    side, out = torch.cuda.Stream(), torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    assert binding.rotary(x, pos, freq, axis, out=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(ValueError, match="freq"):
        binding.rotary(x, pos, freq.float(), axis, stream=side)
    assert torch.cuda.current_stream() != side
