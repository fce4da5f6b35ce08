"""The operators around the attention through torch autograd, alone and run
together as a GraphTransformerLayer, against fp64 on the CPU.

The layer's reference applies the same parameters in fp64 and takes the
attention over the GPU-selected key sets from the oracle, so every gradient is
compared through the whole layer.  The tolerance is the attention block's, 2e-2
of the largest entry for bf16: five half steps of 2^-8, where the layer rounds
to bf16 some eight times in a row and independent roundings add as the root of
their number (2.9 half steps)."""
import math

import pytest
import torch

import oracle
from graph_transformer_sparse_kmip_b200 import binding
from graph_transformer_sparse_kmip_b200 import workloads as wl
from graph_transformer_sparse_kmip_b200.layer import (AxisRotary, GatedFeedForward,
                                                      GraphGroupNorm, GraphTransformerLayer,
                                                      KmipGlobalAttention)
from parity import check_values
from test_gpu_layer import _OracleAttention

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


def _norm64(x, w, b, offsets, groups, eps):
    out = []
    for part in x.split(offsets.diff().tolist()):
        p = part.unflatten(1, (groups, -1))
        if len(p):
            m = p.mean((0, 2), keepdim=True)
            v = (p - m).square().mean((0, 2), keepdim=True)
            p = (p - m) * (v + eps) ** -0.5
        out.append(p.flatten(1))
    return torch.cat(out) * w + b


def _turn64(x, pos, rotary):
    ang = pos.double()[:, rotary._axis] * torch.tensor(rotary._freq, dtype=torch.float64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    P = ang.shape[1]
    u, v = x[..., :P], x[..., P:2 * P]
    return torch.cat([u * c - v * s, u * s + v * c, x[..., 2 * P:]], -1)


@pytest.mark.parametrize("axes", [0, 2, 3])
def test_layer_matches_fp64(dev, axes):
    sizes, hidden, heads, k, width, groups = [300, 45, 0, 517, 129], 128, 4, 15, 344, 8
    d, N = hidden // heads, sum(sizes)
    gen = torch.Generator().manual_seed(40 + axes)
    offsets = wl.offsets_from_sizes(sizes)
    torch.manual_seed(3)
    layer = GraphTransformerLayer(hidden, heads, k, width, groups, axes=axes, device=dev)
    with torch.no_grad():
        for norm in (layer.norm1, layer.norm2):
            norm.weight += 0.2 * torch.randn_like(norm.weight)
            norm.bias += 0.2 * torch.randn_like(norm.bias)
    x = torch.randn((N, hidden), generator=gen).to(BF).to(dev).requires_grad_(True)
    gy = torch.randn((N, hidden), generator=gen).to(BF).to(dev)
    pos = (torch.rand((N, axes), generator=gen) * 4).to(dev) if axes else None
    y = layer(x, offsets.to(dev), pos)
    y.backward(gy)
    torch.cuda.synchronize()
    binding.check_status()

    P = {n: p.detach().cpu().double().requires_grad_(True) for n, p in layer.named_parameters()}
    x64 = x.detach().cpu().double().requires_grad_(True)
    h = _norm64(x64, P["norm1.weight"], P["norm1.bias"], offsets, groups, 1e-5)
    qkv = (h @ P["attn.qkv.weight"].T + P["attn.qkv.bias"]).view(N, 3, heads, d)
    q, kk = qkv[:, 0], qkv[:, 1]
    if axes:
        q, kk = (_turn64(t, pos.cpu(), layer.attn.rotary) for t in (q, kk))
    a = _OracleAttention.apply(q.contiguous(), kk.contiguous(), qkv[:, 2].contiguous(),
                               layer.attn.last_idx.cpu().numpy(), offsets.numpy(),
                               1.0 / math.sqrt(d))
    z = x64 + a.reshape(N, hidden) @ P["attn.proj.weight"].T + P["attn.proj.bias"]
    m = _norm64(z, P["norm2.weight"], P["norm2.bias"], offsets, groups, 1e-5)
    g = torch.nn.functional.silu(m @ P["ffn.gate"].T) * (m @ P["ffn.up"].T)
    y64 = z + g @ P["ffn.down"].T
    y64.backward(gy.cpu().double())

    check_values("y", y, y64.detach(), BF)
    check_values("dx", x.grad, x64.grad, BF)
    for n, p in layer.named_parameters():
        got, ref = p.grad, P[n].grad
        if got.dim() == 1:
            got, ref = got[None], ref[None]
        check_values("d" + n, got, ref, BF)


def test_gradients_match_differences(dev):
    """fp32 modules against central differences of the fp64-summed loss: step
    h = 2^-6 gives a difference quotient that is off by h^2 / 6 of the third
    derivative (under 1e-3 of the gradient's size here) and by the forward's
    fp32 error over h (2^-22 * 64)."""
    torch.manual_seed(1)
    x = torch.randn(40, 32, device=dev)
    offsets = torch.tensor([0, 25, 40], dtype=torch.int32, device=dev)
    pos = torch.rand(40, 2, device=dev)
    rot = AxisRotary(16, 2, interleaved=True)
    cases = [(GraphGroupNorm(32, 4, act="silu", dtype=F32, device=dev), (offsets,)),
             (GatedFeedForward(32, 48, dtype=F32, device=dev), ()),
             (lambda t, p: rot(t.view(40, 2, 16), p).reshape(40, 32), (pos,))]
    for f, extra in cases:
        w = torch.randn(40, 32, device=dev)
        leaf = x.clone().requires_grad_(True)
        (f(leaf, *extra) * w).sum().backward()
        step = 2.0 ** -6
        for i, j in ((0, 0), (7, 31), (24, 16), (39, 5)):
            vals = []
            for sgn in (1, -1):
                t = x.clone()
                t[i, j] += sgn * step
                vals.append((f(t, *extra).double() * w.double()).sum())
            quotient = ((vals[0] - vals[1]) / (2 * step)).item()
            assert abs(quotient - leaf.grad[i, j].item()) <= 5e-3 * max(
                1.0, leaf.grad.abs().max().item())


def test_strided_and_expanded_gradients(dev):
    """Gradients that arrive transposed or broadcast."""
    rot = AxisRotary(32, 2)
    pos = torch.rand(50, 2, device=dev)
    x = torch.randn(50, 4, 32, device=dev, requires_grad=True)
    rot(x, pos).transpose(1, 2).sum(1).sum().backward()
    g1 = x.grad.clone()
    x.grad = None
    y = rot(x, pos)
    y.backward(torch.ones(1, 1, 1, device=dev).expand(50, 4, 32))
    assert torch.equal(g1, x.grad)
    ffn = GatedFeedForward(32, 64, dtype=F32, device=dev)
    norm = GraphGroupNorm(32, 4, dtype=F32, device=dev)
    z = torch.randn(32, 50, device=dev, requires_grad=True)
    ffn(norm(z.t())).sum().backward()       # x itself transposed
    assert z.grad.shape == (32, 50) and torch.isfinite(z.grad).all()


def test_refusals(dev):
    with pytest.raises(ValueError, match="multiple"):
        GraphGroupNorm(30, 4)
    with pytest.raises(ValueError, match="multiples of 8"):
        GatedFeedForward(36, 64)
    with pytest.raises(ValueError, match="activation"):
        GatedFeedForward(32, 64, act="tanh")
    with pytest.raises(ValueError, match="sections"):
        AxisRotary(32, 2, sections=[10, 7])
    rot = AxisRotary(32, 2)
    with pytest.raises(ValueError, match="no gradient"):
        rot(torch.zeros(4, 2, 32, device=dev), torch.zeros(4, 2, device=dev, requires_grad=True))
    blk = KmipGlobalAttention(64, 2, 4, dtype=BF, device=dev, rotary=rot)
    with pytest.raises(ValueError, match="positions"):
        blk(torch.zeros(8, 64, dtype=BF, device=dev))


def test_module_casts_keep_the_frequencies(dev):
    rot = AxisRotary(32, 2)
    m = torch.nn.Sequential(rot).to(BF).to(dev)
    freq, axis = m[0].tables(dev)
    assert freq.dtype == torch.float64 and axis.dtype == torch.int32


def test_captured_training_step(dev):
    """Forward and backward of the layer captured into a graph, replayed with
    new inputs, against the eager gradients."""
    torch.manual_seed(5)
    layer = GraphTransformerLayer(64, 2, 8, 136, 4, axes=2, device=dev)
    offsets = wl.offsets_from_sizes([200, 90]).to(dev)
    x = torch.randn(290, 64, device=dev).to(BF).requires_grad_(True)
    pos = torch.rand(290, 2, device=dev)
    gy = torch.randn(290, 64, device=dev).to(BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(layer(x, offsets, pos), [x, layer.ffn.gate], gy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, offsets, pos)
        dx, dgate = torch.autograd.grad(y, [x, layer.ffn.gate], gy)
    with torch.no_grad():
        x.mul_(0.75)
    graph.replay()
    torch.cuda.synchronize()
    y2 = layer(x, offsets, pos)
    dx2, dgate2 = torch.autograd.grad(y2, [x, layer.ffn.gate], gy)
    torch.cuda.synchronize()
    binding.check_status()
    assert torch.equal(y, y2)
    # dK and dV are fp32 atomic sums whose last bits vary
    assert (dx.float() - dx2.float()).norm() <= 4e-3 * dx2.float().norm()
    assert torch.equal(dgate, dgate2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_odd_strides_and_addresses(dev, dtype, interleaved):
    """Inputs and gradients at odd strides or behind an odd number of elements,
    as torch.cat hands them back, give what their copies give."""
    rot = AxisRotary(4, 2, interleaved=interleaved)
    g = torch.Generator(device=dev).manual_seed(3)

    def n(*s):
        return torch.randn(s, generator=g, device=dev).to(dtype)

    pos = torch.rand((5, 2), generator=g, device=dev)
    for flat in (False, True):
        x, extra = n(5, 2, 4).requires_grad_(True), n(3) if flat else n(5, 3)
        y = rot(x, pos)
        joined = torch.cat([extra, y.flatten(0 if flat else 1)], -1)
        w = n(*joined.shape)
        dx, = torch.autograd.grad(joined, x, w)
        part = w[3:].view(5, 2, 4) if flat else w[:, 3:].reshape(5, 2, 4)
        want, = torch.autograd.grad(rot(x, pos), x, part.clone())
        assert torch.equal(dx, want)
        # the same layouts as inputs
        view = w[3:].view(5, 2, 4) if flat else w[:, 3:].unflatten(1, (2, 4))
        assert torch.equal(rot(view, pos), rot(view.clone(), pos))
    binding.check_status()


def _behind(t, n):
    """t's values as a contiguous view, n elements into its storage."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    buf[n:] = t.detach().flatten()
    return buf[n:].view(t.shape)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_feed_forward_at_any_address(dev, dtype):
    """Rows, weights and gradients that lie behind other elements."""
    torch.manual_seed(2)
    ffn = GatedFeedForward(32, 48, dtype=dtype, device=dev)
    x, gy = (torch.randn(30, 32, device=dev).to(dtype) for _ in range(2))
    leaves = [x.clone().requires_grad_(True), ffn.gate, ffn.up, ffn.down]
    y = ffn(leaves[0])
    want = torch.autograd.grad(y, leaves, gy)
    moved = GatedFeedForward(32, 48, dtype=dtype, device=dev)
    for name in ("gate", "up", "down"):
        setattr(moved, name, torch.nn.Parameter(_behind(getattr(ffn, name), 3)))
    leaves = [_behind(x, 1).requires_grad_(True), moved.gate, moved.up, moved.down]
    y2 = moved(leaves[0])
    got = torch.autograd.grad(torch.cat([torch.zeros_like(gy[0, :3]), y2.flatten()]), leaves,
                              torch.cat([gy[0, :3], gy.flatten()]))
    assert torch.equal(y, y2)
    for a, c in zip(got, want):
        assert torch.equal(a, c)


def test_attention_at_any_address(dev):
    from graph_transformer_sparse_kmip_b200.layer import kmip_attention
    g = torch.Generator(device=dev).manual_seed(4)
    q, k, v, gy = (torch.randn((40, 2, 32), generator=g, device=dev).to(BF) for _ in range(4))
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    y, idx = kmip_attention(*leaves, 5)
    want = torch.autograd.grad(y, leaves, gy)
    leaves = [_behind(t, 1).requires_grad_(True) for t in (q, k, v)]
    y2, idx2 = kmip_attention(*leaves, 5)
    got = torch.autograd.grad(torch.cat([gy[0, 0, :3], y2.flatten()]), leaves,
                              torch.cat([gy[0, 0, :3], gy.flatten()]))
    assert torch.equal(y, y2) and torch.equal(idx, idx2)
    assert torch.equal(got[0], want[0])
    for a, c in zip(got[1:], want[1:]):     # fp32 atomic sums, rounded to bf16
        assert (a.float() - c.float()).norm() <= 4e-3 * c.float().norm()
