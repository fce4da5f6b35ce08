"""Rotary positions with several axes against complex products in fp64.

Tolerance: with e the half step of the output type, an output may be off by
e |out| (its one rounding) plus 2^-20 (|u| + |v|): the reduced angle is
rounded to fp32 (2^-25 revolutions, 1.9e-7 rad), sincospif is good to 2 ulp
(2.4e-7) and the turn takes two fp32 roundings (1.2e-7 each), in all under
2^-20 = 9.5e-7 of the pair's values.
"""
import pytest
import torch

from graph_transformer_sparse_kmip_b200 import binding
from graph_transformer_sparse_kmip_b200.binding import KmipError

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


def _table(P, axes, dev):
    j = torch.arange(P, dtype=torch.float64)
    freq = 100.0 ** (-j / max(P, 1))
    return freq.to(dev), (torch.arange(P, dtype=torch.int32) % axes).to(dev)


def _reference(x, pos, freq, axis, inverse, interleaved):
    """fp64 result and the size of each element's pair."""
    x, P = x.double().cpu(), freq.numel()
    ang = pos.double().cpu()[:, axis.long().cpu()] * freq.cpu()
    turn = torch.polar(torch.ones_like(ang), -ang if inverse else ang)[:, None]
    out, size = x.clone(), torch.zeros_like(x)
    if interleaved:
        u, v = slice(0, 2 * P, 2), slice(1, 2 * P, 2)
    else:
        u, v = slice(0, P), slice(P, 2 * P)
    z = torch.complex(x[..., u], x[..., v]) * turn
    out[..., u], out[..., v] = z.real, z.imag
    size[..., u] = size[..., v] = x[..., u].abs() + x[..., v].abs()
    return out, size


def _check(got, ref, size):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double().cpu() - ref).abs()
    assert (err <= half * ref.abs() + 2.0 ** -20 * size).all(), err.max()


def _inputs(N, H, d, axes, dtype, dev, seed=0, pos_type=F32, span=50.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, H, d), generator=g).to(dtype).to(dev)
    pos = (torch.rand((N, axes), generator=g) * 2 - 1) * span
    return x, pos.to(pos_type).to(dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,d,P,axes", [
    (1, 1, 2, 1, 1), (1, 8, 32, 16, 2), (7, 3, 32, 12, 3), (257, 5, 40, 20, 4),
    (33, 2, 16, 6, 3), (130, 8, 128, 64, 3), (64, 1, 6, 2, 2), (5, 4, 512, 256, 2),
    (9, 70, 64, 32, 1), (100, 2, 34, 17, 2), (3, 300, 10, 5, 5), (20, 2, 8, 0, 1)])
def test_matches_fp64(dev, dtype, interleaved, N, H, d, P, axes):
    x, pos = _inputs(N, H, d, axes, dtype, dev, seed=N + d)
    freq, axis = _table(P, axes, dev)
    for inverse in (False, True):
        out = binding.rotary(x, pos, freq, axis, inverse=inverse, interleaved=interleaved)
        binding.check_status()
        _check(out, *_reference(x, pos, freq, axis, inverse, interleaved))


@pytest.mark.parametrize("pos_type", [F32, torch.int32, torch.int64])
def test_far_positions(dev, pos_type):
    x, pos = _inputs(50, 2, 32, 2, F32, dev, seed=3, pos_type=pos_type, span=1.0e6)
    if pos_type == torch.int64:
        pos = pos + (1 << 33)
    freq, axis = _table(16, 2, dev)
    out = binding.rotary(x, pos, freq, axis)
    # an fp64 angle of 2^33 rad is off by 2^-20: beside the stated tolerance
    ref, size = _reference(x, pos, freq, axis, False, False)
    extra = pos.double().abs().max().item() * 2.0 ** -51 if pos_type == torch.int64 else 0.0
    err = (out.double().cpu() - ref).abs()
    assert (err <= 2.0 ** -24 * ref.abs() + (2.0 ** -20 + extra) * size).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_views_and_in_place(dev, dtype, interleaved):
    N, H, d, axes = 300, 4, 32, 2
    g = torch.Generator().manual_seed(9)
    qkv = torch.randn((N, 3 * H, d), generator=g).to(dtype).to(dev)
    keep = qkv.clone()
    pos = torch.rand((N, axes), generator=g).to(dev) * 9
    freq, axis = _table(16, axes, dev)
    view = qkv[:, : 2 * H]
    ref, size = _reference(view, pos, freq, axis, False, interleaved)
    _check(binding.rotary(view, pos, freq, axis, interleaved=interleaved), ref, size)
    # heads outermost: x[h, n, e]
    perm = view.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = torch.full_like(perm, 7.0)
    binding.rotary(perm, pos, freq, axis, interleaved=interleaved, out=out)
    _check(out, ref, size)
    # an offset that leaves only the element's (or the pair's) alignment
    off = 2
    buf = torch.zeros((N, H * d + off), dtype=dtype, device=dev)
    odd = buf[:, off:].unflatten(1, (H, d))
    odd.copy_(view[:, :H])
    r2, s2 = _reference(odd, pos, freq, axis, False, interleaved)
    _check(binding.rotary(odd, pos, freq, axis, interleaved=interleaved), r2, s2)
    # one query head shown to every head (stride 0)
    one = qkv[:, :1].expand(N, H, d)
    r3, s3 = _reference(one, pos, freq, axis, False, interleaved)
    _check(binding.rotary(one, pos, freq, axis, interleaved=interleaved), r3, s3)
    # in place; the value heads behind the view stay as they were
    binding.rotary(view, pos, freq, axis, interleaved=interleaved, out=view)
    _check(qkv[:, : 2 * H], ref, size)
    assert torch.equal(qkv[:, 2 * H:], keep[:, 2 * H:])


def test_odd_offset_halves(dev):
    """bf16 halves at a 2-byte offset take single elements."""
    buf = torch.randn((40, 2 * 32 + 1), device=dev).to(BF)
    x = buf[:, 1:].unflatten(1, (2, 32))
    pos = torch.rand((40, 1), device=dev)
    freq, axis = _table(16, 1, dev)
    _check(binding.rotary(x, pos, freq, axis), *_reference(x, pos, freq, axis, False, False))


def test_inverse_undoes_the_turn_and_is_the_gradient(dev):
    x, pos = _inputs(60, 4, 32, 3, F32, dev, seed=5)
    freq, axis = _table(15, 3, dev)
    back = binding.rotary(binding.rotary(x, pos, freq, axis), pos, freq, axis, inverse=True)
    assert (back - x).abs().max() <= 2.0 ** -18 * 4.5
    # <turn(x), g> = <x, turn^-1(g)>: the adjoint, hence the gradient
    g = torch.randn_like(x)
    a = (binding.rotary(x, pos, freq, axis).double() * g.double()).sum()
    b = (x.double() * binding.rotary(g, pos, freq, axis, inverse=True).double()).sum()
    assert abs(a - b) <= 2.0 ** -20 * (x.abs().double() * g.abs().double()).sum() * 2


def test_special_values_stay_in_their_pair(dev):
    x, pos = _inputs(4, 2, 16, 1, F32, dev)
    freq, axis = _table(6, 1, dev)
    x[1, 0, 3] = float("nan")
    x[2, 1, 14] = float("inf")          # behind the pairs: copied
    out = binding.rotary(x, pos, freq, axis)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 9] = want[2, 1, 14] = True
    assert torch.equal(bad, want) and out[2, 1, 14] == float("inf")


def test_bad_axis_is_reported_and_skipped(dev):
    x, pos = _inputs(5, 2, 16, 2, F32, dev)
    freq, axis = _table(8, 2, dev)
    axis[3] = 2
    out = binding.rotary(x, pos, freq, axis)
    with pytest.raises(KmipError) as e:
        binding.check_status()
    assert e.value.code == 6
    assert torch.equal(out[..., 3], x[..., 3]) and torch.equal(out[..., 11], x[..., 11])
    binding.check_status()


def test_empty_stream_and_graph_capture(dev):
    freq, axis = _table(16, 2, dev)
    assert binding.rotary(torch.empty((0, 4, 32), device=dev), torch.empty((0, 2), device=dev),
                          freq, axis).shape == (0, 4, 32)
    x, pos = _inputs(100, 4, 32, 2, BF, dev)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.rotary(x, pos, freq, axis, out=out, stream=side)
    side.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.rotary(x, pos, freq, axis, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    pos.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    _check(out, *_reference(x, pos, freq, axis, False, False))


def test_out_is_returned_and_checked(dev):
    x = torch.randn((5, 2, 32), device=dev)
    pos, freq = torch.zeros((5, 1), device=dev), torch.ones(16, dtype=torch.float64, device=dev)
    axis = torch.zeros(16, dtype=torch.int32, device=dev)
    assert binding.rotary(x, pos, freq, axis, out=x) is x
    y = torch.empty_like(x)
    assert binding.rotary(x, pos, freq, axis, out=y, stream=torch.cuda.current_stream()) is y
    assert torch.equal(x, y)
    for out in (y[:4], y.bfloat16(), y.cpu(), y[0], y.transpose(1, 2)):
        with pytest.raises(ValueError, match="out"):
            binding.rotary(x, pos, freq, axis, out=out)
    with pytest.raises(ValueError, match="contiguous"):
        binding.rotary(x, pos, freq.cpu(), axis)
    with pytest.raises(TypeError, match="dtype"):
        binding.rotary(x.double(), pos, freq, axis)
    binding.check_status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_of_single_rows_and_heads_do_not_matter(dev, dtype, interleaved):
    """A dimension of one has whatever stride the view it came from left."""
    freq, axis = _table(16, 1, dev)
    for N, H, strides in ((5, 1, (34, 33, 1)), (1, 5, (33, 32, 1)), (1, 1, (7, 5, 1)),
                          (5, 1, (32, 0, 1)), (1, 1, (0, 0, 1))):
        base, pos = torch.randn(400, device=dev).to(dtype), torch.rand((N, 1), device=dev)
        x = base.as_strided((N, H, 32), strides)
        want = binding.rotary(x.clone(memory_format=torch.contiguous_format), pos, freq, axis,
                              interleaved=interleaved)
        assert torch.equal(binding.rotary(x, pos, freq, axis, interleaved=interleaved), want)
        out = torch.zeros(400, dtype=dtype, device=dev).as_strided((N, H, 32), strides)
        assert torch.equal(binding.rotary(x, pos, freq, axis, interleaved=interleaved, out=out),
                           want)
        assert torch.equal(binding.rotary(x, pos, freq, axis, interleaved=interleaved, out=x),
                           want)
    binding.check_status()


def test_out_between_the_heads_of_x(dev):
    """Other heads of the same rows are another tensor."""
    g = torch.Generator(device=dev).manual_seed(1)
    qkv = torch.randn((300, 12, 32), generator=g, device=dev).to(BF)
    pos = torch.rand((300, 1), generator=g, device=dev)
    freq, axis = _table(16, 1, dev)
    q, k, keep = qkv[:, :4], qkv[:, 4:8], qkv.clone()
    want = binding.rotary(q, pos, freq, axis)
    binding.rotary(q, pos, freq, axis, out=k)
    assert torch.equal(k, want) and torch.equal(qkv[:, :4], keep[:, :4])
    assert torch.equal(qkv[:, 8:], keep[:, 8:])
    with pytest.raises(KmipError) as e:
        binding.rotary(q, pos, freq, axis, out=qkv[:, 3:7])
    assert e.value.code == 1
    with pytest.raises(KmipError):
        binding.rotary(qkv[:299], pos[:299], freq, axis, out=qkv[1:])
    binding.check_status()


def test_a_turn_in_place_is_seen_by_autograd(dev):
    """A tensor that the backward pass needs and that was turned since raises."""
    pos = torch.rand((5, 1), device=dev)
    freq, axis = _table(16, 1, dev)
    for stream in (None, torch.cuda.current_stream()):
        x = torch.randn((5, 2, 32), device=dev, requires_grad=True)
        y = x * 2
        loss = y.square().sum()
        version = y._version
        binding.rotary(y, pos, freq, axis, out=y, stream=stream)
        assert y._version == version + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():
        z = torch.randn((5, 2, 32), device=dev)
        binding.rotary(z, pos, freq, axis, out=z)
    binding.rotary(z, pos, freq, axis, out=z)
    fresh = torch.randn((5, 2, 32), device=dev)
    assert binding.rotary(fresh, pos, freq, axis)._version == 0 and fresh._version == 0
    binding.check_status()
