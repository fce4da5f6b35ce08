"""Group norm per graph with an activation, forward and backward, against
fp64 (the definition for the forward, torch autograd for the gradients).

Tolerances (e = half step of the output type, u = 2^-24):
  y      one rounding, e |y|, plus the fp32 error of z = xhat w + b carried
         through the activation (slope at most 1.13): the mean and rstd of a
         thread's running join move by at most about 64 u of |mean| + |x|
         over the joins of these sizes, so |dz| <= 64 u (|w| (|xhat| +
         rstd (|x| + |mean|)) + |b|), 64 u = 2^-18;
  dx     e |dx| plus 2^-16 rstd (|dy w| + |m1| + |xhat m2|), four times that
         for the two group sums and the products, and slope-of-slope <= 1;
  dw, db e |value| plus 256 u of the sum of the terms' sizes (the longest
         run of fp32 additions of one thread and its joins).
"""
import ctypes

import pytest
import torch

from graph_transformer_sparse_kmip_b200 import binding
from graph_transformer_sparse_kmip_b200 import workloads as wl
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


def _act(z, act):
    f = torch.nn.functional
    return {"none": lambda t: t, "silu": f.silu, "gelu": f.gelu, "relu": f.relu}[act](z)


def _reference(x, w, b, dy, off, groups, act, eps):
    """fp64 values and tolerance scales, on x's device."""
    x = x.double().requires_grad_(True)
    w = (torch.ones(x.shape[1], device=x.device) if w is None else w).double().requires_grad_(True)
    b = (torch.zeros(x.shape[1], device=x.device) if b is None else b).double().requires_grad_(True)
    dy = dy.double()
    C = x.shape[1]
    cg = C // groups
    means, rstds, hats, spread_m, spread_r = [], [], [], [], []
    for part in x.split((off[1:] - off[:-1]).tolist()):
        p = part.unflatten(1, (groups, cg))
        if len(p):
            m = p.mean((0, 2))
            v = (p - m[:, None]).square().mean((0, 2))
        else:
            m = v = x.new_zeros(groups)
        r = (v + eps) ** -0.5
        means.append(m), rstds.append(r)
        hats.append(((p - m[:, None]) * r[:, None]).flatten(1))
        spread_m.append(m.repeat_interleave(cg).expand(len(p), C))
        spread_r.append(r.repeat_interleave(cg).expand(len(p), C))
    xhat = torch.cat(hats)
    z = xhat * w + b
    y = _act(z, act)
    gx, gw, gb = torch.autograd.grad(y, (x, w, b), dy, retain_graph=True)
    dz, = torch.autograd.grad(y, z, dy)
    with torch.no_grad():
        m, r = torch.cat(spread_m).abs(), torch.cat(spread_r)
        ztol = 2.0 ** -18 * (w.abs() * (xhat.abs() + r * (x.abs() + m)) + b.abs())
        g1, g2, lo = [], [], 0
        for n in (off[1:] - off[:-1]).tolist():
            t = (dz * w)[lo:lo + n].unflatten(1, (groups, cg))
            h = xhat[lo:lo + n].unflatten(1, (groups, cg))
            if n:
                g1.append((t.abs().mean((0, 2)).repeat_interleave(cg)).expand(n, C))
                g2.append(((t * h).abs().mean((0, 2)).repeat_interleave(cg)).expand(n, C))
            lo += n
        g1 = torch.cat(g1) if g1 else xhat * 0
        g2 = torch.cat(g2) if g2 else xhat * 0
        cond = 1 + r * (x.abs() + m)          # how far cancellation in x - mean reaches
        xtol = 2.0 ** -16 * r * ((dy * w).abs() * (1 + cond * w.abs()) + g1 + g2 * (xhat.abs() + cond))
        slack = dy.abs() * (1 + cond * w.abs())
        wtol = 2.0 ** -16 * (slack * (xhat.abs() + cond)).sum(0)
        btol = 2.0 ** -16 * slack.sum(0)
    return dict(y=y.detach(), mean=torch.stack(means).detach(), rstd=torch.stack(rstds).detach(),
                dx=gx, dw=gw, db=gb), dict(y=1.13 * ztol, dx=xtol, dw=wtol, db=btol)


def _case(sizes, C, dtype, dev, seed=0, shift=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    N = sum(sizes)

    def n(*s):
        return torch.randn(s, generator=g, device=dev)

    x = (n(N, C) * (0.5 + torch.rand(C, generator=g, device=dev)) + shift * n(C)).to(dtype)
    return (x, (1 + 0.2 * n(C)).to(dtype), (0.2 * n(C)).to(dtype), n(N, C).to(dtype),
            wl.offsets_from_sizes(sizes).to(dev))


def _close(got, ref, tol, name):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - ref).abs()
    assert (err <= half * ref.abs() + tol).all(), (name, (err - half * ref.abs() - tol).max())


def _check(x, w, b, dy, off, groups, act, eps=1e-5, offsets=True):
    go = off if offsets else None
    y, mean, rstd = binding.group_norm_fwd(x, w, b, groups, eps, act, go)
    dx, dw, db = binding.group_norm_bwd(dy, x, w, b, mean, rstd, groups, act, go)
    binding.check_status()
    ref, tol = _reference(x, w, b, dy, off, groups, act, eps)
    scale = x.double().abs().max() if x.numel() else 0.0
    _close(mean, ref["mean"], 2.0 ** -18 * scale, "mean")
    assert ((rstd.double() - ref["rstd"]).abs() <= 2.0 ** -16 * ref["rstd"]
            * (1 + ref["rstd"] * scale * 2.0 ** -4)).all()
    _close(y, ref["y"], tol["y"], "y")
    _close(dx, ref["dx"], tol["dx"], "dx")
    if w is not None:
        _close(dw, ref["dw"], tol["dw"], "dw")
        _close(db, ref["db"], tol["db"], "db")
    else:
        assert dw is None and db is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
@pytest.mark.parametrize("sizes,C,groups", [
    ([300, 45, 0, 517, 129], 128, 8),     # vectors of 8 inside a group
    ([0, 0, 77, 1, 90, 0], 64, 4),        # empty graphs at both ends, one node
    ([200, 133], 345, 15),                # odd channels: single elements
    ([100], 36, 6),                       # 6 channels a group: pairs in bf16
    ([500, 300], 24, 24),                 # one channel a group
    ([64, 1, 30], 48, 1),                 # one group
    ([3, 2], 4608, 1)])                   # a group wider than one tile of a block
def test_small_graphs(dev, dtype, act, sizes, C, groups):
    x, w, b, dy, off = _case(sizes, C, dtype, dev, seed=C)
    if groups == C:
        # a node's only channel: its graph needs more than a few nodes
        assert min(sizes) >= 64
    _check(x, w, b, dy, off, groups, act)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,C,groups", [
    ([0, 60001, 0, 1, 9000, 130], 256, 32),
    ([40000], 345, 15),
    ([20000, 50000], 130, 13),
    ([5000] * 10, 520, 65)])              # more than 64 groups: two slabs
def test_large_graphs(dev, dtype, sizes, C, groups):
    x, w, b, dy, off = _case(sizes, C, dtype, dev, seed=C + 1)
    _check(x, w, b, dy, off, groups, "silu")


def test_one_graph_without_offsets_and_without_parameters(dev):
    x, w, b, dy, off = _case([700], 64, BF, dev)
    _check(x, w, b, dy, off, 8, "silu", offsets=False)
    _check(x, None, None, dy, off, 8, "gelu", offsets=False)


def test_single_node(dev):
    x, w, b, dy, off = _case([1], 128, F32, dev)
    _check(x, w, b, dy, off, 2, "silu")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,groups", [(64, 4), (128, 4), (40, 8)])
def test_more_graphs_than_blocks_fit(dev, dtype, C, groups):
    """Graphs that are kept on the chip and longer ones, several waves of blocks."""
    g = torch.Generator().manual_seed(5)
    sizes = [0, 1, 511, 512, 513] + [int(v) for v in torch.randint(0, 700, (320,), generator=g)]
    x, w, b, dy, off = _case(sizes, C, dtype, dev, seed=6)
    _check(x, w, b, dy, off, groups, "silu")


def test_many_tiny_graphs(dev):
    sizes = [int(v) for v in torch.randint(0, 9, (5000,), generator=torch.Generator().manual_seed(2))]
    x, w, b, dy, off = _case(sizes, 64, F32, dev, seed=4)
    _check(x, w, b, dy, off, 1, "relu")


def test_mean_far_from_zero(dev):
    """A mean of a thousand deviations: no difference of large sums."""
    x, w, b, dy, off = _case([900, 40], 64, F32, dev, seed=6, shift=0.0)
    x = x + 1000.0
    _check(x, w, b, dy, off, 4, "none")


def test_nan_and_inf_stay_in_their_graph_and_group(dev):
    x, w, b, dy, off = _case([50, 60, 70], 64, BF, dev)
    x[60, 5] = float("nan")
    x[120, 40] = float("inf")
    y, mean, rstd = binding.group_norm_fwd(x, w, b, 4, 1e-5, "silu", off)
    bad = ~torch.isfinite(y.float())
    want = torch.zeros_like(bad)
    want[50:110, 0:16] = True
    want[110:180, 32:48] = True
    assert torch.equal(bad, want)
    assert not torch.isfinite(mean[1, 0]) and not torch.isfinite(mean[2, 2])


def test_unaligned_rows(dev):
    """A base pointer off the 16-byte grid takes narrower loads."""
    for dtype in (BF, F32):
        x, w, b, dy, off = _case([130, 20], 64, dtype, dev)
        flat = torch.empty(x.numel() + 1, dtype=dtype, device=dev)
        x1 = flat[1:].view(x.shape)
        x1.copy_(x)
        y0, m0, r0 = binding.group_norm_fwd(x, w, b, 8, 1e-5, "silu", off)
        y1, m1, r1 = binding.group_norm_fwd(x1, w, b, 8, 1e-5, "silu", off)
        assert (y0.float() - y1.float()).abs().max() <= torch.finfo(dtype).eps * 8
        assert torch.allclose(m0, m1, rtol=0, atol=1e-6)
        assert torch.allclose(r0, r1, rtol=2.0 ** -18, atol=0)


@pytest.mark.parametrize("sizes,C", [([300, 45, 517], 128), ([50000, 40000], 128)])
def test_bits_repeat(dev, sizes, C):
    x, w, b, dy, off = _case(sizes, C, BF, dev)
    a = binding.group_norm_fwd(x, w, b, 8, 1e-5, "silu", off)
    c = binding.group_norm_bwd(dy, x, w, b, a[1], a[2], 8, "silu", off)
    for _ in range(3):
        a2 = binding.group_norm_fwd(x, w, b, 8, 1e-5, "silu", off)
        c2 = binding.group_norm_bwd(dy, x, w, b, a2[1], a2[2], 8, "silu", off)
        for p, q in zip(a + c, a2 + c2):
            assert torch.equal(p, q)


@pytest.mark.parametrize("sizes", [[300, 45], [60000, 30000]])
def test_in_place_through_the_c_entry(dev, sizes):
    x, w, b, dy, off = _case(sizes, 128, BF, dev)
    N, C = x.shape
    y, mean, rstd = binding.group_norm_fwd(x, w, b, 8, 1e-5, "silu", off)
    dx, dw, db = binding.group_norm_bwd(dy, x, w, b, mean, rstd, 8, "silu", off)
    lib, p = binding.load(), binding._ptr
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    G = off.numel() - 1
    g = dy.clone()
    dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
    assert lib.kmip_group_norm_bwd(p(g), p(x), p(w), p(b), p(off), p(mean), p(rstd), N, C, 8, 1,
                                   p(g), p(dw2), p(db2), s, G, 0) == 0
    z = x.clone()
    m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
    assert lib.kmip_group_norm_fwd(p(z), p(w), p(b), p(off), N, C, 8, 1e-5, 1, p(z), p(m2), p(r2),
                                   s, G, 0) == 0
    torch.cuda.synchronize()
    for a, c in ((z, y), (m2, mean), (g, dx), (dw2, dw), (db2, db)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("bad", [[0, 30, 20, 50], [1, 20, 50], [0, 20, 49], [0, -5, 50],
                                 [0, 60, 50]])
def test_malformed_offsets_are_reported(dev, bad):
    x, w, b, dy, _ = _case([50], 64, BF, dev)
    off = torch.tensor(bad, dtype=torch.int32, device=dev)
    y, mean, rstd = binding.group_norm_fwd(x, w, b, 4, 1e-5, "silu", off)
    with pytest.raises(KmipError) as e:
        binding.check_status()
    assert e.value.code == 4
    binding.group_norm_bwd(dy, x, w, b, torch.zeros_like(mean), torch.ones_like(rstd), 4, "silu",
                           off)
    with pytest.raises(KmipError) as e:
        binding.check_status()
    assert e.value.code == 4
    binding.check_status()


def test_malformed_offsets_of_large_graphs_are_reported(dev):
    x, w, b, dy, _ = _case([90000], 128, BF, dev)
    for bad in ([0, 60000, 30000, 90000], [0, 90001, 90000], [5, 90000], [0, -7, 90000]):
        off = torch.tensor(bad, dtype=torch.int32, device=dev)
        _, mean, rstd = binding.group_norm_fwd(x, w, b, 4, 1e-5, "silu", off)
        with pytest.raises(KmipError) as e:
            binding.check_status()
        assert e.value.code == 4
        binding.group_norm_bwd(dy, x, w, b, torch.zeros_like(mean), torch.ones_like(rstd), 4,
                               "silu", off)
        with pytest.raises(KmipError) as e:
            binding.check_status()
        assert e.value.code == 4


@pytest.mark.parametrize("at", [1, 1001, 1999])
def test_malformed_offsets_of_many_graphs_are_reported(dev, at):
    """Wherever among many graphs they are, and only there: 2,000 graphs of 30
    nodes with 155 channels, too many bytes for one block a graph."""
    x, w, b, dy, off = _case([30] * 2000, 155, BF, dev)
    mean = torch.zeros((2000, 31), device=dev)
    off[at] += 31  # behind the graph's own end
    binding.group_norm_fwd(x, w, b, 31, 1e-5, "silu", off)
    with pytest.raises(KmipError) as e:
        binding.check_status()
    assert e.value.code == 4
    binding.group_norm_bwd(dy, x, w, b, mean, mean + 1, 31, "silu", off)
    with pytest.raises(KmipError) as e:
        binding.check_status()
    assert e.value.code == 4
    off[at] -= 31
    y, mean, rstd = binding.group_norm_fwd(x, w, b, 31, 1e-5, "silu", off)
    binding.group_norm_bwd(dy, x, w, b, mean, rstd, 31, "silu", off)
    binding.check_status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("sizes,C", [([300, 45], 64), ([90000], 128)])
def test_a_channel_without_a_number_stays_alone(dev, dtype, act, sizes, C):
    x, w, b, dy, off = _case(sizes, C, dtype, dev)
    y, mean, rstd = binding.group_norm_fwd(x, w, b, 4, 1e-5, act, off)
    _, dw, db = binding.group_norm_bwd(dy, x, w, b, mean, rstd, 4, act, off)
    for value in (float("nan"), float("inf"), -float("inf")):
        v, bad = b.clone(), (6, 33)
        v[list(bad)] = value
        yv, mv, rv = binding.group_norm_fwd(x, w, v, 4, 1e-5, act, off)
        _, dwv, dbv = binding.group_norm_bwd(dy, x, w, v, mean, rstd, 4, act, off)
        rest = [c for c in range(C) if c not in bad]
        assert torch.equal(yv[:, rest], y[:, rest])
        assert torch.equal(mv, mean) and torch.equal(rv, rstd)
        assert torch.equal(dwv[rest], dw[rest]) and torch.equal(dbv[rest], db[rest])
        if value != value:
            assert yv[:, list(bad)].isnan().all()
    binding.check_status()


def test_no_nodes(dev):
    x = torch.empty((0, 64), device=dev)
    w, b = torch.ones(64, device=dev), torch.zeros(64, device=dev)
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    y, mean, rstd = binding.group_norm_fwd(x, w, b, 4, 1e-2, "silu", off)
    dx, dw, db = binding.group_norm_bwd(x, x, w, b, mean, rstd, 4, "silu", off)
    assert (mean == 0).all() and torch.allclose(rstd, torch.full_like(rstd, 10.0))
    assert y.shape == dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("sizes", [[300, 45], [60000, 30000]])
def test_captured_graphs_replay_side_by_side(dev, sizes):
    """Two captured graphs (each with its scratch) on two streams, replayed
    with new inputs."""
    work = []
    for seed in (1, 2):
        x, w, b, dy, off = _case(sizes, 128, BF, dev, seed=seed)
        binding.group_norm_fwd(x, w, b, 8, 1e-5, "silu", off)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, mean, rstd = binding.group_norm_fwd(x, w, b, 8, 1e-5, "silu", off)
            grads = binding.group_norm_bwd(dy, x, w, b, mean, rstd, 8, "silu", off)
        work.append((graph, torch.cuda.Stream(), (x, w, b, dy, off), (y, mean, rstd) + grads))
    for _, _, (x, w, b, dy, off), _ in work:
        x.mul_(1.5)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, _, _ in work:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, (x, w, b, dy, off), got in work:
        y, mean, rstd = binding.group_norm_fwd(x, w, b, 8, 1e-5, "silu", off)
        want = (y, mean, rstd) + binding.group_norm_bwd(dy, x, w, b, mean, rstd, 8, "silu", off)
        for a, c in zip(got, want):
            assert torch.equal(a, c)


@pytest.mark.parametrize("dtype,N,C,groups,G", [
    (BF, 60000, 128, 8, 3000),            # resident, short graphs: slabs of a whole row
    (F32, 30000, 264, 33, 120),           # resident, above 16 MB
    (BF, 60000, 154, 7, 700),             # split, narrow loads, few slots a graph
    (F32, 40000, 129, 3, 50)])            # split, 129 channels
def test_many_graphs(dev, dtype, N, C, groups, G):
    g = torch.Generator().manual_seed(C)
    cut = torch.randint(0, N + 1, (G - 1,), generator=g).sort().values.tolist()
    sizes = [b - a for a, b in zip([0] + cut, cut + [N])]
    x, w, b, dy, off = _case(sizes, C, dtype, dev, seed=G)
    _check(x, w, b, dy, off, groups, "silu")


ALIKE = pytest.mark.parametrize("sizes,C,groups", [
    ([1, 700, 3], 64, 8), ([1] * 40, 64, 64), ([90000, 7], 128, 8), ([5, 70000], 129, 3),
    ([600], 36, 6), ([3, 2], 4608, 1)])


def _alike(sizes, C, value, dtype, dev):
    x = torch.full((sum(sizes), C), value, device=dev).to(dtype)
    w, b = torch.full_like(x[0], 2.0), torch.full_like(x[0], 0.5)
    return x, w, b, wl.offsets_from_sizes(sizes).to(dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [1234.567, -1.0e6])
@ALIKE
def test_values_that_are_all_alike(dev, dtype, sizes, C, groups, value):
    """Nodes whose features are one constant (padding, a single node with one
    channel a group): x - mean is zero, so y is act(bias), whatever rstd."""
    x, w, b, off = _alike(sizes, C, value, dtype, dev)
    G = len(sizes)
    y, mean, _ = binding.group_norm_fwd(x, w, b, groups, 1e-5, "none", off)
    assert (mean == x[0, 0].float()).all()
    assert (y.float() == 0.5).all()
    # with the statistics that the definition has
    rstd = torch.full((G, groups), 1e-5 ** -0.5, device=dev)
    dy = torch.randn(x.shape, generator=torch.Generator(device=dev).manual_seed(1),
                     device=dev).to(dtype)
    dx, dw, db = binding.group_norm_bwd(dy, x, w, b, mean, rstd, groups, "none", off)
    assert (dw == 0).all()
    binding.check_status()


def test_mean_far_from_zero_bf16(dev):
    """As for fp32 below the half step of bf16: values around 1,000, a step of 4
    apart, a dozen steps in all."""
    x, w, b, dy, off = _case([900, 40], 64, BF, dev, seed=6, shift=0.0)
    x = (x.float() * 8 + 1000.0).to(BF)
    _check(x, w, b, dy, off, 4, "none")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("seed", range(4))
@ALIKE
def test_statistics_of_values_that_are_all_alike(dev, dtype, sizes, C, groups, seed):
    """Their mean is the value and their variance zero, at any size: nothing is
    subtracted that is not a difference to one of the values."""
    g = torch.Generator().manual_seed(seed)
    for value in (torch.randn(12, generator=g) * 100.0 ** seed).tolist():
        x, w, b, off = _alike(sizes, C, value, dtype, dev)
        y, mean, rstd = binding.group_norm_fwd(x, w, b, groups, 1e-5, "none", off)
        binding.check_status()
        assert (mean == x[0, 0].float()).all()
        # one square root and one rounding
        assert ((rstd.double() * 1e-5 ** 0.5 - 1).abs() <= 2.0 ** -22).all()
        assert (y.float() == 0.5).all()


def _bf16_values(lo, hi, dev):
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(BF)
    v = v[(v.float() >= lo) & (v.float() <= hi) & (v.float().abs() >= 2.0 ** -20)]
    return v[: v.numel() // 8 * 8].to(dev)


@pytest.mark.parametrize("cg", [8, 2, 1])
def test_gelu_of_every_value(dev, cg):
    """With weight 0 the activation's argument is the bias.  One rounding, 2^-8,
    and 2^-16 of the value: the tail of the normal distribution is good to
    2^-17 down to -13, its density likewise."""
    z = _bf16_values(-12.0, 12.0, dev)
    C, zero = z.numel(), torch.zeros_like(z)
    x = torch.randn((3, C), generator=torch.Generator(device=dev).manual_seed(0),
                    device=dev).to(BF)
    y, mean, rstd = binding.group_norm_fwd(x, zero, z, C // cg, 1e-5, "gelu")
    v = z.double()
    cdf = 0.5 * torch.special.erfc(-v / 2 ** 0.5)
    assert ((y.double() - v * cdf).abs() <= (2.0 ** -8 + 2.0 ** -16) * (v * cdf).abs()).all()
    # dbias of one node with dy = 1 is the slope
    one = torch.ones((1, C), dtype=BF, device=dev)
    _, _, db = binding.group_norm_bwd(one, x[:1].contiguous(), zero, z, mean, rstd, C // cg,
                                      "gelu")
    part = v * torch.exp(-0.5 * v * v) / (2 * torch.pi) ** 0.5
    slope = cdf + part
    assert ((db.double() - slope).abs()
            <= 2.0 ** -8 * slope.abs() + 2.0 ** -16 * (cdf + part.abs())).all()
    binding.check_status()
