"""Sums over many nodes with integers that every type and accumulator holds
exactly: what a kernel leaves out, takes twice or takes from another row shows
in the last bit, at any length.

Feed-forward, act "none": rows of Wg and Wu and columns of Wd have a single
entry of +-1, x and dy are in -2 .. 2, so a, b, dh are too, h, dA, dB are in
-4 .. 4 and every sum stays under 2^24.  The outputs are those integers, rounded
once to the type.

Group norm, act "none", weight 1: with mean 0 and rstd 1 given to the backward,
xhat = x and dz = dy, and dweight and dbias are sums of integers.
"""
import pytest
import torch

from graph_transformer_sparse_kmip_b200 import binding
from graph_transformer_sparse_kmip_b200 import workloads as wl

BF, F32 = torch.bfloat16, torch.float32
STEP = 64  # rows of one step of the contraction over nodes


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    yield torch.device("cuda:0")
    torch.cuda.synchronize()
    binding.kmip_scratch_trim()  # other tests measure what the pool holds


def _integers(shape, dev, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=dev).double()


def _single(rows, cols, dev, seed):
    """[rows, cols], one entry of +-1 in each row."""
    g = torch.Generator(device=dev).manual_seed(seed)
    w = torch.zeros((rows, cols), dtype=torch.float64, device=dev)
    at = torch.randint(0, cols, (rows, 1), generator=g, device=dev)
    sign = torch.randint(0, 2, (rows, 1), generator=g, device=dev).double() * 2 - 1
    return w.scatter_(1, at, sign)


def _ffn_case(N, C, F, dev):
    return (_integers((N, C), dev, 1), _single(F, C, dev, 2), _single(F, C, dev, 3),
            _single(F, C, dev, 4).t().contiguous(), _integers((N, C), dev, 5))


def _ffn_sums(x, wg, wu, wd, dy):
    a, b, dh = x @ wg.T, x @ wu.T, dy @ wd
    h, da, db = a * b, dh * b, dh * a
    return dict(y=h @ wd.T, dx=da @ wg + db @ wu, dwg=da.T @ x, dwu=db.T @ x, dwd=dy.T @ h)


def _without(t, lo, n):
    return torch.cat([t[:lo], t[lo + n:]])


FFN = [(40000, 128, 512), (40001, 128, 512), (100003, 64, 136), (9000, 1024, 1408),
       (4097, 264, 520), (64, 128, 256), (17, 40, 96), (16, 40, 96), (3, 8, 8)]


@pytest.mark.parametrize("N,C,F", [(40000, 128, 512), (9000, 128, 256)])
def test_a_lost_step_shows_in_the_integers(N, C, F):
    """On the oracle: one step of the contraction left out, or one row taken
    twice, is seen in every gradient, rounded to bf16."""
    case = _ffn_case(N, C, F, "cpu")
    whole = _ffn_sums(*case)
    for lo in (0, N // 2 // STEP * STEP, N - STEP):
        x, wg, wu, wd, dy = case
        part = _ffn_sums(_without(x, lo, STEP), wg, wu, wd, _without(dy, lo, STEP))
        for k in ("dwg", "dwu", "dwd"):
            changed = (whole[k].to(BF) != part[k].to(BF)).float().mean()
            assert changed > 0.3, (k, lo, changed)
    twice = [torch.cat([t, t[N // 3: N // 3 + 1]]) if t.shape[0] == N else t for t in case]
    again = _ffn_sums(*twice)
    for k in ("dwg", "dwu", "dwd"):
        assert (whole[k].to(BF) != again[k].to(BF)).any(), k


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,C,F", FFN)
def test_feed_forward_sums(dev, dtype, N, C, F):
    case = _ffn_case(N, C, F, dev)
    want = _ffn_sums(*case)
    assert max(v.abs().max() for v in want.values()) < 2 ** 24
    x, wg, wu, wd, dy = (t.to(dtype) for t in case)
    got = dict(zip(("dx", "dwg", "dwu", "dwd"), binding.ffn_bwd(dy, x, wg, wu, wd, "none")),
               y=binding.ffn_fwd(x, wg, wu, wd, "none"))
    binding.check_status()
    for k, v in want.items():
        assert torch.equal(got[k], v.to(dtype)), k


NORM = [([0, 60001, 0, 1, 9000, 130], 256, 32), ([40000], 345, 15), ([20000, 50000], 130, 13),
        ([5000] * 10, 520, 65), ([300, 45, 0, 517, 129], 128, 8), ([30] * 2000, 155, 31),
        ([450] * 256, 128, 8), ([1], 64, 4), ([7, 0, 3000], 40, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,C,groups", NORM)
def test_group_norm_parameter_sums(dev, dtype, sizes, C, groups):
    N, G = sum(sizes), len(sizes)
    x, dy = _integers((N, C), dev, 6), _integers((N, C), dev, 7)
    ones = torch.ones(C, dtype=dtype, device=dev)
    mean = torch.zeros((G, groups), device=dev)
    _, dw, db = binding.group_norm_bwd(dy.to(dtype), x.to(dtype), ones, ones * 0, mean, mean + 1,
                                       groups, "none", wl.offsets_from_sizes(sizes).to(dev))
    binding.check_status()
    assert torch.equal(dw, (dy * x).sum(0).to(dtype))
    assert torch.equal(db, dy.sum(0).to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,C,groups", NORM)
def test_group_norm_means(dev, dtype, sizes, C, groups):
    """A mean of integers: a thread's mean of up to 2^12 values of at most 2 is
    rounded once a batch, 2^-23 at most each time, and those roundings go either
    way; the joins are fp64.  2^-21 of the values, and half a step of the mean.
    (One node of 69,000 with 8 channels a group left out: 2^-19 a unit.)"""
    N = sum(sizes)
    x = _integers((N, C), dev, 8)
    off = wl.offsets_from_sizes(sizes)
    _, mean, rstd = binding.group_norm_fwd(x.to(dtype), None, None, groups, 1e-5, "none",
                                           off.to(dev))
    binding.check_status()
    for g, part in enumerate(x.unflatten(1, (groups, C // groups)).split(sizes)):
        if not len(part):
            continue
        m = part.mean((0, 2))
        v = (part - m[:, None]).square().mean((0, 2))
        assert ((mean[g].double() - m).abs() <= 2.0 ** -21).all()
        # twice the mean's error times the mean, and as many roundings of squares
        assert ((1 / rstd[g].double().square() - 1e-5 - v).abs() <= 2.0 ** -18 * (v + 1e-5)).all()
