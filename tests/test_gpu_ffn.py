"""Gated feed-forward block, forward and backward, against fp64.

Every tolerance is an interval bound carried through the formulas.  With r the
half step of the type that h, dA and dB are rounded to (fp32: 2^-22 for the
few fp32 operations of the activation), and acc(K) the relative error of a
K-long sum of products against the sum of their sizes -- tensor cores: one
truncation (2^-23) per 16 products, which are exact; fp32: one rounding (2^-24)
per product, splits included in the spare 16 --

  ta = acc(C) |x| |Wg|^T,  tb, tdh likewise
  th  = 1.13 ta (|b| + tb) + |f| tb + r |h|         slopes of silu, gelu <= 1.13
  tdA = |g| (|b| tdh + |dh| tb) + |dh b| ta + r |dA|    (slope of slope <= 1;
        relu: the whole term where |a| <= ta)
  tdB = |f| tdh + 1.13 |dh| ta + r |dB|
  ty  = th |Wd|^T + acc(F) |h| |Wd|^T + half |y|, and so on.

The fast bf16 activation adds 2^-18 of its value (inside 1.02 r).
"""
import pytest
import torch

from graph_transformer_sparse_kmip_b200 import binding

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


def _case(N, C, F, dtype, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)

    def n(*s):
        return torch.randn(s, generator=g, device=dev)

    return ((n(N, C)).to(dtype), (n(F, C) / C ** 0.5).to(dtype), (n(F, C) / C ** 0.5).to(dtype),
            (n(C, F) / F ** 0.5).to(dtype), n(N, C).to(dtype))


def _reference(x, wg, wu, wd, dy, act):
    dtype = x.dtype
    bf = dtype == BF
    half = torch.finfo(dtype).eps / 2
    r = 1.02 * half if bf else 2.0 ** -22
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    (N, C), F = x.shape, wg.shape[0]

    def acc(K):
        return (K / 16 + 4) * 2.0 ** -23 if bf else (K + 16) * 2.0 ** -24

    fn = torch.nn.functional
    a = (x @ wg.T).requires_grad_(True)
    f = {"none": lambda t: t * 1.0, "silu": fn.silu, "gelu": fn.gelu, "relu": fn.relu}[act](a)
    g, = torch.autograd.grad(f.sum(), a)
    a, f = a.detach(), f.detach()
    b, dh = x @ wu.T, dy @ wd
    h, da, db = f * b, dh * b * g, dh * f
    X, G, U, D, Y = (t.abs() for t in (x, wg, wu, wd, dy))
    ta, tb, tdh = acc(C) * (X @ G.T), acc(C) * (X @ U.T), acc(C) * (Y @ D)
    th = 1.13 * ta * (b.abs() + tb) + f.abs() * tb + r * h.abs()
    bend = (dh * b).abs() * (ta if act != "relu" else (a.abs() <= ta).double())
    tda = g.abs() * (b.abs() * tdh + dh.abs() * tb) + bend + r * da.abs()
    tdb = f.abs() * tdh + 1.13 * dh.abs() * ta + r * db.abs()
    ref = dict(y=h @ wd.T, dx=da @ wg + db @ wu, dwg=da.T @ x, dwu=db.T @ x, dwd=dy.T @ h)
    H, A, B = h.abs(), da.abs(), db.abs()
    tol = dict(y=th @ D.T + acc(F) * (H @ D.T),
               dx=tda @ G + tdb @ U + acc(2 * F) * (A @ G + B @ U),
               dwg=tda.T @ X + acc(N) * (A.T @ X), dwu=tdb.T @ X + acc(N) * (B.T @ X),
               dwd=Y.T @ th + acc(N) * (Y.T @ H))
    return ref, {k: v + half * ref[k].abs() for k, v in tol.items()}


def _run(x, wg, wu, wd, dy, act):
    y = binding.ffn_fwd(x, wg, wu, wd, act)
    dx, dwg, dwu, dwd = binding.ffn_bwd(dy, x, wg, wu, wd, act)
    binding.check_status()
    return dict(y=y, dx=dx, dwg=dwg, dwu=dwu, dwd=dwd)


def _check(args, act):
    got = _run(*args, act)
    ref, tol = _reference(*args, act)
    for k, v in got.items():
        err = (v.double() - ref[k]).abs()
        assert v.dtype == args[0].dtype and v.shape == ref[k].shape
        assert (err <= tol[k]).all(), (k, (err - tol[k]).max().item(), (err > tol[k]).sum().item())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,C,F", [
    (1, 8, 8), (1, 128, 344), (3, 40, 96), (16, 64, 128), (17, 128, 512), (64, 264, 136),
    (127, 128, 64), (128, 256, 256), (129, 8, 1000), (256, 64, 128), (257, 520, 72),
    (1000, 128, 344), (700, 328, 264), (2049, 16, 24)])
def test_sizes(dev, dtype, N, C, F):
    _check(_case(N, C, F, dtype, dev, seed=N + C), "silu")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "gelu", "relu"])
def test_activations(dev, dtype, act):
    _check(_case(300, 136, 200, dtype, dev, seed=3), act)


@pytest.mark.parametrize("dtype,N,C,F", [(BF, 40000, 128, 512), (BF, 9000, 1024, 1408),
                                         (F32, 20000, 64, 128), (F32, 3000, 512, 1024)])
def test_large(dev, dtype, N, C, F):
    _check(_case(N, C, F, dtype, dev, seed=5), "silu")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bits_repeat(dev, dtype):
    args = _case(5000, 128, 344, dtype, dev)
    first = _run(*args, "silu")
    for _ in range(3):
        for k, v in _run(*args, "silu").items():
            assert torch.equal(v, first[k]), k


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_do_not_meet(dev, dtype):
    """A NaN row spoils its own output rows and every weight gradient it
    reaches, and no other row."""
    x, wg, wu, wd, dy = _case(300, 64, 128, dtype, dev)
    x[150] = float("nan")
    got = _run(x, wg, wu, wd, dy, "silu")
    for k in ("y", "dx"):
        bad = torch.isnan(got[k]).any(1)
        assert bad[150] and bad.sum() == 1
    assert torch.isnan(got["dwg"]).all() and torch.isnan(got["dwd"]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_a_gate_without_a_number_stays_alone(dev, dtype, act):
    """Rows of Wg that hold a NaN spoil y and dx, and of the weights' gradients
    their own rows only."""
    x, wg, wu, wd, dy = _case(300, 64, 136, dtype, dev)
    before = binding.ffn_bwd(dy, x, wg, wu, wd, act)
    bad = [6, 33, 135]
    rest = [f for f in range(136) if f not in bad]
    wg[bad, 3] = float("nan")
    dx, dwg, dwu, dwd = binding.ffn_bwd(dy, x, wg, wu, wd, act)
    assert torch.equal(dwg[rest], before[1][rest]) and torch.equal(dwu[rest], before[2][rest])
    assert torch.equal(dwd[:, rest], before[3][:, rest])
    assert dwu[bad].isnan().all() and dx.isnan().all()
    assert binding.ffn_fwd(x, wg, wu, wd, act).isnan().all()
    binding.check_status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_rows(dev, dtype):
    x, wg, wu, wd, dy = _case(0, 64, 128, dtype, dev)
    got = _run(x, wg, wu, wd, dy, "silu")
    assert got["y"].shape == got["dx"].shape == (0, 64)
    for k in ("dwg", "dwu", "dwd"):
        assert (got[k] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_side_stream_and_captured_graphs(dev, dtype):
    """Two captured steps on two streams at once, replayed with new inputs."""
    work = []
    for seed in (1, 2):
        args = _case(900, 128, 264, dtype, dev, seed=seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _run(*args, "silu")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = binding.ffn_fwd(*args[:4], "silu")
            grads = binding.ffn_bwd(args[4], *args[:4], "silu")
        work.append((graph, side, args, dict(zip(("y", "dx", "dwg", "dwu", "dwd"), (y,) + grads))))
    for _, _, args, _ in work:
        args[0].mul_(0.5)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, side, _, _ in work:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, args, got in work:
        for k, v in _run(*args, "silu").items():
            assert torch.equal(v, got[k]), k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 3, 16])
def test_few_rows_see_the_projections_of_their_own_call(dev, dtype, N):
    """Calls of a few rows in close succession, each with the scratch of the one
    before it: the second kernel starts before the first has written."""
    g = torch.Generator(device=dev).manual_seed(N)
    _, wg, wu, wd, _ = _case(1, 1024, 2816, dtype, dev)
    xs = [torch.randn((N, 1024), generator=g, device=dev).to(dtype) for _ in range(8)]
    want = []
    for x in xs:
        want.append(binding.ffn_fwd(x, wg, wu, wd))
        torch.cuda.synchronize()
    for _ in range(20):
        got = [binding.ffn_fwd(x, wg, wu, wd) for x in xs]
        for a, c in zip(got, want):
            assert torch.equal(a, c)
    binding.check_status()


@pytest.mark.parametrize("N", [1, 20])
def test_gelu_of_every_value(dev, N):
    """x = e_0, Wu's first column 1 and Wd the identity hand out gelu of Wg's
    first column: roundings to bf16 (twice the same) and 2^-16 of the value."""
    z = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(BF)
    z = z[(z.float() >= -12.0) & (z.float() <= -0.5)]
    z = z[: z.numel() // 8 * 8].to(dev)
    F = z.numel()
    x, wg, wu = (torch.zeros((n, F), dtype=BF, device=dev) for n in (N, F, F))
    x[:, 0], wg[:, 0], wu[:, 0] = 1.0, z, 1.0
    y = binding.ffn_fwd(x, wg, wu, torch.eye(F, dtype=BF, device=dev), "gelu")
    ref = z.double() * 0.5 * torch.special.erfc(-z.double() / 2 ** 0.5)
    assert ((y.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs()).all()
    binding.check_status()
