"""Timed cases of the operators around k-MIP attention in a graph-transformer
layer: rotary positions with several axes, group norm per graph with an
activation, and the gated feed-forward block.

Formulas (fp32 or wider inside, one rounding at the end):

  rotary      angle[n, p] = pos[n, axis[p]] * freq[p], p < P pairs of every head;
              (u, v) -> (u cos - v sin, u sin + v cos); the backward pass (and
              "inverse") turns by the negative angle.
  group norm  x [N, C], channels last; mean and variance over the nodes of one
              graph and the C / groups channels of one group;
              y = act((x - mean) / sqrt(var + eps) * w + b).
  ffn         y = (act(x Wg^T) * (x Wu^T)) Wd^T, Wg, Wu [F, C], Wd [C, F].

``own`` False: ``run`` computes with elementary torch operations.  True: it
calls the package's entry points.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One node joins a stored graph: its query and key heads are turned
        # (4 heads of 32, image coordinates).  Latency.
        dict(name="rotary_one_node", op="rotary", N=1, H=8, d=32, rot=32, axes=2, pos="coords",
             packed=True, interleaved=False, inverse=False, dtype="bf16"),
        # 64 superpixel graphs of 300 to 600 nodes (28,072 in all): q and k
        # turned where the fused projection left them, by (x, y) in pixels.
        dict(name="rotary_superpixels", op="rotary", N=28072, H=8, d=32, rot=32, axes=2,
             pos="coords", packed=True, interleaved=False, inverse=False, dtype="bf16"),
        # A point cloud of 524,288 nodes, heads of 16, (x, y, z).
        dict(name="rotary_pointcloud", op="rotary", N=524288, H=8, d=16, rot=12, axes=3,
             pos="coords", packed=True, interleaved=True, inverse=False, dtype="bf16"),
        # Gradient of q and k for video patches at (time, height, width) far
        # along the time axis, fp32, wide heads.
        dict(name="rotary_video_bwd", op="rotary", N=100003, H=8, d=128, rot=128, axes=3,
             pos="grid", packed=False, interleaved=False, inverse=True, dtype="f32"),
        # The small check size: one graph of 1,024 nodes, fp32, inference.
        dict(name="norm_tiny", op="norm", sizes="one", G=1, N=1024, C=32, groups=4, act="silu",
             train=False, dtype="f32"),
        # Training step on 64 superpixel graphs, hidden width 128.
        dict(name="norm_batched_train", op="norm", sizes="ragged", G=64, N=28072, C=128, groups=8,
             act="silu", train=True, dtype="bf16"),
        # One graph of 31,623 nodes, an odd channel count, fp32 training.
        dict(name="norm_odd_train", op="norm", sizes="one", G=1, N=31623, C=345, groups=15,
             act="none", train=True, dtype="f32"),
        # The point cloud, inference, hidden width 256.
        dict(name="norm_pointcloud", op="norm", sizes="one", G=1, N=524288, C=256, groups=32,
             act="silu", train=False, dtype="bf16"),
        # One node through a wide block: the time to read the weights.
        dict(name="ffn_one_node", op="ffn", N=1, C=1024, F=2816, act="silu", train=False,
             dtype="bf16"),
        # The small check size in fp32, hidden width 128: training step.
        dict(name="ffn_tiny_train", op="ffn", N=1024, C=128, F=344, act="gelu", train=True,
             dtype="f32"),
        # One graph of 100,000 nodes, hidden 128: training step.
        dict(name="ffn_graph_train", op="ffn", N=100000, C=128, F=512, act="silu", train=True,
             dtype="bf16"),
        # One graph of 31,623 nodes through a wide block: training step.
        dict(name="ffn_wide_train", op="ffn", N=31623, C=1024, F=2816, act="silu", train=True,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "ffn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotary":
        d = rng.choice([16, 32, 40, 64, 128])
        axes = rng.choice([1, 2, 3, 4])
        rot = rng.choice([d, d, 2 * rng.randint(max(1, d // 4), d // 2)])
        H = rng.randint(1, 24)
        N = _log(rng, 1, min(524288, 48_000_000 // (H * d)))
        return dict(op=op, N=N, H=H, d=d, rot=rot, axes=axes, pos=rng.choice(["coords", "grid"]),
                    packed=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, dtype=dtype)
    if op == "norm":
        groups = rng.choice([1, 2, 4, 8, 16, 32])
        C = groups * rng.randint(1, max(1, 512 // groups))
        # at least 64 values in a group on average: with two or three the
        # gradient of x is what rounding leaves of equal terms
        least = -(-64 * groups // C)
        N = _log(rng, least, min(524288, 24_000_000 // C))
        sizes = rng.choice(["one", "ragged"])
        G = 1 if sizes == "one" else _log(rng, 1, max(1, min(2000, N // least)))
        return dict(op=op, sizes=sizes, G=G, N=N, C=C, groups=groups,
                    act=rng.choice(["none", "silu", "relu"]), train=rng.random() < 0.6,
                    dtype=dtype)
    C, F = 8 * _log(rng, 2, 128), 8 * _log(rng, 4, 352)
    top = 31623 if dtype == "bf16" else 4096
    return dict(op="ffn", N=_log(rng, 1, top), C=C, F=F, act=rng.choice(["silu", "gelu", "relu"]),
                train=rng.random() < 0.6, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _sections(pairs, axes):
    """Rotation pairs of each axis, as even as they go."""
    return [pairs // axes + (a < pairs % axes) for a in range(axes)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    s = dict(case)
    if case["op"] == "rotary":
        N, H, d, P = case["N"], case["H"], case["d"], case["rot"] // 2
        if case["packed"]:
            # q and k heads inside a fused projection's [N, (q | k | v)] rows
            v = max(1, H // 2)
            s["x"] = normal(N, H + v, d).to(dt)[:, :H]
        else:
            s["x"] = normal(N, H, d).to(dt)
        if case["pos"] == "coords":
            s["pos"] = torch.rand((N, case["axes"]), generator=g, device=dev) * 500.0
        else:
            s["pos"] = torch.randint(0, 200_000, (N, case["axes"]), generator=g, device=dev,
                                     dtype=torch.int32)
        freq, axis = [], []
        for a, n in enumerate(_sections(P, case["axes"])):
            freq += [10000.0 ** (-j / n) for j in range(n)]
            axis += [a] * n
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(axis, dtype=torch.int32, device=dev)
        return s
    if case["op"] == "norm":
        N, C, G = case["N"], case["C"], case["G"]
        if case["sizes"] == "one":
            off = torch.tensor([0, N], device=dev)
        else:
            # even sizes with a third of jitter
            cut = torch.arange(1, G, device=dev, dtype=torch.float64) * (N / G)
            cut += (torch.rand(G - 1, generator=g, device=dev, dtype=torch.float64) - 0.5) * (
                N / G * 0.66)
            cut = cut.round().long().clamp(0, N).sort().values
            off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), N)])
        s["offsets"] = off.to(torch.int32)
        scale = 0.5 + torch.rand(C, generator=g, device=dev)
        s["x"] = (normal(N, C) * scale + normal(C)).to(dt)
        s["w"] = (1.0 + 0.2 * normal(C)).to(dt)
        s["b"] = (0.2 * normal(C)).to(dt)
        if case["train"]:
            s["dy"] = normal(N, C).to(dt)
        return s
    N, C, F = case["N"], case["C"], case["F"]
    s["x"] = normal(N, C).to(dt)
    s["wg"] = (normal(F, C) / math.sqrt(C)).to(dt)
    s["wu"] = (normal(F, C) / math.sqrt(C)).to(dt)
    s["wd"] = (normal(C, F) / math.sqrt(F)).to(dt)
    if case["train"]:
        s["dy"] = normal(N, C).to(dt)
    return s


# ------------------------------------------------------------- plain forms
_EPS = 1e-5


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    return z


def _act_grad(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(
            -0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _plain_rotary(s):
    x, P = s["x"], s["rot"] // 2
    angle = s["pos"].double()[:, s["axis"].long()] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if s["inverse"]:
        sin = -sin
    xf = x.float()
    out = xf.clone(memory_format=torch.contiguous_format)
    if s["interleaved"]:
        u, v = xf[..., 0:2 * P:2], xf[..., 1:2 * P:2]
        out[..., 0:2 * P:2], out[..., 1:2 * P:2] = u * cos - v * sin, u * sin + v * cos
    else:
        u, v = xf[..., :P], xf[..., P:2 * P]
        out[..., :P], out[..., P:2 * P] = u * cos - v * sin, u * sin + v * cos
    return out.to(x.dtype)


def _plain_norm(s):
    x, off, groups = s["x"], s["offsets"].long(), s["groups"]
    N, C = x.shape
    G, cg = off.numel() - 1, C // groups
    n = off[1:] - off[:-1]
    gid = torch.repeat_interleave(torch.arange(G, device=x.device), n, output_size=N)
    count = (n * cg).clamp(min=1).double()

    def per_graph(t):                       # [N, C] -> [G, groups]
        rows = t.view(N, groups, cg).sum(-1, dtype=torch.float64).t()
        upto = torch.cat([rows.new_zeros(groups, 1), rows.cumsum(1)], 1)
        return ((upto[:, off[1:]] - upto[:, off[:-1]]) / count).t()

    def spread(t):                          # [G, groups] -> [N, C]
        return t.float()[gid].repeat_interleave(cg, 1)

    xf, w, b = x.float(), s["w"].float(), s["b"].float()
    mean = per_graph(xf)
    cen = xf - spread(mean)
    rstd = torch.rsqrt(per_graph(cen * cen) + _EPS)
    xhat = cen * spread(rstd)
    z = xhat * w + b
    y = _act(z, s["act"]).to(x.dtype)
    mean, rstd = mean.float(), rstd.float()
    if not s["train"]:
        return y, mean, rstd
    dz = s["dy"].float() * _act_grad(z, s["act"])
    t = dz * w
    dx = spread(rstd) * (t - spread(per_graph(t)) - xhat * spread(per_graph(t * xhat)))
    dw = (dz * xhat).sum(0, dtype=torch.float64)
    db = dz.sum(0, dtype=torch.float64)
    return y, mean, rstd, dx.to(x.dtype), dw.to(x.dtype), db.to(x.dtype)


def _plain_ffn(s):
    dt = s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
    a, b = x @ wg.t(), x @ wu.t()
    f = _act(a, s["act"])
    h = f * b
    y = (h @ wd.t()).to(dt)
    if not s["train"]:
        return y
    dy = s["dy"].float()
    dh = dy @ wd
    da, db = dh * b * _act_grad(a, s["act"]), dh * f
    dx = da @ wg + db @ wu
    return y, dx.to(dt), (da.t() @ x).to(dt), (db.t() @ x).to(dt), (dy.t() @ h).to(dt)


# --------------------------------------------------------------------- run
def run(s):
    if own:
        from graph_transformer_sparse_kmip_b200 import binding as kb
        if s["op"] == "rotary":
            return kb.rotary(s["x"], s["pos"], s["freq"], s["axis"], inverse=s["inverse"],
                             interleaved=s["interleaved"])
        if s["op"] == "norm":
            y, mean, rstd = kb.group_norm_fwd(s["x"], s["w"], s["b"], s["groups"], eps=_EPS,
                                              act=s["act"], graph_offsets=s["offsets"])
            if not s["train"]:
                return y, mean, rstd
            return (y, mean, rstd) + kb.group_norm_bwd(
                s["dy"], s["x"], s["w"], s["b"], mean, rstd, s["groups"], act=s["act"],
                graph_offsets=s["offsets"])
        y = kb.ffn_fwd(s["x"], s["wg"], s["wu"], s["wd"], act=s["act"])
        if not s["train"]:
            return y
        return (y,) + kb.ffn_bwd(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], act=s["act"])
    return {"rotary": _plain_rotary, "norm": _plain_norm, "ffn": _plain_ffn}[s["op"]](s)


# -------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    N = case["N"]
    if case["op"] == "rotary":
        P = case["rot"] // 2
        return {"bytes": 2 * e * N * case["H"] * case["d"] + 4 * N * case["axes"] + 12 * P,
                "flops": 6 * N * case["H"] * P}
    if case["op"] == "norm":
        C, stats = case["C"], 8 * case["G"] * case["groups"]
        rows = 5 if case["train"] else 2    # x, y and, for training, x, dy, dx
        return {"bytes": e * N * C * rows + stats + e * C * (4 if case["train"] else 2),
                "flops": N * C * (30 if case["train"] else 10)}
    C, F = case["C"], case["F"]
    per = 18 if case["train"] else 6
    rows, mats = (4, 6) if case["train"] else (2, 3)
    return {"bytes": e * (rows * N * C + mats * C * F), "flops": per * N * C * F}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits: complex products for the rotary positions,
    autograd for the gradients."""
    s = prepare(case, seed)
    if case["op"] == "rotary":
        x, P = s["x"].double(), case["rot"] // 2
        turn = s["pos"].double().index_select(1, s["axis"].long()) * s["freq"]
        turn = torch.polar(torch.ones_like(turn), -turn if case["inverse"] else turn)[:, None]
        head, rest = x[..., :2 * P], x[..., 2 * P:]
        if case["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (P, 2)).contiguous()) * turn
            out = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :P].contiguous(), head[..., P:].contiguous()) * turn
            out = torch.cat([z.real, z.imag], -1)
        return torch.cat([out, rest], -1)

    def act(z):
        f = torch.nn.functional
        return {"silu": f.silu, "gelu": f.gelu, "relu": f.relu, "none": lambda t: t}[case["act"]](z)

    if case["op"] == "norm":
        x = s["x"].double().requires_grad_(case["train"])
        w = s["w"].double().requires_grad_(case["train"])
        b = s["b"].double().requires_grad_(case["train"])
        groups, cg = case["groups"], case["C"] // case["groups"]
        ys, means, rstds = [], [], []
        for part in x.unflatten(1, (groups, cg)).split(s["offsets"].diff().tolist()):
            if part.shape[0]:
                var, mean = torch.var_mean(part, dim=(0, 2), correction=0)
            else:
                var = mean = x.new_zeros(groups)
            rstd = (var + _EPS) ** -0.5
            ys.append((part - mean[:, None]) * rstd[:, None])
            means.append(mean.detach())
            rstds.append(rstd.detach())
        y = act(torch.cat(ys).flatten(1) * w + b)
        head = (y.detach(), torch.stack(means), torch.stack(rstds))
        if not case["train"]:
            return head
        return head + torch.autograd.grad(y, (x, w, b), s["dy"].double())

    leaves = [s[k].double().requires_grad_(case["train"]) for k in ("x", "wg", "wu", "wd")]
    x, wg, wu, wd = leaves
    lin = torch.nn.functional.linear
    y = lin(act(lin(x, wg)) * lin(x, wu), wd)
    if not case["train"]:
        return y
    return (y.detach(),) + torch.autograd.grad(y, leaves, s["dy"].double())
