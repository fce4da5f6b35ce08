"""Refusals of the operators around the attention, checked on the host: the
entry points return a status before they touch a device, and the binding
raises on tensors it cannot pass."""
import ctypes

import pytest
import torch

from graph_transformer_sparse_kmip_b200 import binding

INVALID, UNSUP = 1, 2
A = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from graph_transformer_sparse_kmip_b200 import build
    build.build()
    return binding.load()


def _rotary(lib, x=A, x_row=64, x_head=32, pos=A, pos_type=0, axes=2, freq=A, axis=A, pairs=16,
            inter=0, N=4, H=2, d=32, out=2 * A, out_row=64, out_head=32, dtype=0):
    return lib.kmip_rotary(x, x_row, x_head, pos, pos_type, axes, freq, axis, pairs, inter, 0, N,
                           H, d, out, out_row, out_head, None, dtype)


def test_rotary_refusals(lib):
    for kw in (dict(N=-1), dict(N=1 << 31), dict(H=0), dict(d=0), dict(axes=0), dict(pairs=-1),
               dict(pairs=17), dict(dtype=2), dict(pos_type=3), dict(x=None), dict(out=None),
               dict(pos=None), dict(freq=None), dict(axis=None), dict(x=A + 1), dict(out=A + 1),
               dict(inter=1, x=A + 2), dict(dtype=1, x=A + 2), dict(x_row=-64), dict(x_head=-1),
               # in place needs the same strides
               dict(out=A, out_head=64, out_row=128),
               # heads or rows of the output that share elements
               dict(out_head=31), dict(out_row=63), dict(out_row=0), dict(H=1, out_row=16),
               dict(out_row=32, out_head=100)):
        assert _rotary(lib, **kw) == INVALID, kw
    for kw in (dict(d=33), dict(d=514), dict(H=4097, out_row=4097 * 32), dict(axes=65),
               dict(inter=1, x_row=65), dict(inter=1, x_head=33)):
        assert _rotary(lib, **kw) == UNSUP, kw
    assert _rotary(lib, N=0, x=None, out=None, pos=None) == 0


def _norm_fwd(lib, x=A, w=A, b=A, off=None, N=8, C=32, groups=4, eps=1e-5, act=1, y=A, mean=A,
              rstd=A, G=1, dtype=0):
    return lib.kmip_group_norm_fwd(x, w, b, off, N, C, groups, eps, act, y, mean, rstd, None, G,
                                   dtype)


def _norm_bwd(lib, dy=A, x=A, w=A, b=A, off=None, mean=A, rstd=A, N=8, C=32, groups=4, act=1,
              dx=2 * A, dw=A, db=A, G=1, dtype=0):
    return lib.kmip_group_norm_bwd(dy, x, w, b, off, mean, rstd, N, C, groups, act, dx, dw, db,
                                   None, G, dtype)


def test_group_norm_refusals(lib):
    nan, inf = float("nan"), float("inf")
    both = (dict(N=-1), dict(N=1 << 31), dict(C=0), dict(groups=0), dict(groups=5),
            dict(groups=64), dict(act=4), dict(act=-1), dict(dtype=3), dict(off=A, G=0),
            dict(x=None), dict(w=None), dict(b=None), dict(mean=None), dict(rstd=None),
            dict(x=A + 1), dict(dtype=1, w=A + 2))
    for kw in both + (dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(y=None)):
        assert _norm_fwd(lib, **kw) == INVALID, kw
    for kw in both + (dict(dy=None), dict(dx=None), dict(dw=None), dict(db=None), dict(dx=A)):
        assert _norm_bwd(lib, **kw) == INVALID, kw
    for kw in (dict(C=65537, groups=1), dict(N=(1 << 31) - 1), dict(N=1 << 30, C=2048),
               dict(off=A, G=(1 << 31) - 1), dict(off=A, N=1 << 28, G=(1 << 31) - (1 << 22))):
        assert _norm_fwd(lib, **kw) == UNSUP and _norm_bwd(lib, **kw) == UNSUP, kw


def _ffn_fwd(lib, x=A, wg=A, wu=A, wd=A, N=8, C=32, F=64, act=1, y=2 * A, dtype=0):
    return lib.kmip_ffn_fwd(x, wg, wu, wd, N, C, F, act, y, None, dtype)


def _ffn_bwd(lib, dy=A, x=A, wg=A, wu=A, wd=A, N=8, C=32, F=64, act=1, dx=2 * A, dwg=3 * A,
             dwu=4 * A, dwd=5 * A, dtype=0):
    return lib.kmip_ffn_bwd(dy, x, wg, wu, wd, N, C, F, act, dx, dwg, dwu, dwd, None, dtype)


def test_ffn_refusals(lib):
    both = (dict(N=-1), dict(N=1 << 31), dict(C=0), dict(F=0), dict(act=4), dict(act=-1),
            dict(dtype=2), dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None),
            dict(x=A + 8), dict(wg=A + 2), dict(wd=A + 4))
    for kw in both + (dict(y=None), dict(y=A + 8)):
        assert _ffn_fwd(lib, **kw) == INVALID, kw
    for kw in both + (dict(dy=None), dict(dx=None), dict(dwg=None), dict(dwu=None),
                      dict(dwd=None), dict(dx=A + 8), dict(dwd=A + 8)):
        assert _ffn_bwd(lib, **kw) == INVALID, kw
    for kw in (dict(C=36), dict(F=60), dict(C=65544), dict(F=65544), dict(N=(1 << 31) - 1),
               dict(N=1 << 30, F=65536)):
        assert _ffn_fwd(lib, **kw) == UNSUP and _ffn_bwd(lib, **kw) == UNSUP, kw
    assert _ffn_fwd(lib, N=0, x=None, y=None) == 0


def test_ffn_refuses_outputs_that_overlap(lib):
    # x, y and their gradients take 512 bytes here, a weight 4,096
    B = 6 * A
    for kw in (dict(y=A), dict(x=B, y=B + 496), dict(x=B, y=B - 496), dict(wg=B, y=B + 4080),
               dict(wu=B, y=B - 496), dict(wd=B, y=B + 16)):
        assert _ffn_fwd(lib, **kw) == INVALID, kw
    for kw in (dict(dx=A), dict(x=B, dx=B + 496), dict(dy=B, dx=B - 496), dict(wd=B, dx=B + 4080),
               dict(dwg=A), dict(dwu=3 * A), dict(dwd=4 * A + 4080), dict(dwg=2 * A + 496),
               dict(wu=B, dwu=B), dict(dy=B, dwd=B - 4080)):
        assert _ffn_bwd(lib, **kw) == INVALID, kw


def test_binding_refuses_what_it_cannot_pass():
    x = torch.zeros(4, 2, 32)
    pos, freq = torch.zeros(4, 2), torch.zeros(16, dtype=torch.float64)
    axis = torch.zeros(16, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.rotary(x, pos, freq, axis)
    with pytest.raises(ValueError, match="adjacent"):
        binding.rotary(x.transpose(1, 2), pos, freq, axis)
    with pytest.raises(TypeError, match="position"):
        binding.rotary(x, pos.double(), freq, axis)
    with pytest.raises(ValueError, match="pos"):
        binding.rotary(x, pos[:3], freq, axis)
    with pytest.raises(ValueError, match="freq"):
        binding.rotary(x, pos, freq.float(), axis)
    with pytest.raises(ValueError, match="axis"):
        binding.rotary(x, pos, freq, axis[:8])
    y, w = torch.zeros(6, 32), torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.group_norm_fwd(y, w, w, 4)
    with pytest.raises(ValueError, match="N, C"):
        binding.group_norm_fwd(y[0], w, w, 4)
    with pytest.raises(ValueError, match="graph_offsets"):
        binding.group_norm_fwd(y, w, w, 4, graph_offsets=torch.tensor([0, 6]))
    g, d = torch.zeros(64, 32), torch.zeros(32, 64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.ffn_fwd(y, g, g, d)
    with pytest.raises(ValueError, match="expected"):
        binding.ffn_fwd(y, g[0], g, d)


def test_host_module_refuses_what_is_not_a_tensor(lib):
    x, w = torch.zeros(4, 32), torch.zeros(64, 32)
    h = torch.zeros(4, 2, 32)
    for call in (lambda: binding.rotary(h, None, None, None),
                 lambda: binding.rotary([0.0], h, h, h),
                 lambda: binding.group_norm_fwd(x, 1.0, None, 4),
                 lambda: binding.group_norm_fwd(x, None, None, "4"),
                 lambda: binding.group_norm_fwd(x, None, None, 4, "small"),
                 lambda: binding.group_norm_bwd(None, x, None, None, x, x, 4),
                 lambda: binding.ffn_fwd(x, w, w, None),
                 lambda: binding.ffn_bwd(None, x, w, w, w.T.contiguous()),
                 lambda: binding.load_host().rotary(h)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: binding.group_norm_fwd(h, None, None, 4),
                 lambda: binding.group_norm_fwd(x, None, None, -4),
                 lambda: binding.group_norm_fwd(x, None, None, 1 << 31),
                 lambda: binding.group_norm_fwd(x, None, None, 4, act="tanh"),
                 lambda: binding.group_norm_fwd(x, None, None, 4, graph_offsets=torch.zeros(3)),
                 lambda: binding.ffn_fwd(h, w, w, w),
                 lambda: binding.ffn_fwd(x, w, w, w.T.contiguous())):
        with pytest.raises(ValueError):
            call()


def test_rotary_tables_made_in_inference_mode_can_train():
    """A layer that answers first and trains later keeps its tables."""
    from graph_transformer_sparse_kmip_b200.layer import AxisRotary
    r = AxisRotary(32, 2)
    with torch.inference_mode():
        freq, axis = r.tables("cpu")
    assert not freq.is_inference() and not axis.is_inference()
    w = torch.ones(16, dtype=torch.float64, requires_grad=True)
    (w * freq).sum().backward()
    assert torch.equal(w.grad, freq)


def test_module_refusals():
    from graph_transformer_sparse_kmip_b200.layer import AxisRotary, GraphGroupNorm
    for kw in (dict(axes=0), dict(axes=-1), dict(axes=2, sections=[8]), dict(axes=1, pairs=17),
               dict(axes=2, sections=[-1, 4])):
        with pytest.raises(ValueError):
            AxisRotary(32, **kw)
    for channels, groups in ((32, 0), (32, 5), (32, -4)):
        with pytest.raises(ValueError):
            GraphGroupNorm(channels, groups)


def test_rotary_refuses_an_out_that_overlaps(lib):
    # heads of 32 elements (64 bytes), two to a row of 64: x takes 512 bytes
    for kw in (dict(out=A + 64), dict(out=A + 2), dict(out=A - 2), dict(out=A + 128),
               dict(out=A - 128), dict(out=A + 448), dict(out=A - 448), dict(out=A + 510),
               # rows of 128 elements, the other half of each free
               dict(x_row=128, out_row=128, out=A + 64), dict(x_row=128, out_row=128, out=A + 126),
               dict(x_row=128, out_row=128, out=A + 256), dict(x_row=128, out_row=128, out=A - 66),
               dict(x_row=128, out_row=128, out=A + 256 + 130),
               # heads outermost
               dict(x_row=32, x_head=128, out_row=32, out_head=128, out=A + 192),
               dict(x_row=32, x_head=128, out_row=32, out_head=128, out=A - 256),
               # other strides: by the ranges
               dict(x_row=128, out=A + 128), dict(out_row=128, out=A - 256),
               dict(x_head=0, x_row=32, out=A + 64),
               # one row, one head
               dict(N=1, out=A + 64), dict(N=1, out=A + 32), dict(H=1, N=1, out=A + 62),
               dict(H=1, x_row=64, out_row=64, out=A + 62)):
        assert _rotary(lib, **kw) == INVALID, kw


def test_rotary_overlap_rule_against_sets_of_elements(tmp_path):
    """The rule itself, compiled on the host, for all small layouts."""
    import os
    import re
    import subprocess
    from graph_transformer_sparse_kmip_b200.build import CSRC, CXX
    text = open(os.path.join(CSRC, "kmip_rotary.cu")).read()
    rule = re.search(r"bool shares_elements\(.*?\n}\n", text, re.S).group(0)
    src, so = tmp_path / "rule.cpp", tmp_path / "rule.so"
    src.write_text("#include <cstdint>\n" + rule + """
extern "C" bool rule(int64_t delta, int64_t N, int64_t H, int64_t d, int64_t a, int64_t b,
                     int64_t c, int64_t e) { return shares_elements(delta, N, H, d, a, b, c, e); }
""")
    subprocess.run([CXX, "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    fn = ctypes.CDLL(str(so)).rule
    fn.argtypes, fn.restype = [ctypes.c_int64] * 8, ctypes.c_bool
    seen = [0, 0]
    for N, H, d in ((1, 1, 2), (3, 1, 2), (1, 3, 2), (3, 2, 2), (2, 3, 4)):
        for row, head in ((H * d, d), (2 * H * d, d), (2 * H * d + 1, d + 1), (d, N * d),
                          (2 * d, 2 * N * d + 3)):
            if N == 1:
                row = 0
            if H == 1:
                head = 0
            x = {n * row + h * head + e for n in range(N) for h in range(H) for e in range(d)}
            for delta in range(-60, 61):
                if delta == 0:
                    continue
                meet = any(v + delta in x for v in x)
                assert fn(delta, N, H, d, row, head, row, head) == meet, (N, H, d, row, head, delta)
                seen[meet] += 1
    assert min(seen) > 100


def test_group_norm_refuses_outputs_that_overlap(lib):
    # x, y, dy and dx take 512 bytes here, parameters 64, statistics 16
    B = 8 * A
    fwd = dict(x=A, w=2 * A, b=3 * A, y=4 * A, mean=5 * A, rstd=6 * A)
    for kw in (dict(y=A + 2), dict(y=A - 510), dict(y=2 * A + 62), dict(b=B, y=B),
               dict(mean=6 * A), dict(mean=6 * A + 12), dict(rstd=4 * A + 508), dict(mean=A + 508),
               dict(rstd=2 * A), dict(y=A, mean=A + 16), dict(off=B, y=B + 4),
               dict(off=B, mean=B + 4), dict(rstd=A - 12)):
        assert _norm_fwd(lib, **{**fwd, **kw}) == INVALID, kw
    bwd = dict(dy=A, x=2 * A, w=3 * A, b=4 * A, mean=5 * A, rstd=6 * A, dx=7 * A, dw=9 * A,
               db=10 * A)
    for kw in (dict(dx=2 * A), dict(dx=2 * A + 16), dict(dx=A + 16), dict(dx=A - 510),
               dict(dw=10 * A), dict(db=9 * A + 62), dict(dw=3 * A), dict(db=4 * A + 2),
               dict(dw=7 * A + 510), dict(db=2 * A), dict(dw=A), dict(dx=A, dw=A + 32),
               dict(dx=5 * A + 12), dict(db=6 * A), dict(off=B, dw=B + 4), dict(off=B, dx=B - 508)):
        assert _norm_bwd(lib, **{**bwd, **kw}) == INVALID, kw


def test_host_module_belongs_to_its_torch_and_python(lib, monkeypatch):
    """One that was built for others is not loaded, and named as what to build."""
    import os
    import sysconfig
    from graph_transformer_sparse_kmip_b200 import build
    here = build.host_path()
    assert os.path.exists(here) and binding.load_host() is binding.load_host()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0")
        other = build.host_path()
        assert other != here
        m.setattr(binding, "_host", None)
        with pytest.raises(ImportError, match="build it"):
            binding.load_host()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-999")
        assert build.host_path() not in (here, other)
    assert build.host_path() == here
