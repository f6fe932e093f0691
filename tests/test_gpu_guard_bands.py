"""Every buffer of a call stands between guard bands of NaN: the linear layer and the
group normalisation through the C entry points, on every path. A value read past an
end turns up in a result, a value written past one in a band; inputs stay as they
are, and what a workspace held before does not matter."""
import ctypes

import pytest
import torch

import deformable_convolution_dcn_b200 as dcn
import op_reference as ref

pytestmark = pytest.mark.gpu

BAND = 1 << 16  # bytes on either side
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


class Pen:
    """`shape` values of `dtype` between two bands; all bytes are 0xff (NaN in either type)."""

    def __init__(self, shape, dtype, values=None, shift=0):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((n + 2 * BAND,), 0xFF, dtype=torch.uint8, device="cuda")
        self.first, self.last = BAND + shift, BAND + shift + n
        self.t = self.raw[self.first:self.last].view(dtype).view(shape)
        self.kept = None
        if values is not None:
            self.t.copy_(values)
            self.kept = self.t.clone()

    @property
    def p(self):
        return ctypes.c_void_p(self.t.data_ptr())

    def check(self, name):
        assert bool((self.raw[:self.first] == 0xFF).all()) and bool((self.raw[self.last:] == 0xFF).all()), name
        if self.kept is not None:
            assert torch.equal(self.t, self.kept), name


def p(pen):
    return None if pen is None else pen.p


def run(fn, *args):
    rc = fn(*args, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0, dcn._load().dcn_last_error_string().decode()
    dcn.check_status()


def normal(g, dtype, *shape, k=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * k).to(TYPES[dtype])


# a few rows, single values and odd sizes, one output (rows on the tensor cores' columns), a result written transposed, split
# reductions, several tiles, rows that are not whole vectors
LINEAR = [(5, 600, 520), (1, 1, 8), (8, 331, 264), (17, 33, 65), (129, 136, 72), (19005, 1, 12544), (262144, 1, 512), (9, 331, 512),
          (64, 3, 4096), (33, 24, 4104), (2500, 40, 48), (20000, 8, 64), (9999, 520, 136), (9999, 521, 135)]


@pytest.mark.parametrize("size", LINEAR, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shift", [0, 4], ids=["aligned", "shifted"])
def test_linear_between_guard_bands(size, dtype, shift):
    M, N, K = size
    t = TYPES[dtype]
    lib, g = dcn._load(), torch.Generator(device="cuda").manual_seed(22)
    x = Pen((M, K), t, normal(g, dtype, M, K), shift)
    w = Pen((N, K), t, normal(g, dtype, N, K, k=K ** -0.5), shift)
    b, r = Pen((N,), t, normal(g, dtype, N), shift), Pen((M, N), t, normal(g, dtype, M, N), shift)
    gy = Pen((M, N), t, normal(g, dtype, M, N), shift)
    for act, bias, residual in (("relu", b, r), ("gelu", b, None), ("none", None, r)):
        q = dcn.LinearParams(M, N, K, dcn.ACTIVATIONS[act], int(dtype == "bf16"), 0)
        y, z = Pen((M, N), t, shift=shift), Pen((M, N), t, shift=shift) if act == "gelu" else None
        ws = Pen((dcn.linear_workspace_size(q, dcn.OP_FORWARD),), torch.uint8)
        run(lib.dcn_linear_forward, ctypes.byref(q), x.p, w.p, p(bias), p(residual), y.p, p(z), ws.p, ws.t.numel())
        want = ref.linear_forward(x.t, w.t, bias and bias.t, residual and residual.t, act)
        ref.check("y", y.t, *want["y"])
        if z:
            ref.check("z", z.t, *want["z"])
        kept = y if act == "relu" else z
        if kept:
            kept.kept = kept.t.clone()
        out = [Pen((M, K), t, shift=shift), Pen((N, K), torch.float32, shift=shift), Pen((N,), torch.float32, shift=shift),
               Pen((M, N), t, shift=shift)]
        ws2 = Pen((dcn.linear_workspace_size(q, dcn.OP_BACKWARD),), torch.uint8)
        run(lib.dcn_linear_backward, ctypes.byref(q), x.p, w.p, p(kept), gy.p, *(o.p for o in out), ws2.p, ws2.t.numel())
        want = ref.linear_backward(x.t, w.t, kept and kept.t, gy.t, act)
        for o, k in zip(out, want):
            ref.check(k, o.t, *want[k])
        for name, pen in dict(x=x, w=w, b=b, r=r, gy=gy, y=y, z=z, ws=ws, ws2=ws2, gx=out[0], gw=out[1], gb=out[2],
                              gr=out[3]).items():
            if pen:
                pen.check(name)


# a cluster's maps, the ring's, the queue's (single values; over 1024 channels; groups wider than a unit), many samples
NORM = [(1, 7, 10, 256, 32), (2, 40, 41, 96, 8), (5, 3, 3, 24, 2), (3, 129, 131, 96, 32), (200, 33, 31, 64, 8),
        (1, 257, 129, 1024, 32), (3, 65, 67, 33, 3), (1, 3, 3, 4104, 2), (1, 64, 64, 1088, 64), (2, 1, 1, 64, 8),
        (700, 2, 3, 40, 8), (1, 300, 301, 3, 1)]


@pytest.mark.parametrize("size", NORM, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shift", [0, 4], ids=["aligned", "shifted"])
def test_group_norm_between_guard_bands(size, dtype, shift):
    B, H, W, C, groups = size
    t = TYPES[dtype]
    lib, g = dcn._load(), torch.Generator(device="cuda").manual_seed(23)
    x, gy = (Pen((B, H, W, C), t, normal(g, dtype, B, H, W, C), shift) for _ in range(2))
    ga, be = Pen((C,), t, 1 + normal(g, dtype, C, k=0.3), shift), Pen((C,), t, normal(g, dtype, C, k=0.3), shift)
    q = dcn.NormParams(B, H, W, C, groups, EPS, dcn.ACTIVATIONS["silu"], int(dtype == "bf16"), 0)
    aligned = dcn.OP_ALIGNED if shift == 0 else 0
    y, stats = Pen((B, H, W, C), t, shift=shift), Pen((B, groups, 2), torch.float32, shift=shift)
    ws = Pen((dcn.group_norm_workspace_size(q, dcn.OP_FORWARD | aligned),), torch.uint8)
    run(lib.dcn_group_norm_forward, ctypes.byref(q), x.p, ga.p, be.p, y.p, stats.p, ws.p, ws.t.numel())
    want = ref.norm_forward(x.t, ga.t, be.t, groups, EPS, "silu")
    ref.check("mean", stats.t[..., 0], *want["mean"])
    ref.check("rstd", stats.t[..., 1], *want["rstd"])
    ref.check("y", y.t, *want["y"])
    stats.kept = stats.t.clone()
    gx, gg, gb = Pen((B, H, W, C), t, shift=shift), Pen((C,), torch.float32, shift=shift), Pen((C,), torch.float32, shift=shift)
    ws2 = Pen((dcn.group_norm_workspace_size(q, dcn.OP_BACKWARD | aligned),), torch.uint8)
    run(lib.dcn_group_norm_backward, ctypes.byref(q), x.p, ga.p, be.p, stats.p, gy.p, gx.p, gg.p, gb.p, ws2.p, ws2.t.numel())
    want = ref.norm_backward(x.t, ga.t, be.t, stats.t, gy.t, groups, "silu")
    for pen, k in ((gx, "grad_x"), (gg, "grad_gamma"), (gb, "grad_beta")):
        ref.check(k, pen.t, *want[k])
    for name, pen in dict(x=x, gy=gy, ga=ga, be=be, y=y, stats=stats, ws=ws, gx=gx, gg=gg, gb=gb, ws2=ws2).items():
        pen.check(name)
