"""The linear layer at sizes that give a block of the persistent product kernel
several tiles, by CTA pairs and single CTAs, tiles of 64 to 256 columns, short and
long reductions; and the accuracy of long reductions by norm.

By norm: a float32 result is a sum of chunks of 128 products (bfloat16 results are
not looked at). Within one, the tensor cores cut the running sum off at each of
eight steps, by half a unit in the last place on average, of running sums that grow
evenly where all products are positive: at most 2^-23 (1/2) sum_i i/8 = 2.25 x 2^-23
of the chunk. The n chunks are added in registers, each sum off by 0.29 units rms of
a running sum that grows evenly: 0.29 sqrt(n/3) x 2^-23, 0.17 sqrt(n) x 2^-23. Twice
that chain, and what the split in three terms leaves out (2^-25 of a product), is
allowed. One product of a step further left out (2^-18, 1e-6 rms), or sums cut off
over the whole reduction (6e-5 of 12544 positive products), are not within it.
"""
import math

import pytest
import torch

import deformable_convolution_dcn_b200 as dcn
import op_reference as ref
from test_gpu_linear import check_backward, make

pytestmark = pytest.mark.gpu

# M, N, K, the columns and CTAs of a tile that they are here for
SIZES = [(19993, 1032, 264),   # 256, pairs: five tiles a pair
         (9999, 2056, 520),    # 256, pairs; with z 128
         (2048, 4096, 4096),   # 256, pairs: a long reduction, one slot a warp
         (19993, 1024, 72),    # 256, single
         (40003, 264, 64),     # 128, single: one stage a tile
         (30000, 64, 520),     # 64: half of the epilogue's warps have no columns
         (19993, 1031, 264),   # rows that are not whole vectors
         (700, 2048, 6144)]    # a split reduction of pairs
name = lambda s: "x".join(map(str, s))  # noqa: E731


def on_gpu(M, N, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    n = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(t)  # noqa: E731
    return dict(x=n(M, K), w=n(N, K, k=K ** -0.5), b=n(N), r=n(M, N), gy=n(M, N))


@pytest.mark.parametrize("size", SIZES, ids=name)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act,bias,residual,preact", [("relu", True, True, False), ("none", False, False, False),
                                                      ("gelu", True, False, True), ("silu", True, True, True)],
                         ids=["relu_shortcut", "plain", "gelu_z", "silu_z_shortcut"])
def test_linear_forward_of_several_tiles(size, dtype, act, bias, residual, preact):
    d = on_gpu(*size, dtype, 18)
    b, r = d["b"] if bias else None, d["r"] if residual else None
    want = ref.linear_forward(d["x"], d["w"], b, r, act)
    for _ in range(2):
        got = dcn.linear_forward(d["x"], d["w"], b, r, act, need_preact=preact)
        torch.cuda.synchronize()
        dcn.check_status()
        y = got[0] if preact else got
        ref.check("y", y, *want["y"])
        if preact:
            ref.check("z", got[1], *want["z"])
    if residual:  # y over the residual
        dcn.linear_forward(d["x"], d["w"], b, r, act, out=r)
        assert torch.equal(r, y)


@pytest.mark.parametrize("size,act", [((19993, 1032, 264), "relu"), ((9999, 2056, 520), "gelu"), ((512, 2048, 8192), "none"),
                                      ((1000, 2048, 4096), "silu"), ((20000, 256, 1024), "relu"),
                                      ((20011, 256, 1031), "gelu")], ids=lambda v: v if isinstance(v, str) else name(v))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_backward_of_several_tiles(size, act, dtype):
    check_backward(make(*size, dtype, seed=19), act)


def norm_off(got, want):
    return float((got.double() - want).norm() / want.norm())


def allowed(red):
    return 2.0 ** -23 * (2.25 + 2 * 0.17 * math.sqrt(red / 128)) + 2.0 ** -25


def product64(a, b):
    """a b^T in float64, in blocks of the reduction."""
    out = torch.zeros((a.shape[0], b.shape[0]), dtype=torch.float64, device=a.device)
    for k in range(0, a.shape[1], 8192):
        out += a[:, k:k + 8192].double() @ b[:, k:k + 8192].double().t()
    return out


@pytest.mark.parametrize("positive", [False, True], ids=["signed", "positive"])
@pytest.mark.parametrize("size", [(300, 264, 12544), (1000, 520, 4104), (64, 2056, 8200), (12544, 264, 72)], ids=name)
def test_linear_float32_accuracy_by_norm(size, positive):
    M, N, K = size
    d = on_gpu(M, N, K, "f32", 20)
    if positive:
        d = {k: v.abs() for k, v in d.items()}
    y = dcn.linear_forward(d["x"], d["w"])
    gx, gw, _, _ = dcn.linear_backward(d["x"], d["w"], None, d["gy"], "none", need_bias=False)
    torch.cuda.synchronize()
    dcn.check_status()
    assert norm_off(y, product64(d["x"], d["w"])) <= allowed(K)
    assert norm_off(gx, product64(d["gy"], d["w"].t())) <= allowed(N)
    assert norm_off(gw, product64(d["gy"].t(), d["x"].t())) <= allowed(M)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("size", [(12544, 264, 72), (5000, 512, 256), (4104, 65, 520)], ids=name)
def test_linear_bfloat16_parameter_gradients_by_norm(size, act):
    """float32 results of a bfloat16 layer: dz in as many terms as it takes. Slopes of silu and gelu are off by a few of
    2^-22 (approximate reciprocal and power of two, erf to 1.5e-7): 2^-21 by norm."""
    M, N, K = size
    d = on_gpu(M, N, K, "bf16", 21)
    saved = None if act == "none" else d["r"]
    _, gw, gb, _ = dcn.linear_backward(d["x"], d["w"], saved, d["gy"], act, need_input=False)
    torch.cuda.synchronize()
    dcn.check_status()
    dz = d["gy"].double() * (1 if act == "none" else ref.slope(saved.double(), act))
    tol = allowed(M) + (2.0 ** -21 if act in ("silu", "gelu") else 0)
    assert norm_off(gw, product64(dz.t(), d["x"].t())) <= tol
    assert norm_off(gb, dz.sum(0)) <= tol + 2.0 ** -23 * math.sqrt(M) / 8  # (chains of up to a sixteenth of the rows)


@pytest.mark.parametrize("size", [(4000, 1024, 12544), (700, 264, 25088), (9, 520, 12544), (300, 72, 65536), (1000, 96, 12545),
                                  (2000, 40, 6272)], ids=name)
def test_linear_bfloat16_long_reductions_round_once(size):
    """Positive products, whose sum cut off at each step drifts down. The accumulator is taken out every 256 steps at
    most: it loses 256 x 2^-24 / 2 of it (units of 2^-24 to 2^-23, half of one a step, running sums of half the size),
    7.6e-6, and a value flips to its neighbour where it is within that of the middle: 2^8 to 2^9 of 7.6e-6, 0.4 %, twice
    that allowed. (The whole of 12544 in the accumulator: 5.8e-5, over 1.5 %.)"""
    M, N, K = size
    d = on_gpu(M, N, K, "bf16", 25)
    x, w = d["x"].abs(), d["w"].abs()
    y, z = dcn.linear_forward(x, w, activation="silu", need_preact=True)
    torch.cuda.synchronize()
    dcn.check_status()
    want = product64(x, w)
    assert float((z != want.bfloat16()).double().mean()) <= 0.008
    r = torch.randn_like(z)  # with the rest of the epilogue
    y = dcn.linear_forward(x, w, d["b"], r, "relu")
    want = want + d["b"].double() + r.double()
    ref.check("y", y, want.clamp(min=0), 2.0 ** -16 * want.abs() + 2.0 ** -8 * want.abs() + 1e-30)
    # grad_x of as long a reduction
    gx = dcn.linear_backward(x[:, :N].contiguous(), torch.ones((K, N), dtype=x.dtype, device="cuda"), None, x, "none",
                             need_weight=False, need_bias=False)[0]
    want = x.double().sum(1, keepdim=True).expand(M, N)
    assert float((gx != want.bfloat16()).double().mean()) <= 0.02 and float(((gx.double() - want) / want).abs().max()) <= 1.02 * 2.0 ** -8
