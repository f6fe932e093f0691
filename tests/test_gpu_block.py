"""The operators together, as a bottleneck block runs them: 1x1 convolution with
relu, offset/mask predictor, deformable convolution, group normalisation with
relu, 1x1 convolution with shortcut and relu; forward and backward against the
same chain in float64 (the deformable layer by the oracle)."""
import numpy as np
import pytest
import torch

import deformable_convolution_dcn_b200 as dcn
import op_reference as ref
import oracle
from parity import assert_close

pytestmark = pytest.mark.gpu


def block(x, p, offset, mask, groups):
    h = dcn.linear(x, p["w1"], p["b1"], None, "relu")
    d = dcn.deform_conv2d(h, offset, p["wd"], None, 1, 1, 1, mask)
    n = dcn.group_norm(d, p["ga"], p["be"], groups, 1e-5, "relu")
    return dcn.linear(n, p["w3"], p["b3"], x, "relu")


def block64(x, p, offset, mask, groups, gy):
    """The chain in float64 on the CPU: y and the gradients of x and the parameters."""
    B, H, W, C = x.shape
    f = {k: v.detach().double().cpu().requires_grad_() for k, v in p.items()}
    x = x.detach().double().cpu().requires_grad_()
    off, m = offset.double().cpu().numpy(), mask.double().cpu().numpy()

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, w):
            ctx.save_for_backward(h, w)
            return torch.from_numpy(oracle.forward(h.detach().numpy(), off, m, w.detach().numpy(), None, 1, 1, 1, 1))

        @staticmethod
        def backward(ctx, g):
            h, w = ctx.saved_tensors
            r = oracle.backward(h.detach().numpy(), off, m, w.detach().numpy(), np.ascontiguousarray(g.numpy()), 1, 1, 1,
                                1)
            return torch.from_numpy(r["grad_x"]), torch.from_numpy(r["grad_weight"])

    h = ref.act(x.reshape(-1, C) @ f["w1"].t() + f["b1"], "relu").reshape(B, H, W, -1)
    d = Layer.apply(h, f["wd"])
    mean, rstd = ref.norm_stats(d, groups, 1e-5)
    n = (d - ref._spread(mean, d.shape[-1])) * ref._spread(rstd, d.shape[-1]) * f["ga"] + f["be"]
    n = ref.act(n, "relu")
    y = ref.act(n.reshape(-1, n.shape[-1]) @ f["w3"].t() + f["b3"] + x.reshape(-1, C), "relu").reshape(B, H, W, C)
    y.backward(gy.double().cpu())
    return y.detach().numpy(), x.grad.numpy(), {k: v.grad.numpy() for k, v in f.items()}


@pytest.mark.parametrize("shape", [(2, 9, 8, 24, 16, 4), (1, 13, 14, 64, 32, 8)], ids=["odd", "aligned"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bottleneck_block(shape, dtype):
    B, H, W, C, mid, groups = shape
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(17)
    n = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).to(t).cuda()  # noqa: E731
    x, gy = n(B, H, W, C), n(B, H, W, C)
    p = dict(w1=n(mid, C, k=C ** -0.5), b1=n(mid, k=0.3), wd=n(mid, 3, 3, mid, k=(9 * mid) ** -0.5),
             ga=1 + n(mid, k=0.2), be=n(mid, k=0.3), w3=n(C, mid, k=mid ** -0.5), b3=n(C, k=0.3))
    p = {k: v.to(t) for k, v in p.items()}
    wp, bp = n(27, 3, 3, mid, k=0.3 * (9 * mid) ** -0.5), n(27, k=0.2)
    with torch.no_grad():
        offset, mask = dcn.predict_offset_mask(dcn.linear(x, p["w1"], p["b1"], None, "relu"), wp, bp, 3, 1, 1)
    leaves = {k: v.requires_grad_() for k, v in p.items()}
    xl = x.clone().requires_grad_()
    y = block(xl, leaves, offset, mask, groups)
    y.backward(gy)
    torch.cuda.synchronize()
    dcn.check_status()
    ry, rgx, rg = block64(x, p, offset, mask, groups, gy)
    if dtype == "f32":
        assert_close(y.detach().cpu().numpy(), ry, "f32", "y")
        # a value within float32's rounding of relu's border may take the other side; none does at these seeds
        assert_close(xl.grad.cpu().numpy(), rgx, "f32", "grad_x")
        for k, v in rg.items():
            # sums over B H W pixels: their size, not one
            scale = max(1.0, float(np.abs(v).max()))
            assert_close(leaves[k].grad.cpu().numpy() / scale, v / scale, "f32", k)
    else:
        # five roundings to bfloat16 (2^-8 of a value each, 2^-9.2 in the mean square) on the way, and relu's border
        # crossed by values that were rounded: normwise 4e-2 forward, 1e-1 for gradients through three relus
        for name, got, want, tol in [("y", y, ry, 4e-2), ("grad_x", xl.grad, rgx, 1e-1)] + [
                (k, leaves[k].grad, rg[k], 1e-1) for k in rg]:
            off = np.linalg.norm(got.detach().double().cpu().numpy() - want) / np.linalg.norm(want)
            assert off <= tol, (name, off)


def test_block_captured_and_replayed():
    """The block's forward and backward in one CUDA graph, replayed on new inputs, give an eager step's bits."""
    torch.manual_seed(3)
    C, mid, groups = 64, 32, 8
    n = lambda *s, k=1.0: (torch.randn(s, device="cuda") * k).bfloat16()  # noqa: E731
    p = dict(w1=n(mid, C, k=0.1), b1=n(mid), wd=n(mid, 3, 3, mid, k=0.05), ga=n(mid), be=n(mid), w3=n(C, mid, k=0.2),
             b3=n(C))
    offset, mask = n(2, 18, 10, 11), torch.sigmoid(n(2, 9, 10, 11))
    inputs = [(n(2, 10, 11, C), n(2, 10, 11, C)) for _ in range(2)]

    def step(x, gy):
        h = dcn.linear_forward(x, p["w1"], p["b1"], None, "relu")
        d = dcn.forward(h, offset, mask, p["wd"], None, 1, 1, 1)
        m, st = dcn.group_norm_forward(d, p["ga"], p["be"], groups, 1e-5, "relu")
        y = dcn.linear_forward(m, p["w3"], p["b3"], x, "relu")
        gm, gw3, gb3, gr = dcn.linear_backward(m, p["w3"], y, gy, "relu", need_residual=True)
        gd, gg, gb = dcn.group_norm_backward(d, p["ga"], p["be"], st, gm, groups, "relu")
        return y, gw3, gb3, gr, gd, gg, gb

    want = [step(*i) for i in inputs]
    x, gy = (t.clone() for t in inputs[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(x, gy)
    for (a, b), w in zip(inputs, want):
        x.copy_(a)
        gy.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, w))
    dcn.check_status()
