"""Cases for the linear layer with a fused epilogue and for group normalisation.

The two operators stand next to the deformable convolution in the blocks that
use it: 1x1 convolutions (matrix products over the pixels of an NHWC map) before
and after it, group normalisation with the activation behind it, and the fully
connected layers behind deformable RoI pooling.

  linear      y = act(x W^T + bias + residual), x [M, K], W [N, K]
  group norm  y = act(gamma * (x - mean) * rstd + beta), x [B, H, W, C], statistics
              over each sample's groups of C / groups channels

Activations: none, relu, silu, gelu (with erf). float32 and bfloat16.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MOST_FLOPS = 1.0e11  # of a drawn linear case
MOST_ELEMENTS = 4.0e7  # of a drawn map, and of a linear layer's matrices
EPS = 1e-5


def _linear(name, op, dtype, M, N, K, act, bias=True, residual=False, preact=False):
    c = {"op": op, "dtype": dtype, "M": M, "N": N, "K": K, "act": act, "bias": bias, "residual": residual,
         "preact": preact}
    return dict(c, name=name) if name else c


def _norm(name, op, dtype, B, H, W, C, groups, act, affine=True):
    c = {"op": op, "dtype": dtype, "B": B, "H": H, "W": W, "C": C, "groups": groups, "act": act, "affine": affine}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the first fully connected layer behind 7x7 RoI pooling of 256 channels, for the few RoIs left in one image:
        # bound by the weight's bytes, latency counts
        _linear("linear_fwd_few_rois", "linear_fwd", "bf16", 5, 1024, 12544, "relu"),
        # the same layer for a training batch of RoIs: bound by the matrix product, few output tiles
        _linear("linear_fwd_many_rois", "linear_fwd", "bf16", 4000, 1024, 12544, "relu"),
        # the 1x1 convolution that ends a conv4 bottleneck block, with its shortcut: bound by bytes
        _linear("linear_fwd_expand", "linear_fwd", "bf16", 20000, 1024, 256, "relu", residual=True),
        # the first layer of an MLP over a conv5-sized map, its pre-activation kept for the backward pass
        _linear("linear_fwd_mlp", "linear_fwd", "bf16", 5000, 2048, 512, "gelu", preact=True),
        # a float32 layer of odd sizes
        _linear("linear_fwd_f32_odd", "linear_fwd", "f32", 1237, 331, 515, "silu"),
        # backward of the 1x1 convolution that opens a conv4 bottleneck block
        _linear("linear_bwd_reduce", "linear_bwd", "bf16", 20000, 256, 1024, "relu"),
        # backward of the MLP's first layer
        _linear("linear_bwd_mlp", "linear_bwd", "bf16", 5000, 2048, 512, "gelu"),
        # backward of a float32 1x1 convolution with a shortcut
        _linear("linear_bwd_f32", "linear_bwd", "f32", 4900, 512, 256, "relu", residual=True),
        # the smallest map of a feature pyramid: latency counts
        _norm("norm_fwd_small_map", "norm_fwd", "bf16", 1, 7, 10, 256, 32, "relu"),
        # behind the conv4 deformable layer
        _norm("norm_fwd_conv4", "norm_fwd", "bf16", 8, 50, 50, 256, 32, "relu"),
        # behind a 200x200 layer of a batch: bound by bytes, statistics over long rows
        _norm("norm_fwd_large", "norm_fwd", "bf16", 8, 200, 200, 128, 32, "silu"),
        # training step of a 100x100 map
        _norm("norm_bwd_large", "norm_bwd", "bf16", 8, 100, 100, 256, 32, "relu"),
    ]


def _size(rng, lo, hi, step=1):
    """Log-uniform in [lo, hi], a multiple of `step` most of the time."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if step > 1 and v >= step and rng.random() < 0.7:
        v = v // step * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("linear_fwd", "linear_bwd", "norm_fwd", "norm_bwd"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    act = rng.choice(ACTS)
    if op.startswith("linear"):
        M, N, K = _size(rng, 1, 80000), _size(rng, 8, 4096, 8), _size(rng, 8, 12544, 8)
        most = MOST_FLOPS / (4 if op == "linear_bwd" else 2)
        M = max(1, min(M, int(most / (N * K)), int(MOST_ELEMENTS / max(N, K))))
        return _linear(None, op, dtype, M, N, K, act, bias=rng.random() < 0.8, residual=rng.random() < 0.4,
                       preact=op == "linear_fwd" and act in ("silu", "gelu") and rng.random() < 0.5)
    groups = rng.choice((1, 2, 3, 8, 16, 32, 32, 32, 64))
    C = groups * _size(rng, 1, max(1, 1024 // groups))
    B, H, W = rng.randint(1, 16), _size(rng, 1, 200), _size(rng, 1, 200)
    B = max(1, min(B, int(MOST_ELEMENTS / (H * W * C))))
    return _norm(None, op, dtype, B, H, W, C, groups, act, affine=rng.random() < 0.9)


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    """d act / dz; relu: 0 at 0."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def prepare(case, seed):
    """The layer's input and parameters; for a backward pass also what its forward pass left and grad_y."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(t)

    s = dict(case)
    if case["op"].startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = normal(M, K)
        s["w"] = normal(N, K, scale=math.sqrt(2.0 / K))
        s["b"] = normal(N, scale=0.5) if case["bias"] else None
        s["r"] = normal(M, N) if case["residual"] else None
        if case["op"] == "linear_bwd":
            z = _linear_z(s["x"], s["w"], s["b"], s["r"])
            # relu keeps its output, silu and gelu their pre-activation
            s["saved"] = None if case["act"] == "none" else _act(z, "relu").to(t) if case["act"] == "relu" else z.to(t)
            s["gy"] = normal(M, N)
        return s
    B, H, W, C = (case[k] for k in "BHWC")
    # channels of different level and spread, as a convolution leaves them
    level = torch.randn((C,), generator=g, device="cuda") * 0.5
    spread = torch.rand((C,), generator=g, device="cuda") + 0.5
    s["x"] = (torch.randn((B, H, W, C), generator=g, device="cuda") * spread + level).to(t)
    s["gamma"] = normal(C, scale=0.2, shift=1.0) if case["affine"] else None
    s["beta"] = normal(C, scale=0.2) if case["affine"] else None
    if case["op"] == "norm_bwd":
        s["stats"] = _moments(s["x"], case["groups"], torch.float64).float()
        s["gy"] = normal(B, H, W, C)
    return s


def _linear_z(x, w, b, r):
    z = x.float() @ w.float().t()
    if b is not None:
        z = z + b.float()
    if r is not None:
        z = z + r.float()
    return z


def _moments(x, groups, t):
    """[B, groups, 2]: mean and 1 / sqrt(variance + eps) of each sample's groups of channels."""
    B, H, W, C = x.shape
    v = x.to(t).view(B, H * W, groups, C // groups)
    mean = v.mean(dim=(1, 3))
    var = (v - mean[:, None, :, None]).square().mean(dim=(1, 3))
    return torch.stack((mean, 1 / torch.sqrt(var + EPS)), dim=-1)


def run(state):
    if own:
        return _call(state)
    return _plain(state)


def _call(s):
    import deformable_convolution_dcn_b200 as dcn

    if s["op"] == "linear_fwd":
        return dcn.linear_forward(s["x"], s["w"], s["b"], s["r"], s["act"], need_preact=s["preact"])
    if s["op"] == "linear_bwd":
        gx, gw, gb, gr = dcn.linear_backward(s["x"], s["w"], s["saved"], s["gy"], s["act"], need_bias=s["bias"],
                                             need_residual=s["residual"])
        return {k: v for k, v in (("grad_x", gx), ("grad_weight", gw), ("grad_bias", gb), ("grad_residual", gr))
                if v is not None}
    if s["op"] == "norm_fwd":
        return dcn.group_norm_forward(s["x"], s["gamma"], s["beta"], s["groups"], EPS, s["act"])
    gx, gg, gb = dcn.group_norm_backward(s["x"], s["gamma"], s["beta"], s["stats"], s["gy"], s["groups"], s["act"])
    return {k: v for k, v in (("grad_x", gx), ("grad_gamma", gg), ("grad_beta", gb)) if v is not None}


def _plain(s):
    t = s["x"].dtype
    if s["op"] == "linear_fwd":
        z = _linear_z(s["x"], s["w"], s["b"], s["r"])
        y = _act(z, s["act"]).to(t)
        return (y, z.to(t)) if s["preact"] else y
    if s["op"] == "linear_bwd":
        x, w, gy = s["x"].float(), s["w"].float(), s["gy"].float()
        dz = gy if s["act"] == "none" else gy * _act_slope(s["saved"].float(), s["act"])
        out = {"grad_x": (dz @ w).to(t), "grad_weight": dz.t() @ x}
        if s["bias"]:
            out["grad_bias"] = dz.sum(0)
        if s["residual"]:
            out["grad_residual"] = dz.to(t)
        return out
    B, H, W, C = s["x"].shape
    G = s["groups"]
    if s["op"] == "norm_fwd":
        stats = _moments(s["x"], G, torch.float32)
        z = _normed(s["x"].float(), stats, G)
        if s["affine"]:
            z = z * s["gamma"].float() + s["beta"].float()
        return _act(z, s["act"]).to(t), stats
    # z next to relu's border decides between grad_y and 0: in 64 bits
    wide = torch.float64 if s["act"] == "relu" else torch.float32
    hat = _normed(s["x"].to(wide), s["stats"].to(wide), G)
    z = hat * s["gamma"].to(wide) + s["beta"].to(wide) if s["affine"] else hat
    dz = s["gy"].float() * _act_slope(z, s["act"]).float()
    hat = hat.float()
    dh = dz * s["gamma"].float() if s["affine"] else dz
    by = lambda v: v.view(B, H * W, G, C // G)  # noqa: E731
    c1 = by(dh).mean(dim=(1, 3), keepdim=True)
    c2 = by(dh * hat).mean(dim=(1, 3), keepdim=True)
    rstd = s["stats"][:, None, :, 1, None]
    out = {"grad_x": (rstd * (by(dh) - c1 - by(hat) * c2)).view(B, H, W, C).to(t)}
    if s["affine"]:
        out["grad_gamma"] = (dz * hat).sum(dim=(0, 1, 2))
        out["grad_beta"] = dz.sum(dim=(0, 1, 2))
    return out


def _normed(x, stats, groups):
    B, H, W, C = x.shape
    v = x.view(B, H * W, groups, C // groups)
    return ((v - stats[:, None, :, 0, None]) * stats[:, None, :, 1, None]).view(B, H, W, C)


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        if case["op"] == "linear_fwd":
            extra = N * case["bias"] + M * N * (case["residual"] + case["preact"])
            return {"bytes": es * (M * K + N * K + M * N + extra), "flops": 2.0 * M * N * K}
        reads = es * (M * K + N * K + M * N * (1 + (case["act"] != "none")))
        writes = es * (M * K + M * N * case["residual"]) + 4 * (N * K + N * case["bias"])
        return {"bytes": reads + writes, "flops": 4.0 * M * N * K}
    n = case["B"] * case["H"] * case["W"] * case["C"]
    stats, c = 8 * case["B"] * case["groups"], 2 * case["C"] * case["affine"]
    if case["op"] == "norm_fwd":
        return {"bytes": es * (2 * n + c) + stats, "flops": 8.0 * n}
    return {"bytes": es * (3 * n + c) + stats + 4 * c, "flops": 16.0 * n}


def exact(case, seed):
    """What run() returns, from the definitions, in float64: gradients through autograd where there are any."""
    s = prepare(case, seed)
    d = lambda k: None if s.get(k) is None else s[k].double()  # noqa: E731

    def f(z):
        if case["act"] == "relu":
            return torch.where(z > 0, z, torch.zeros_like(z))
        if case["act"] == "silu":
            return z * torch.sigmoid(z)
        if case["act"] == "gelu":
            return z * torch.special.ndtr(z)
        return z

    if case["op"] == "linear_fwd":
        z = torch.einsum("mk,nk->mn", d("x"), d("w"))
        z = z if s["b"] is None else z + d("b")
        z = z if s["r"] is None else z + d("r")
        return (f(z), z) if case["preact"] else f(z)
    if case["op"] == "linear_bwd":
        dz = d("gy")
        if case["act"] != "none":  # relu's output has the slope of its pre-activation
            z = d("saved").requires_grad_()
            (dz,) = torch.autograd.grad(f(z), z, dz)
        out = {"grad_x": torch.einsum("mn,nk->mk", dz, d("w")), "grad_weight": torch.einsum("mn,mk->nk", dz, d("x"))}
        if case["bias"]:
            out["grad_bias"] = torch.einsum("mn->n", dz)
        if case["residual"]:
            out["grad_residual"] = dz
        return out
    B, H, W, C = (case[k] for k in "BHWC")
    G = case["groups"]
    x = d("x").reshape(B, H * W, G, C // G)
    ga, be = (d(k).reshape(G, C // G) if case["affine"] else None for k in ("gamma", "beta"))
    if case["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, dim=(1, 3), correction=0)
        stats = torch.stack((mean, (var + EPS).rsqrt()), dim=2)
        z = (x - mean.reshape(B, 1, G, 1)) * stats[..., 1].reshape(B, 1, G, 1)
        z = z * ga + be if case["affine"] else z
        return f(z).reshape(B, H, W, C), stats
    mean, rstd = (d("stats")[..., k].reshape(B, 1, G, 1) for k in (0, 1))
    hat = (x - mean) * rstd
    z = (hat * ga + be if case["affine"] else hat).requires_grad_()
    (dz,) = torch.autograd.grad(f(z), z, d("gy").reshape(x.shape))
    n = H * W * (C // G)
    dh = dz * ga if case["affine"] else dz
    gx = rstd * (dh - torch.einsum("bpgc->bg", dh).reshape(B, 1, G, 1) / n
                 - hat * torch.einsum("bpgc,bpgc->bg", dh, hat).reshape(B, 1, G, 1) / n)
    out = {"grad_x": gx.reshape(B, H, W, C)}
    if case["affine"]:
        out["grad_gamma"] = torch.einsum("bpgc,bpgc->gc", dz, hat).reshape(C)
        out["grad_beta"] = torch.einsum("bpgc->gc", dz).reshape(C)
    return out
