"""Group normalisation on the GPU against float64, forward and backward."""
import pytest
import torch

import deformable_convolution_dcn_b200 as dcn
import op_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "silu", "gelu")
EPS = 1e-5
# B, H, W, C, groups: one value a group, one pixel, odd channels, groups that straddle a vector, one group, a group
# a channel, wide channels, groups wider than a block, long maps, many samples
SIZES = [(1, 1, 1, 1, 1), (2, 1, 1, 64, 8), (3, 5, 7, 30, 3), (1, 7, 10, 256, 32), (2, 9, 13, 66, 6), (2, 8, 8, 24, 2),
         (1, 6, 5, 40, 40), (2, 11, 3, 12, 1), (1, 50, 50, 256, 32), (2, 100, 90, 64, 16), (5, 4, 4, 2048, 32),
         (1, 3, 3, 4104, 2), (1, 2, 5, 2049, 1), (1, 130, 257, 8, 1), (70, 3, 2, 16, 4), (2, 33, 31, 96, 32),
         (1, 200, 210, 128, 32), (2, 40, 40, 520, 40), (1, 64, 64, 1088, 64),
         # long maps by the queue with a ring: many samples, uneven runs, a group a channel, one group, wide rows
         (3, 129, 131, 96, 32), (9, 90, 101, 64, 64), (2, 150, 140, 72, 1), (1, 257, 129, 1024, 32), (160, 33, 31, 64, 8),
         # the same without whole vectors, and blocks of groups wider than a unit
         (3, 129, 131, 33, 3), (2, 61, 67, 1536, 2), (1, 300, 301, 3, 1)]


def make(B, H, W, C, dtype, affine=True, level=0.7, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + B * 31 + H * 17 + W * 5 + C)
    t = TYPES[dtype]
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = n(B, H, W, C) * (torch.rand(C, generator=g) + 0.5) + level * n(C)
    d = dict(x=x.to(t).cuda(), gy=n(B, H, W, C).to(t).cuda(), ga=None, be=None)
    if affine:
        d.update(ga=(1 + 0.3 * n(C)).to(t).cuda(), be=(0.3 * n(C)).to(t).cuda())
    return d


def check_forward(d, groups, act, eps=EPS):
    y, stats = dcn.group_norm_forward(d["x"], d["ga"], d["be"], groups, eps, act)
    torch.cuda.synchronize()
    dcn.check_status()
    want = ref.norm_forward(d["x"], d["ga"], d["be"], groups, eps, act)
    ref.check("mean", stats[..., 0], *want["mean"])
    ref.check("rstd", stats[..., 1], *want["rstd"])
    ref.check("y", y, *want["y"])
    return y, stats


def given_stats(d, groups, eps=EPS):
    return torch.stack(ref.norm_stats(d["x"], groups, eps), dim=-1).float()


def check_backward(d, groups, act):
    stats = given_stats(d, groups)
    got = dcn.group_norm_backward(d["x"], d["ga"], d["be"], stats, d["gy"], groups, act)
    torch.cuda.synchronize()
    dcn.check_status()
    want = ref.norm_backward(d["x"], d["ga"], d["be"], stats, d["gy"], groups, act)
    for name, v in zip(("grad_x", "grad_gamma", "grad_beta"), got):
        if name == "grad_x" or d["ga"] is not None:
            ref.check(name, v, *want[name])
        else:
            assert v is None
    gx = dcn.group_norm_backward(d["x"], d["ga"], d["be"], stats, d["gy"], groups, act, need_params=False)
    assert gx[1] is None and gx[2] is None and torch.equal(gx[0], got[0])
    if d["ga"] is not None:
        gp = dcn.group_norm_backward(d["x"], d["ga"], d["be"], stats, d["gy"], groups, act, need_input=False)
        assert gp[0] is None and torch.equal(gp[1], got[1]) and torch.equal(gp[2], got[2])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_group_norm_forward_matches(size, dtype):
    i = SIZES.index(size)
    check_forward(make(*size[:4], dtype, affine=i % 4 != 2), size[4], ACTS[i % 4])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_group_norm_backward_matches(size, dtype):
    i = SIZES.index(size)
    check_backward(make(*size[:4], dtype, affine=i % 4 != 3, seed=1), size[4], ACTS[(i + 1) % 4])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
def test_group_norm_every_activation(act, dtype):
    d = make(2, 12, 11, 48, dtype, seed=2)
    check_forward(d, 6, act)
    check_backward(d, 6, act)


@pytest.mark.parametrize("size", [(2, 20, 20, 32), (1, 150, 140, 64)], ids=["small", "long"])
def test_group_norm_level_far_from_zero(size):
    """A level a thousand spreads from zero costs the digits that x itself has lost, no more."""
    d = make(*size, "f32", seed=3)
    d["x"] = d["x"] + 1000.0
    check_forward(d, 4, "silu")
    check_backward(d, 4, "none")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_group_norm_constant_groups(dtype):
    """No spread at all: y = act(beta), rstd = 1 / sqrt(eps)."""
    d = make(2, 6, 6, 32, dtype, seed=4)
    d["x"] = torch.full_like(d["x"], 3.25)
    y, stats = check_forward(d, 8, "none")
    assert torch.equal(y, d["be"].expand_as(y))
    assert torch.allclose(stats[..., 1], torch.full_like(stats[..., 1], EPS ** -0.5), rtol=1e-6)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [(2, 6, 7, 32), (2, 60, 70, 32)], ids=["small", "long"])
def test_group_norm_infinity_and_nan_stay_in_their_group(size, dtype):
    d = make(*size, dtype, seed=5)
    clean, _ = dcn.group_norm_forward(d["x"], d["ga"], d["be"], 4, EPS, "silu")
    d["x"][0, 2, 3, 9] = float("nan")
    d["x"][1, 5, 0, 31] = float("inf")
    d["x"][1, 0, 0, 0] = float("-inf")  # the first pixel, which sums are taken about
    y, stats = dcn.group_norm_forward(d["x"], d["ga"], d["be"], 4, EPS, "silu")
    torch.cuda.synchronize()
    for b, g in ((0, 1), (1, 3), (1, 0)):
        assert torch.isnan(y[b, ..., g * 8:g * 8 + 8]).all()
        y[b, ..., g * 8:g * 8 + 8] = clean[b, ..., g * 8:g * 8 + 8]
    assert torch.equal(y, clean)


def test_group_norm_in_place_and_unaligned():
    d = make(2, 9, 9, 48, "bf16", seed=6)
    y, stats = check_forward(d, 6, "relu")
    buf = d["x"].clone()
    z, stats2 = dcn.group_norm_forward(buf, d["ga"], d["be"], 6, EPS, "relu", out=buf)
    assert z.data_ptr() == buf.data_ptr() and torch.equal(z, y) and torch.equal(stats, stats2)
    flat = torch.empty(d["x"].numel() + 1, dtype=torch.bfloat16, device="cuda")
    for name in ("x", "gy"):
        e = dict(d)
        flat[1:] = d[name].flatten()
        e[name] = flat[1:].view(d["x"].shape)
        check_forward(e, 6, "silu")
        check_backward(e, 6, "relu")
    for dtype in TYPES:
        e = make(1, 8, 9, 33, dtype, seed=7)
        for k in ("ga", "be"):  # parameters that start on an element
            e[k] = torch.cat([e[k][:1], e[k]])[1:]
        check_forward(e, 11, "gelu")


@pytest.mark.parametrize("size", [(2, 50, 50, 64), (3, 128, 128, 96)], ids=["small", "long"])
def test_group_norm_calls_are_independent(size):
    a, b = make(*size, "bf16", seed=8), make(*size, "bf16", seed=9)
    run = lambda d: (*(f := dcn.group_norm_forward(d["x"], d["ga"], d["be"], 8, EPS, "silu")),  # noqa: E731
                     *dcn.group_norm_backward(d["x"], d["ga"], d["be"], f[1], d["gy"], 8, "silu"))
    wa, wb = run(a), run(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = run(a)
        with torch.cuda.stream(s2):
            gb = run(b)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(ga + gb, wa + wb))
    c = {k: v.clone() for k, v in a.items()}
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(c)
        graphs.append((g, out))
    for d, want in ((a, wa), (b, wb)):
        for k in c:
            c[k].copy_(d[k])
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(u, v) for u, v in zip(out, want))
    dcn.check_status()


@pytest.mark.parametrize("act", ACTS)
def test_group_norm_gradients_against_differences(act):
    d = make(2, 5, 6, 24, "f32", seed=10)
    leaves = {k: d[k].requires_grad_() for k in ("x", "ga", "be")}
    dcn.group_norm(leaves["x"], leaves["ga"], leaves["be"], 4, EPS, act).backward(d["gy"])

    def loss(v):
        mean, rstd = ref.norm_stats(v["x"], 4, EPS)
        z = (v["x"] - ref._spread(mean, 24)) * ref._spread(rstd, 24) * v["ga"] + v["be"]
        return float((ref.act(z, act) * d["gy"].double()).sum())

    g = torch.Generator(device="cuda").manual_seed(11)
    base = {k: v.detach().double() for k, v in leaves.items()}
    h = 1e-6
    for k in leaves:
        v = torch.randn(base[k].shape, generator=g, device="cuda", dtype=torch.float64)
        slope = (loss({**base, k: base[k] + h * v}) - loss({**base, k: base[k] - h * v})) / (2 * h)
        got = float((leaves[k].grad.double() * v).sum())
        size = float((leaves[k].grad.double() * v).abs().sum())
        assert abs(got - slope) <= 1e-4 * size + 1e-6, k


def test_group_norm_refusals_on_the_device():
    d = make(2, 4, 4, 16, "bf16")
    with pytest.raises(dcn.DcnError, match="multiple of groups"):
        dcn.group_norm_forward(d["x"], None, None, 3)
    with pytest.raises(dcn.DcnError, match="groups"):
        dcn.group_norm_forward(d["x"], None, None, 0)
    with pytest.raises(dcn.DcnError, match="eps"):
        dcn.group_norm_forward(d["x"], None, None, 4, eps=0.0)
    with pytest.raises(ValueError, match="gamma"):
        dcn.group_norm_forward(d["x"], d["ga"][:-1], None, 4)
    with pytest.raises(ValueError, match="contiguous"):
        dcn.group_norm_forward(d["x"].permute(0, 2, 1, 3), None, None, 4)
    with pytest.raises(ValueError, match="stats"):
        dcn.group_norm_backward(d["x"], None, None, torch.zeros(2, 3, 2, device="cuda"), d["gy"], 4)
    ws = torch.empty(8, dtype=torch.uint8, device="cuda")
    p = dcn.NormParams(2, 4, 4, 16, 4, EPS, 0, dcn.DCN_BF16, 0)
    assert dcn.group_norm_workspace_size(p, dcn.OP_BACKWARD | dcn.OP_ALIGNED) > 8
    with pytest.raises(dcn.DcnError, match="workspace"):
        dcn.group_norm_backward(d["x"], None, None, given_stats(d, 4), d["gy"], 4, workspace=ws)
    # a small aligned map takes none forward; the same map off its alignment does
    assert dcn.group_norm_workspace_size(p, dcn.OP_FORWARD | dcn.OP_ALIGNED) == 0
    dcn.group_norm_forward(d["x"], None, None, 4, workspace=ws)
    off = torch.cat([d["x"].flatten()[:1], d["x"].flatten()])[1:].view(d["x"].shape)
    with pytest.raises(dcn.DcnError, match="workspace"):
        dcn.group_norm_forward(off, None, None, 4, workspace=ws)


# a cluster's map, one of the ring, one of single values
@pytest.mark.parametrize("size", [(2, 20, 21, 64, 8), (3, 129, 131, 96, 32), (3, 129, 131, 33, 3)])
@pytest.mark.parametrize("dtype", TYPES)
def test_group_norm_in_place_on_every_path(size, dtype):
    import ctypes
    B, H, W, C, groups = size
    d = make(B, H, W, C, dtype, seed=11)
    y, stats = dcn.group_norm_forward(d["x"], d["ga"], d["be"], groups, EPS, "silu")
    gx, gg, gb = dcn.group_norm_backward(d["x"], d["ga"], d["be"], stats, d["gy"], groups, "silu")
    x = d["x"].clone()
    dcn.group_norm_forward(x, d["ga"], d["be"], groups, EPS, "silu", out=x)
    assert torch.equal(x, y)
    p = dcn.NormParams(B, H, W, C, groups, EPS, dcn.ACTIVATIONS["silu"], int(dtype == "bf16"), 0)
    ws = torch.empty(dcn.group_norm_workspace_size(p, dcn.OP_BACKWARD), dtype=torch.uint8, device="cuda")
    gy, gg2, gb2 = d["gy"].clone(), torch.empty_like(gg), torch.empty_like(gb)
    rc = dcn._load().dcn_group_norm_backward(
        ctypes.byref(p), d["x"].data_ptr(), d["ga"].data_ptr(), d["be"].data_ptr(), stats.data_ptr(), gy.data_ptr(),
        gy.data_ptr(), gg2.data_ptr(), gb2.data_ptr(), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    dcn.check_status()
    assert torch.equal(gy, gx) and torch.equal(gg2, gg) and torch.equal(gb2, gb)


def test_group_norm_refuses_overlaps():
    buf = torch.zeros(2 * 8 * 8 * 16 + 16, device="cuda")
    n = 2 * 8 * 8 * 16
    x, y = buf[:n].view(2, 8, 8, 16), buf[16:].view(2, 8, 8, 16)
    with pytest.raises(dcn.DcnError, match="overlaps"):
        dcn.group_norm_forward(x, None, None, 4, out=y)


# the ring (units of several runs; a unit a sample), the queue with vectors (over 1024 channels), with single values
@pytest.mark.parametrize("size", [(1, 300, 300, 32, 4), (160, 120, 120, 16, 2), (2, 90, 120, 1088, 64), (12, 300, 300, 3, 1),
                                  (2, 40, 41, 64, 8)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("zeros", [1, 3, 500], ids=lambda z: "first%d" % z)
def test_group_norm_level_behind_a_border(size, zeros):
    """First pixels that are nothing like the others (a border of zeros before a level of 1000): the sums are not taken
    about them for good. The mean is off by at most 64 u of the level; squares about a mean that is off by a few u of the
    level m are off by (4 u m)^2 a value, and their sum by 64 u, so rstd by half of both."""
    B, H, W, C, groups = size
    g = torch.Generator(device="cuda").manual_seed(13)
    x = 1000.0 + torch.randn((B, H * W, C), generator=g, device="cuda")
    x[:, :zeros] = 0
    x = x.view(B, H, W, C)
    y, stats = dcn.group_norm_forward(x, None, None, groups, EPS, "none")
    torch.cuda.synchronize()
    dcn.check_status()
    mean, rstd = ref.norm_stats(x, groups, EPS)
    ref.check("mean", stats[..., 0], mean, 64 * ref.U * mean.abs())
    ref.check("rstd", stats[..., 1], rstd, rstd * (64 * ref.U + (4 * ref.U * mean * rstd) ** 2))


# by clusters, by the ring, by the queue (channels that are not whole vectors), and a few samples of each
@pytest.mark.parametrize("size", [(20000, 2, 2, 64, 8), (4096, 7, 7, 72, 8), (70000, 1, 1, 40, 8), (300, 45, 45, 512, 32),
                                  (3000, 3, 3, 33, 3), (33, 2, 2, 40, 8), (65, 2, 2, 40, 8), (64, 3, 3, 33, 3),
                                  (40, 100, 100, 64, 8)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", list(TYPES))
def test_group_norm_parameters_of_many_samples(size, dtype):
    """Equal samples with a constant grad_y, whose sums round the same way each time: no chain grows with them."""
    B, H, W, C, groups = size
    d = make(1, H, W, C, dtype, seed=14)
    d["x"] = d["x"].expand(B, H, W, C).contiguous()
    d["gy"] = torch.full_like(d["x"], 1.013)
    check_backward(d, groups, "none")


# the ring, the queue with vectors and with single values: thousands of pixels a thread
@pytest.mark.parametrize("size", [(16, 200, 200, 512, 32), (150, 160, 160, 64, 8), (2, 500, 500, 1088, 64), (1, 700, 700, 1025, 1),
                                  (1, 1000, 1000, 512, 32)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("value", [1.013, 1.1])
def test_group_norm_constant_gradients_of_large_maps(size, value):
    """The mean's gradient, the same everywhere, rounds the same way at each step of a sum: no chain grows with the map.
    (Runs of 64, chains of up to 130 runs, at most 512 units: 64 u, as for any gradient.)"""
    B, H, W, C, groups = size
    x = torch.randn((B, H, W, C), generator=torch.Generator(device="cuda").manual_seed(24), device="cuda")
    gy = torch.full_like(x, value)
    ga, be = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    stats = torch.stack(ref.norm_stats(x, groups, EPS), dim=-1).float()
    gx, gg, gb = dcn.group_norm_backward(x, ga, be, stats, gy, groups)
    torch.cuda.synchronize()
    dcn.check_status()
    want = float(gy.flatten()[0]) * B * H * W
    ref.check("grad_beta", gb, torch.full_like(gb, want, dtype=torch.float64), torch.full_like(gb, 64 * ref.U * want))
