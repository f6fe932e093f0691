"""The linear layer on the GPU against float64, forward and backward, over sizes
from one value to long reductions, odd sizes, both types, every activation, with
and without bias and residual."""
import pytest
import torch

import deformable_convolution_dcn_b200 as dcn
import op_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "silu", "gelu")
# M, N, K: single values, odd sizes, one past a tile, few rows with a long reduction, long columns (grad_weight's
# reduction), several tiles in every direction, an output of one column
SIZES = [(1, 1, 1), (1, 8, 8), (3, 7, 5), (2, 1, 300), (17, 33, 65), (64, 64, 64), (128, 128, 64), (129, 136, 72),
         (200, 257, 130), (1000, 64, 24), (5, 1024, 520), (33, 24, 4104), (300, 72, 2056), (2500, 40, 48),
         (777, 520, 264), (4099, 16, 8), (260, 1032, 96),
         # a few rows: every count of them, weights of one row and of more than the GPU has blocks for
         (1, 1024, 2056), (2, 81, 1024), (3, 600, 64), (4, 1, 8), (6, 2001, 264), (7, 593, 4), (8, 331, 12544), (9, 331, 512)]


def make(M, N, K, dtype, bias=True, residual=True, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed * 7919 + M * 31 + N * 17 + K)
    t = TYPES[dtype]
    n = lambda *s: torch.randn(s, generator=g).to(t).to(device)  # noqa: E731
    return dict(x=n(M, K), w=(n(N, K) * K ** -0.5).to(t), b=n(N) if bias else None, r=n(M, N) if residual else None,
                gy=n(M, N))


def forward(d, act, **kw):
    y, z = dcn.linear_forward(d["x"], d["w"], d["b"], d["r"], act, need_preact=True, **kw)
    torch.cuda.synchronize()
    dcn.check_status()
    return y, z


def check_forward(d, act, **kw):
    y, z = forward(d, act, **kw)
    want = ref.linear_forward(d["x"], d["w"], d["b"], d["r"], act)
    ref.check("z", z, *want["z"])
    ref.check("y", y, *want["y"])
    only = dcn.linear_forward(d["x"], d["w"], d["b"], d["r"], act, **kw)
    assert torch.equal(only, y)


def check_backward(d, act, **kw):
    want_z = ref.linear_forward(d["x"], d["w"], d["b"], d["r"], act)
    saved = None if act == "none" else (want_z["y"][0] if act == "relu" else want_z["z"][0]).to(d["x"].dtype)
    got = dcn.linear_backward(d["x"], d["w"], saved, d["gy"], act, need_residual=True, **kw)
    torch.cuda.synchronize()
    dcn.check_status()
    want = ref.linear_backward(d["x"], d["w"], saved, d["gy"], act)
    for name, v in zip(("grad_x", "grad_weight", "grad_bias", "grad_residual"), got):
        ref.check(name, v, *want[name])
    # each alone gives the same bits
    for i, name in enumerate(("need_input", "need_weight", "need_bias", "need_residual")):
        flags = {k: k == name for k in ("need_input", "need_weight", "need_bias", "need_residual")}
        one = dcn.linear_backward(d["x"], d["w"], saved, d["gy"], act, **flags, **kw)
        assert [v is not None for v in one] == list(flags.values())
        assert torch.equal(one[i], got[i]), name
    return got


@pytest.mark.parametrize("generic", [True, False], ids=["generic", "default"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_linear_forward_matches(size, dtype, generic):
    i = SIZES.index(size)
    act = ACTS[(i + generic) % 4]
    check_forward(make(*size, dtype, bias=i % 3 != 1, residual=i % 2 == 0), act, generic=generic)


@pytest.mark.parametrize("generic", [True, False], ids=["generic", "default"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_linear_backward_matches(size, dtype, generic):
    check_backward(make(*size, dtype, seed=1), ACTS[(SIZES.index(size) + 2 * generic) % 4], generic=generic)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
def test_linear_every_activation(act, dtype):
    d = make(140, 72, 88, dtype, seed=2)
    check_forward(d, act)
    check_backward(d, act)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_linear_no_rows(dtype):
    t = TYPES[dtype]
    x, w = torch.empty((0, 12), dtype=t, device="cuda"), torch.randn((20, 12), device="cuda").to(t)
    assert dcn.linear_forward(x, w).shape == (0, 20)
    y, z = dcn.linear_forward(x.view(3, 0, 12), w, activation="gelu", need_preact=True)
    assert y.shape == z.shape == (3, 0, 20)
    gy = torch.empty((0, 20), dtype=t, device="cuda")
    gx, gw, gb, gr = dcn.linear_backward(x, w, gy, gy, "silu", need_residual=True)
    assert gx.shape == (0, 12) and gr.shape == (0, 20)
    assert torch.all(gw == 0) and torch.all(gb == 0)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_linear_unaligned_views(dtype):
    """Inputs and outputs that start on an element, not on 16 bytes."""
    d = make(70, 48, 40, dtype, seed=3)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    for name in ("x", "w", "b", "r", "gy"):
        e = dict(d)
        e[name] = shifted(d[name])
        check_forward(e, "silu")
        check_backward(e, "gelu")
    out = shifted(torch.zeros_like(d["r"]))
    got = dcn.linear_forward(d["x"], d["w"], d["b"], d["r"], "relu", out=out)
    assert got.data_ptr() == out.data_ptr()
    ref.check("y", got, *ref.linear_forward(d["x"], d["w"], d["b"], d["r"], "relu")["y"])


def test_linear_map_shapes_and_residual_in_place():
    """NHWC maps and a 1x1 convolution's weight; y over the residual; nothing past the rows is written."""
    d = make(2 * 9 * 11, 64, 32, "bf16", seed=4)
    want = ref.linear_forward(d["x"], d["w"], d["b"], d["r"], "relu")["y"]
    x, w, r = d["x"].view(2, 9, 11, 32), d["w"].view(64, 1, 1, 32), d["r"].view(2, 9, 11, 64)
    y = dcn.linear_forward(x, w, d["b"], r, "relu")
    assert y.shape == (2, 9, 11, 64)
    ref.check("y", y.view(-1, 64), *want)
    room = torch.full((2 * 9 * 11 + 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    room[:-3] = d["r"]
    out = room[:-3].view(2, 9, 11, 64)
    dcn.linear_forward(x, w, d["b"], out, "relu", out=out)
    assert torch.equal(out, y)
    assert torch.all(room[-3:] == 7)
    gx, gw, gb, _ = dcn.linear_backward(x, w, y, d["gy"].view(2, 9, 11, 64), "relu")
    assert gx.shape == x.shape and gw.shape == w.shape and gb.shape == (64,)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [(150, 72, 64), (6, 80, 640)], ids=["tiles", "few_rows"])
def test_linear_infinity_and_nan_stay_in_their_rows(size, dtype):
    M, N, K = size
    d = make(M, N, K, dtype, seed=5)
    clean = dcn.linear_forward(d["x"], d["w"], d["b"], d["r"], "relu")
    d["x"][1, 3] = float("inf")
    d["x"][3, 0] = float("nan")
    d["r"][4, 2] = float("-inf")
    y = dcn.linear_forward(d["x"], d["w"], d["b"], d["r"], "relu")
    torch.cuda.synchronize()
    assert not torch.isfinite(y[1]).all() and torch.isnan(y[3]).all()
    assert y[4, 2] == 0 and torch.equal(y[4, 3:], clean[4, 3:])
    rest = [i for i in range(M) if i not in (1, 3, 4)]
    assert torch.equal(y[rest], clean[rest])
    # relu's gradient keeps an infinite grad_y out of closed places
    gy = d["gy"].clone()
    gy[0] = torch.where(clean[0] > 0, gy[0], torch.full_like(gy[0], float("inf")))
    gx, gw, gb, gr = dcn.linear_backward(make(M, N, K, dtype, seed=5)["x"], d["w"], clean, gy, "relu",
                                         need_residual=True)
    for v in (gx, gw, gb, gr):
        assert torch.isfinite(v).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_linear_large_values_do_not_overflow_early(dtype):
    """Values next to the type's largest times small weights: the float32 sums stay finite."""
    t = TYPES[dtype]
    big = torch.finfo(t).max
    x = torch.full((130, 64), big, dtype=t, device="cuda")
    w = torch.full((40, 64), 2.0 ** -10, dtype=t, device="cuda")
    y = dcn.linear_forward(x, w)
    want = x.double() @ w.double().t()
    ref.check("y", y, want, (64 + 16) * ref.U * want + ref.half_step(t) * want * 1.01)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [(1000, 136, 72), (5, 1024, 520)], ids=["tiles", "few_rows"])
def test_linear_calls_are_independent(size, dtype):
    """Two calls on two streams at once, repeated, captured and replayed with new inputs: equal bits to a call alone."""
    a, b = make(*size, dtype, seed=6), make(*size, dtype, seed=7)
    run = lambda d: (dcn.linear_forward(d["x"], d["w"], d["b"], d["r"], "relu"),  # noqa: E731
                     *dcn.linear_backward(d["x"], d["w"], d["r"], d["gy"], "relu", need_residual=True))
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
    for _ in range(2):  # two graphs of the same inputs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(c)
        graphs.append((g, out))
    for d, want in ((a, wa), (b, wb)):
        for k in c:
            c[k].copy_(d[k])
        torch.cuda.synchronize()
        streams = (s1, s2)
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(u, v) for u, v in zip(out, want))
    dcn.check_status()


@pytest.mark.parametrize("act", ACTS)
def test_linear_gradients_against_differences(act):
    """Autograd's gradients along random directions against central differences of the float64 layer."""
    d = make(37, 24, 40, "f32", seed=8)
    leaves = {k: d[k].requires_grad_() for k in ("x", "w", "b", "r")}
    y = dcn.linear(leaves["x"], leaves["w"], leaves["b"], leaves["r"], act)
    y.backward(d["gy"])

    def loss(v):
        z = v["x"] @ v["w"].t() + v["b"] + v["r"]
        return float((ref.act(z, act) * d["gy"].double()).sum())

    g = torch.Generator(device="cuda").manual_seed(9)
    base = {k: v.detach().double() for k, v in leaves.items()}
    h = 1e-6
    for k in leaves:
        v = torch.randn(base[k].shape, generator=g, device="cuda", dtype=torch.float64)
        slope = (loss({**base, k: base[k] + h * v}) - loss({**base, k: base[k] - h * v})) / (2 * h)
        got = float((leaves[k].grad.double() * v).sum())
        size = float((leaves[k].grad.double() * v).abs().sum())
        # float32 gradients (2000 roundings of u at most) and, for relu, steps across its border
        assert abs(got - slope) <= 1e-4 * size + 1e-6, k


def test_linear_autograd_only_what_is_needed():
    d = make(40, 16, 24, "bf16", seed=10)
    w = d["w"].requires_grad_()
    y = dcn.linear(d["x"], w, d["b"], d["r"], "silu")
    y.backward(d["gy"])
    assert w.grad.dtype == torch.bfloat16 and d["x"].grad is None
    with torch.no_grad():
        assert not dcn.linear(d["x"], w, d["b"], d["r"], "silu").requires_grad
    r = d["r"].detach().requires_grad_()
    dcn.linear(d["x"], d["w"].detach(), None, r, "none").backward(d["gy"])
    assert torch.equal(r.grad, d["gy"])


def test_linear_refusals_on_the_device():
    d = make(6, 16, 24, "bf16")
    with pytest.raises(ValueError, match="contiguous"):
        dcn.linear_forward(d["x"].t().contiguous().t(), d["w"])
    with pytest.raises(TypeError, match="bfloat16"):
        dcn.linear_forward(d["x"], d["w"].float())
    with pytest.raises(ValueError, match="bias"):
        dcn.linear_forward(d["x"], d["w"], d["b"][:-1])
    with pytest.raises(ValueError, match="residual"):
        dcn.linear_forward(d["x"], d["w"], None, d["r"][:1])
    with pytest.raises(ValueError, match="grad_y"):
        dcn.linear_backward(d["x"], d["w"], None, d["x"], "none")
    with pytest.raises(ValueError, match="CUDA"):
        dcn.linear_forward(d["x"], d["w"], d["b"].cpu())


@pytest.mark.parametrize("M", [3, 64])
def test_linear_refuses_overlaps(M):
    x, w = torch.zeros(M, 64, device="cuda"), torch.zeros(64, 64, device="cuda")
    with pytest.raises(dcn.DcnError, match="overlaps"):
        dcn.linear_forward(x, w, out=x)
    if M == 64:
        with pytest.raises(dcn.DcnError, match="overlaps"):
            dcn.linear_forward(x, w, out=w)


# one output a row (a one-channel 1x1 convolution): bfloat16 rows on the tensor cores' columns (the first three), and not
@pytest.mark.parametrize("size", [(262144, 1, 512), (170519, 1, 1024), (19005, 1, 12544), (60000, 1, 2048), (4099, 1, 33)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
def test_linear_one_output(size, dtype, residual):
    """The bias is one value, whatever lies behind it."""
    M, N, K = size
    g = torch.Generator(device="cuda").manual_seed(12)
    n = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(TYPES[dtype])  # noqa: E731
    room = torch.full((M + 64,), float("nan"), dtype=TYPES[dtype], device="cuda")
    room[0] = 0.75
    x, w, r = n(M, K), n(1, K, k=K ** -0.5), n(M, 1) if residual else None
    y = dcn.linear_forward(x, w, room[:1], r, "relu")
    torch.cuda.synchronize()
    dcn.check_status()
    ref.check("y", y, *ref.linear_forward(x, w, room[:1], r, "relu")["y"])
    if residual:
        dcn.linear_forward(x, w, room[:1], r, "relu", out=r)
        assert torch.equal(r, y)


def spread_of(t):
    """0 where finite, 1 and -1 for the infinities, 2 for NaN."""
    return torch.where(torch.isnan(t), 2.0, torch.where(torch.isinf(t), torch.sign(t), 0.0)).cpu()


@pytest.mark.parametrize("size", [(8, 72, 64), (9, 72, 64), (150, 72, 64), (150, 72, 67), (2500, 8, 24), (33, 24, 4104),
                                  (40000, 64, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", list(TYPES))
def test_linear_infinities_spread_as_in_the_sums(size, dtype):
    """The same signs and NaN as the products' sums, whatever the number of rows."""
    M, N, K = size
    d = make(M, N, K, dtype, seed=15)
    inf = float("inf")
    d["x"][1, 3], d["x"][2, 0], d["x"][2, 1], d["x"][3, 0], d["x"][3, 2], d["x"][5, 4] = inf, inf, inf, inf, -inf, -inf
    d["w"][4, 3], d["w"][6, 5], d["gy"][7, 2], d["gy"][0, 4] = 0.0, -inf, inf, -inf  # (0 times infinity is NaN)
    d["w"][2, 6] = 1.0  # exact in one term
    y = dcn.linear_forward(d["x"], d["w"], d["b"], d["r"], "none")
    gx, gw, gb, gr = dcn.linear_backward(d["x"], d["w"], None, d["gy"], "none", need_residual=True)
    torch.cuda.synchronize()
    dcn.check_status()
    # the sums in float64 on the CPU (a product at a time: a library product need not keep the signs)
    x, w, gy = (d[k].double().cpu() for k in ("x", "w", "gy"))
    rows = slice(0, 12)
    want = (x[rows, None, :] * w).sum(-1) + (d["b"].double() + d["r"].double()[rows]).cpu()
    assert torch.equal(spread_of(y[rows]), spread_of(want).to(y.dtype))
    assert torch.isfinite(y[12:, :6]).all() and torch.isfinite(y[12:, 7:]).all()
    want = (gy[rows, :, None] * w).sum(1)
    assert torch.equal(spread_of(gx[rows]), spread_of(want).to(gx.dtype))
    want = torch.stack([(gy[:, n, None] * x).sum(0) for n in range(8)])
    assert torch.equal(spread_of(gw[:8]), spread_of(want).float())
    assert torch.equal(spread_of(gb), spread_of(gy.sum(0)).float()) and torch.equal(gr, d["gy"])
    # silu and gelu: grad_weight of a bfloat16 layer splits dz
    z = make(M, N, K, dtype, seed=16)["r"]
    gw = dcn.linear_backward(d["x"], d["w"], z, d["gy"], "gelu")[1]
    dz = gy * ref.slope(z.double().cpu(), "gelu")
    want = torch.stack([(dz[:, n, None] * x).sum(0) for n in range(8)])
    assert torch.equal(spread_of(gw[:8]), spread_of(want).float())


@pytest.mark.parametrize("size", [(300, 264, 72), (1000, 2056, 136), (9, 40, 24), (5000, 512, 256), (129, 65, 513),
                                  (20000, 264, 520), (5, 1024, 12544), (64, 512, 4096), (2, 300, 2056)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_linear_grad_x_of_bfloat16_does_not_round_dz(size, act):
    """grad_x = dz W is rounded once, at its end: two bfloat16 terms of dz leave out at most 2^-18 of it."""
    M, N, K = size
    d = make(M, N, K, "bf16", seed=17)
    saved = d["r"]
    gx = dcn.linear_backward(d["x"], d["w"], saved, d["gy"], act, need_weight=False, need_bias=False)[0]
    torch.cuda.synchronize()
    dcn.check_status()
    w, gy, z = d["w"].double(), d["gy"].double(), saved.double()
    dz = gy * ref.slope(z, act)
    want = dz @ w
    edz = 16 * ref.U * gy.abs() * (1 + z.abs()) + 2.0 ** -18 * dz.abs()
    err = (N + 16) * ref.U * (dz.abs() @ w.abs()) + edz @ w.abs()
    ref.check("grad_x", gx, want, err + ref.half_step(torch.bfloat16) * (want.abs() + err))
    # as far from the exact one as its rounding alone
    rounded = (want.bfloat16().double() - want).norm()
    assert float((gx.double() - want).norm()) <= 1.05 * float(rounded)
