"""Host-side checks of the linear layer and the group normalisation (no GPU
needed): bad arguments are rejected with the documented codes before anything
reaches the device. No call here passes valid device pointers."""
import ctypes

import pytest
import torch

import deformable_convolution_dcn_b200 as dcn

OK, EINVAL, EUNSUP, EWS = 0, -1, -2, -5
F = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from deformable_convolution_dcn_b200 import build
    build.build()
    return dcn._load()


def LP(**kw):
    d = dict(M=5, N=6, K=7, act=1, dtype=1, flags=0)
    d.update(kw)
    return dcn.LinearParams(*(d[k] for k in ("M", "N", "K", "act", "dtype", "flags")))


def NP(**kw):
    d = dict(B=2, H=3, W=4, C=12, groups=3, eps=1e-5, act=1, dtype=1, flags=0)
    d.update(kw)
    return dcn.NormParams(*(d[k] for k in ("B", "H", "W", "C", "groups", "eps", "act", "dtype", "flags")))


def lin_fwd(lib, p, x=F, w=F, b=None, r=None, y=F, z=None, ws=F, n=BIG):
    return lib.dcn_linear_forward(ctypes.byref(p), x, w, b, r, y, z, ws, n, None)


def lin_bwd(lib, p, x=F, w=F, s=F, gy=F, gx=F, gw=F, gb=F, gr=F, ws=F, n=BIG):
    return lib.dcn_linear_backward(ctypes.byref(p), x, w, s, gy, gx, gw, gb, gr, ws, n, None)


def gn_fwd(lib, p, x=F, ga=None, be=None, y=F, st=F, ws=F, n=BIG):
    return lib.dcn_group_norm_forward(ctypes.byref(p), x, ga, be, y, st, ws, n, None)


def gn_bwd(lib, p, x=F, ga=None, be=None, st=F, gy=F, gx=F, gg=F, gb=F, ws=F, n=BIG):
    return lib.dcn_group_norm_backward(ctypes.byref(p), x, ga, be, st, gy, gx, gg, gb, ws, n, None)


@pytest.mark.parametrize("bad,code", [
    (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(act=4), EINVAL), (dict(act=-1), EINVAL),
    (dict(dtype=2), EUNSUP), (dict(M=1 << 20, N=1 << 12), EUNSUP), (dict(M=1 << 20, K=1 << 12), EUNSUP),
    (dict(N=1 << 20, K=1 << 12), EUNSUP), (dict(M=(1 << 30) + 1, N=1, K=1), EUNSUP),
    (dict(M=1, N=1, K=(1 << 30) + 1), EUNSUP),
])
def test_linear_params_rejected(lib, bad, code):
    p = LP(**bad)
    assert lin_fwd(lib, p) == code
    assert lib.dcn_last_error_string().decode() != ""
    assert lin_bwd(lib, p) == code
    assert dcn.linear_workspace_size(p, dcn.OP_FORWARD) == 0
    assert dcn.linear_workspace_size(p, dcn.OP_BACKWARD) == 0


def test_linear_pointers(lib):
    p = LP()
    for kw in (dict(x=None), dict(w=None), dict(y=None)):
        assert lin_fwd(lib, p, **kw) == EINVAL
    for kw in (dict(x=ODD), dict(w=ODD), dict(b=ODD), dict(r=ODD), dict(y=ODD), dict(z=ODD)):
        assert lin_fwd(lib, p, **kw) == EUNSUP
    for kw in (dict(x=None), dict(w=None), dict(s=None), dict(gy=None)):
        assert lin_bwd(lib, p, **kw) == EINVAL
    for kw in (dict(s=ODD), dict(gy=ODD), dict(gx=ODD), dict(gw=ctypes.c_void_p((1 << 20) + 2)), dict(gr=ODD)):
        assert lin_bwd(lib, p, **kw) == EUNSUP
    assert lib.dcn_linear_forward(None, F, F, None, None, F, None, None, 0, None) == EINVAL


def test_linear_without_rows_or_outputs_enqueues_nothing(lib):
    n = dcn.launch_count()
    assert lin_fwd(lib, LP(M=0), x=None, y=None) == OK
    assert lin_bwd(lib, LP(), gx=None, gw=None, gb=None, gr=None) == OK
    assert lin_bwd(lib, LP(M=0), x=None, s=None, gy=None, gw=None, gb=None) == OK
    assert dcn.launch_count() == n


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), EINVAL), (dict(H=0), EINVAL), (dict(W=-2), EINVAL), (dict(C=0), EINVAL), (dict(groups=0), EINVAL),
    (dict(groups=5), EINVAL), (dict(eps=0.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(act=9), EINVAL), (dict(dtype=3), EUNSUP),
    (dict(B=1 << 10, H=1 << 10, W=1 << 10), EUNSUP), (dict(B=1, H=1 << 16, W=(1 << 14) + 1, C=1, groups=1), EUNSUP),
    (dict(B=(1 << 28) + 1, H=1, W=1, C=1, groups=1), EUNSUP),
])
def test_group_norm_params_rejected(lib, bad, code):
    p = NP(**bad)
    assert gn_fwd(lib, p) == code
    assert lib.dcn_last_error_string().decode() != ""
    assert gn_bwd(lib, p) == code
    assert dcn.group_norm_workspace_size(p, dcn.OP_FORWARD) == 0
    assert dcn.group_norm_workspace_size(p, dcn.OP_BACKWARD) == 0


def test_group_norm_pointers_and_workspace(lib):
    p = NP()
    for kw in (dict(x=None), dict(y=None)):
        assert gn_fwd(lib, p, **kw) == EINVAL
    for kw in (dict(x=ODD), dict(ga=ODD), dict(be=ODD), dict(y=ODD), dict(st=ctypes.c_void_p((1 << 20) + 2))):
        assert gn_fwd(lib, p, **kw) == EUNSUP
    for kw in (dict(x=None), dict(st=None), dict(gy=None)):
        assert gn_bwd(lib, p, **kw) == EINVAL
    assert gn_bwd(lib, p, gx=None, gg=None, gb=None) == OK
    off = ctypes.c_void_p((1 << 20) + 2)
    for op, call in ((dcn.OP_FORWARD, lambda *a, **k: gn_fwd(*a, x=off, **k)),
                     (dcn.OP_BACKWARD, lambda *a, **k: gn_bwd(*a, x=off, **k))):
        n = dcn.group_norm_workspace_size(p, op)
        assert n >= dcn.group_norm_workspace_size(p, op | dcn.OP_ALIGNED)
        if n:
            assert call(lib, p, ws=None) == EWS
            assert call(lib, p, n=n - 1) == EWS
            assert str(n) in lib.dcn_last_error_string().decode()
            assert call(lib, p, ws=ctypes.c_void_p((1 << 20) + 8)) == EUNSUP


def test_binding_rejects_shapes():
    x, w = torch.zeros(2, 3, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dcn.linear_forward(x, w)
    with pytest.raises(ValueError, match="weight"):
        dcn.linear_forward(x, torch.zeros(4, 9))
    with pytest.raises(ValueError, match="1, 1"):
        dcn.linear_forward(x, torch.zeros(4, 3, 3, 8))
    with pytest.raises(ValueError, match="empty"):
        dcn.linear_forward(torch.zeros(2, 0), torch.zeros(4, 0))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        dcn.linear_forward(x.half(), w.half())
    with pytest.raises(ValueError, match="activation"):
        dcn.linear_forward(x, w, activation="tanh")
    with pytest.raises(ValueError, match="saved must be None"):
        dcn.linear_backward(x, w, x, x, "none")
    with pytest.raises(ValueError, match="saved must be the output"):
        dcn.linear_backward(x, w, None, x, "relu")
    m = torch.zeros(1, 2, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dcn.group_norm_forward(m, None, None, 2)
    with pytest.raises(ValueError, match="B, H, W, C"):
        dcn.group_norm_forward(x, None, None, 2)
    with pytest.raises(ValueError, match="activation"):
        dcn.group_norm_forward(m, None, None, 2, activation="elu")


def test_workspace_sizes(lib):
    # the tensor-core kernels of a layer without rows or kept off them need none
    assert dcn.linear_workspace_size(LP(M=0), dcn.OP_FORWARD) == 0
    assert dcn.linear_workspace_size(LP(flags=dcn.DCN_FLAG_GENERIC), dcn.OP_BACKWARD) == 0
    # bfloat16 rows of whole vectors are read in place; others are copied, float32 in three terms
    assert dcn.linear_workspace_size(LP(M=4096, N=256, K=64), dcn.OP_FORWARD) == 0
    assert dcn.linear_workspace_size(LP(M=4096, N=256, K=65), dcn.OP_FORWARD) >= 2 * (4096 + 256) * 72
    assert dcn.linear_workspace_size(LP(M=4096, N=256, K=64, dtype=0), dcn.OP_FORWARD) >= 6 * (4096 + 256) * 64
    n = dcn.linear_workspace_size(LP(M=4096, N=256, K=65), dcn.OP_FORWARD)
    p = LP(M=4096, N=256, K=65)
    assert lin_fwd(lib, p, ws=None) == EWS
    assert lin_fwd(lib, p, n=n - 1) == EWS
    assert str(n) in lib.dcn_last_error_string().decode()
    assert lin_fwd(lib, p, ws=ctypes.c_void_p((1 << 20) + 128)) == EUNSUP
    n = dcn.linear_workspace_size(p, dcn.OP_BACKWARD)
    assert n > 0 and lin_bwd(lib, p, n=n - 1) == EWS
    # sizes do not depend on where they are asked for, nor grow past what the tensors justify
    assert dcn.linear_workspace_size(LP(M=8, N=1024, K=12544), dcn.OP_FORWARD) == 0
    assert dcn.linear_workspace_size(LP(M=9, N=1024, K=12544), dcn.OP_FORWARD) <= 64 * 9 * 1024 * 4
    assert dcn.group_norm_workspace_size(NP(B=8, H=200, W=200, C=128, groups=32), dcn.OP_FORWARD) < 1 << 22


def at(k, size=0):
    """An address in a place of its own, far from the other places."""
    return ctypes.c_void_p((k << 30) + size)


@pytest.mark.parametrize("M", [5, 200])  # the few rows' kernel, tensor cores
@pytest.mark.parametrize("out,of", [("y", "x"), ("y", "w"), ("y", "b"), ("z", "x"), ("z", "r"), ("z", "y"), ("ws", "x")])
def test_linear_forward_refuses_overlaps(lib, M, out, of):
    p = LP(M=M, N=64, K=64 if M == 5 or out != "ws" else 65)
    if out == "ws" and lib.dcn_linear_workspace_size(ctypes.byref(p), 0) == 0:
        pytest.skip("no workspace")
    place = {k: at(i + 1) for i, k in enumerate(("x", "w", "b", "r", "y", "z", "ws"))}
    assert M == 5 or lib.dcn_linear_workspace_size(ctypes.byref(p), 0) <= 1 << 30
    place[out] = ctypes.c_void_p(place[of].value)
    assert lin_fwd(lib, p, **place) == EINVAL
    assert "overlaps" in lib.dcn_last_error_string().decode()


def test_linear_forward_refuses_a_shifted_residual(lib):
    p = LP(M=200, N=64, K=64)
    assert lin_fwd(lib, p, at(1), at(2), at(3), at(4), at(4, 16), None) == EINVAL
    assert lin_fwd(lib, p, at(1), at(2), at(3), at(4, 16), at(4), None) == EINVAL


@pytest.mark.parametrize("out", ["gx", "gw", "gb", "gr", "ws"])
@pytest.mark.parametrize("of", ["x", "w", "s", "gy"])
def test_linear_backward_refuses_overlaps(lib, out, of):
    p = LP(M=200, N=64, K=64)
    place = {k: at(i + 1) for i, k in enumerate(("x", "w", "s", "gy", "gx", "gw", "gb", "gr", "ws"))}
    place[out] = place[of]
    assert lin_bwd(lib, p, **place) == EINVAL
    place = {k: at(i + 1) for i, k in enumerate(("x", "w", "s", "gy", "gx", "gw", "gb", "gr", "ws"))}
    place["gr"] = place["gx"]
    assert lin_bwd(lib, p, **place) == EINVAL


@pytest.mark.parametrize("side", [7, 333])
def test_group_norm_refuses_overlaps(lib, side):
    p = NP(B=2, H=side, W=side, C=64, groups=8)
    fwd, bwd = lib.dcn_group_norm_forward, lib.dcn_group_norm_backward
    q = ctypes.byref(p)
    assert fwd(q, at(1), at(2), at(3), at(1, 16), at(5), at(6), BIG, None) == EINVAL
    assert fwd(q, at(1), at(2), at(3), at(2), at(5), at(6), BIG, None) == EINVAL
    assert fwd(q, at(1), at(2), at(3), at(4), at(1), at(6), BIG, None) == EINVAL
    assert bwd(q, at(1), at(2), at(3), at(4), at(5), at(1), at(7), at(8), at(9), BIG, None) == EINVAL
    assert bwd(q, at(1), at(2), at(3), at(4), at(5), at(5, 16), at(7), at(8), at(9), BIG, None) == EINVAL
    assert bwd(q, at(1), at(2), at(3), at(4), at(5), at(6), at(2), at(8), at(9), BIG, None) == EINVAL
    assert bwd(q, at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(7), at(9), BIG, None) == EINVAL


def test_norm_warps_leave_together():
    """In the kernel whose warps wait by themselves, a failed wait leads out through a barrier that all of them meet at,
    and no bounded wait but the last (of the copies in flight) goes without the block's flag."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(dcn.__file__), "csrc", "group_norm_stream.cu")).read()
    src = re.sub(r"//[^\n]*", "", src)
    waits = re.findall(r"mbar_wait\([^;]*;", src)
    assert len(waits) == 7 and sum("aborted" in w for w in waits) == 6
    # computing warps of both kernels, joining warps: decided by all, at the loop's end and at a unit's
    assert len(re.findall(r"if \(!there \|\| headers\[stage\]\.pass < 0\) \{\s+if \(agree_to_leave<COMPUTING, NC>\(!there\)\) "
                          r"return;\s+break;", src)) == 2
    assert src.count("if (agree_to_leave<COMPUTING, NC>(false)) return;") == 3
    assert src.count("if (agree_to_leave<JOINING, JOINERS>(!ok || set < 0)) return;") == 1
    body = src[src.index("void join_sets"):src.index("template <typename F, typename... Q>")]
    ways_out = len(re.findall(r"\breturn;", body))
    assert ways_out == 2 + 3 + 1 + 4, ways_out  # (the kernels' dispatch of the joining and the producer warps)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode, torch.enable_grad])
@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_linear_keeps_the_preactivation_only_for_a_backward_pass(monkeypatch, mode, activation):
    asked = []

    def forward(x, weight, bias=None, residual=None, activation="none", *, need_preact=False, **kw):
        asked.append(need_preact)
        y = x @ weight.t()
        return (y, y.clone()) if need_preact else y

    monkeypatch.setattr(dcn, "linear_forward", forward)
    x, w = torch.ones(3, 4), torch.ones(5, 4, requires_grad=True)
    with mode():
        y = dcn.linear(x, w, None, None, activation)
    assert asked == [mode is torch.enable_grad] and y.requires_grad == (mode is torch.enable_grad)
    dcn.linear(x, w.detach(), None, None, activation)  # gradients recorded, none required
    assert asked[-1] is False
