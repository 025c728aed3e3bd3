"""Refusals of the expert block's entry points (host validation, no GPU) and the registers of
its kernels."""
import ctypes

import pytest

import weight_only_int4_group_amd as w4
from tests.test_kernel_sources import _device_asm, _kernel_metadata
from weight_only_int4_group_amd import experts as ex

ODD = (1 << 20) + 2


def at(i):
    """Aligned stand-in addresses, 64 MB apart (never dereferenced)."""
    return (1 + i) << 26


def norm(kind=1, weight=None, bias=None, eps=1e-6):
    return ex.NormStruct(weight, bias, eps, kind)


NONE = (0, None, None, 0.0)


def norm_call(**kw):
    f = dict(x=at(0), y=at(1), gate=at(2), post=norm(), pre=norm(2, at(3), at(4)), r=at(5), h=at(6), T=4, D=64,
             gate_rows=2, alpha=1.0, dtype=0)
    f.update(kw)
    return ex.NormCallStruct(*f.values())


def norm_rc(**kw):
    return w4.lib().w4a16_norm_block(ctypes.byref(norm_call(**kw)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(T=1 << 22), -1), (dict(D=0), -1), (dict(D=16385), -1), (dict(dtype=2), -3),
    (dict(x=None), -1), (dict(r=None, h=None), -1), (dict(h=None), -1), (dict(pre=norm(*NONE)), -1),
    (dict(post=norm(3)), -3), (dict(pre=norm(-1)), -3), (dict(post=norm(0, at(3))), -1),
    (dict(post=norm(0, None, at(3))), -1), (dict(pre=norm(1, eps=-1.0)), -1),
    (dict(pre=norm(1, eps=float("nan"))), -1), (dict(pre=norm(1, eps=float("inf"))), -1),
    (dict(gate_rows=0), -1), (dict(y=None), -1), (dict(y=None, gate=None), -1),
    (dict(y=None, post=norm(*NONE)), -1), (dict(x=ODD), -2), (dict(y=ODD), -2), (dict(gate=ODD), -2),
    (dict(r=ODD), -2), (dict(h=ODD), -2), (dict(post=norm(1, ODD)), -2), (dict(pre=norm(1, None, ODD)), -2),
    (dict(r=at(0) + 496), -1), (dict(h=at(1) + 16), -1), (dict(r=at(6)), -1), (dict(h=at(2)), -1),
    (dict(r=at(3)), -1), (dict(T=0, x=None), 0),
])
def test_norm_refusals(kw, code):
    assert norm_rc(**kw) == code


def norm_backward(**kw):
    f = dict(dr=at(0), dh=at(1), y=at(2), r=at(3), gate=at(4), post=norm(1, at(5)), pre=norm(2, at(6), at(7)),
             dx=at(8), dy=at(9), dgate=at(10), dpost_weight=at(11), dpost_bias=at(12), dpre_weight=at(13),
             dpre_bias=at(14), T=4, D=64, gate_rows=2, alpha=1.0, dtype=0)
    f.update(kw)
    return ex.NormBackwardStruct(*f.values())


def norm_backward_rc(ws=at(20), nbytes=1 << 20, **kw):
    return w4.lib().w4a16_norm_block_backward(ctypes.byref(norm_backward(**kw)), ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(D=0), -1), (dict(D=20000), -1), (dict(dtype=7), -3), (dict(post=norm(5)), -3),
    (dict(dh=None), -1), (dict(r=None), -1), (dict(y=None), -1), (dict(gate=None), -1), (dict(gate_rows=-2), -1),
    (dict(pre=norm(*NONE)), -1), (dict(post=norm(*NONE)), -1),
    (dict(pre=norm(*NONE), dpre_weight=None, dpre_bias=None), -1),
    (dict(pre=norm(*NONE), dpre_weight=None, dpre_bias=None, dh=None, dr=None), -1),
    (dict(ws=None), -1), (dict(nbytes=16), -1), (dict(ws=at(20) + 16), -2), (dict(dx=ODD), -2), (dict(dgate=ODD), -2),
    (dict(dpre_bias=ODD), -2), (dict(dx=at(0)), -1), (dict(dy=at(2)), -1), (dict(dx=at(9) + 128), -1),
    (dict(dgate=at(4)), -1), (dict(dpost_weight=at(11), dpost_bias=at(11) + 128), -1), (dict(dx=at(20)), -1),
    (dict(dpre_weight=at(6)), -1),
])
def test_norm_backward_refusals(kw, code):
    assert norm_backward_rc(**kw) == code


def test_norm_backward_sizes():
    n = ctypes.c_size_t()
    size = w4.lib().w4a16_norm_block_backward_workspace_size
    none = dict.fromkeys(("dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"))
    assert size(ctypes.byref(norm_backward(T=4096, D=4096, **none)), ctypes.byref(n)) == 0 and n.value == 0
    assert size(ctypes.byref(norm_backward(T=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert size(ctypes.byref(norm_backward(T=4096, D=4096)), ctypes.byref(n)) == 0 and n.value > 0
    assert size(ctypes.byref(norm_backward(D=0)), ctypes.byref(n)) == -1
    assert size(ctypes.byref(norm_backward()), None) == -1 and size(None, ctypes.byref(n)) == -1
    assert w4.lib().w4a16_norm_block(None, None) == -1
    assert w4.lib().w4a16_norm_block_backward(None, None, 0, None) == -1


def routing(**kw):
    f = dict(T=4, E=64, k=8, score=0, groups=1, topk_groups=1, renormalize=1, scale=1.0, dtype=2)
    f.update(kw)
    return ex.RoutingStruct(*f.values())


ROUTING_REFUSALS = [
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(E=0), -1), (dict(E=1025), -1), (dict(k=0), -1), (dict(k=65), -1),
    (dict(E=4), -1), (dict(score=2), -3), (dict(score=-1), -3), (dict(dtype=3), -3), (dict(scale=float("inf")), -1),
    (dict(scale=float("nan")), -1), (dict(groups=0), -1), (dict(groups=3), -1), (dict(groups=128, E=256), -1),
    (dict(groups=8, topk_groups=9), -1), (dict(groups=8, topk_groups=0), -1), (dict(groups=16, topk_groups=1), -1),
]


@pytest.mark.parametrize("kw,code", ROUTING_REFUSALS)
def test_routing_refusals(kw, code):
    r = routing(**kw)
    L = w4.lib()
    assert L.w4a16_route(ctypes.byref(r), at(0), at(1), at(2), at(3), None) == code
    assert L.w4a16_route_backward(ctypes.byref(r), at(0), at(1), at(2), at(3), None) == code


def test_route_pointers():
    L, r = w4.lib(), routing()
    good = [at(0), at(1), at(2), at(3)]
    for i in range(4):
        for value, code in ((None, -1), (ODD, -2)):
            args = list(good)
            args[i] = value
            if not (i == 1 and value is None):     # (no bias)
                assert L.w4a16_route(ctypes.byref(r), *args, None) == code
            assert L.w4a16_route_backward(ctypes.byref(r), *args, None) == code
    assert L.w4a16_route(ctypes.byref(r), at(0), at(1), at(2), at(2), None) == -1
    assert L.w4a16_route(ctypes.byref(r), at(0), at(1), at(0) + 64, at(2), None) == -1
    assert L.w4a16_route(ctypes.byref(r), at(0), at(1), at(2), at(1) + 128, None) == -1
    for i in range(3):
        args = list(good)
        args[3] = args[i]
        assert L.w4a16_route_backward(ctypes.byref(r), *args, None) == -1
    assert L.w4a16_route(None, *good, None) == -1
    r = routing(T=0)
    assert L.w4a16_route(ctypes.byref(r), None, None, None, None, None) == 0
    assert L.w4a16_route_backward(ctypes.byref(r), None, None, None, None, None) == 0


def experts_call(**kw):
    weight = [ex.ExpertWeightStruct(at(40 + 3 * i), at(41 + 3 * i), at(42 + 3 * i)) for i in range(3)]
    f = dict(X=at(0), ids=at(1), weights=at(2), gate=weight[0], up=weight[1], down=weight[2], s=at(3), s_down=at(4),
             residual=at(5), G=at(6), U=at(7), Y=at(8), T=4, E=8, k=2, D=256, N=128, act=2, dtype=0)
    f.update(kw)
    return ex.ExpertsStruct(*f.values())


def experts_rc(ws=at(20), nbytes=1 << 25, **kw):
    return w4.lib().w4a16_experts(ctypes.byref(experts_call(**kw)), ws, nbytes, None)


EXPERT_SHAPES = [
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(E=0), -1), (dict(E=1025), -1), (dict(k=0), -1), (dict(k=65), -1),
    (dict(D=0), -1), (dict(D=64), -1), (dict(D=200), -1), (dict(N=192), -1), (dict(N=1 << 21), -1),
    (dict(D=1 << 16, N=1 << 16), -1), (dict(act=5), -3), (dict(act=-1), -3), (dict(dtype=2), -3),
]


@pytest.mark.parametrize("kw,code", EXPERT_SHAPES + [
    (dict(X=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(Y=None), -1), (dict(G=None), -1),
    (dict(U=None), -1), (dict(gate=ex.ExpertWeightStruct(at(1), None, at(2))), -1),
    (dict(down=ex.ExpertWeightStruct(at(1), at(2), ODD)), -2), (dict(X=ODD), -2), (dict(ids=ODD), -2),
    (dict(weights=ODD), -2), (dict(s=ODD), -2), (dict(s_down=ODD), -2), (dict(residual=ODD), -2), (dict(G=ODD), -2),
    (dict(Y=ODD), -2), (dict(ws=None), -1), (dict(nbytes=64), -1), (dict(ws=at(20) + 16), -2), (dict(Y=at(0)), -1),
    (dict(Y=at(5) + 16), -1), (dict(G=at(7)), -1), (dict(Y=at(20)), -1), (dict(U=at(40)), -1), (dict(Y=at(4)), -1),
    (dict(ws=at(0)), -1), (dict(G=at(5)), -1), (dict(T=0, X=None), 0),
])
def test_experts_refusals(kw, code):
    assert experts_rc(**kw) == code


def experts_backward(**kw):
    weight = [ex.ExpertTransposedStruct(at(40 + 2 * i), at(41 + 2 * i)) for i in range(3)]
    f = dict(dY=at(0), ids=at(1), weights=at(2), G=at(3), U=at(4), gate=weight[0], up=weight[1], down=weight[2], s=at(5),
             s_down=at(6), add=at(7), dX=at(8), dweights=at(9), T=4, E=8, k=2, D=256, N=128, act=2, dtype=0)
    f.update(kw)
    return ex.ExpertsBackwardStruct(*f.values())


def experts_backward_rc(ws=at(20), nbytes=1 << 25, **kw):
    return w4.lib().w4a16_experts_backward(ctypes.byref(experts_backward(**kw)), ws, nbytes, None)


@pytest.mark.parametrize("kw,code", EXPERT_SHAPES + [
    (dict(dY=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(G=None), -1), (dict(U=None), -1),
    (dict(dX=None), -1), (dict(dX=None, add=None, dweights=None), -1),
    (dict(up=ex.ExpertTransposedStruct(None, at(2))), -1), (dict(gate=ex.ExpertTransposedStruct(at(1), ODD)), -2),
    (dict(dY=ODD), -2), (dict(G=ODD), -2), (dict(add=ODD), -2), (dict(dX=ODD), -2), (dict(dweights=ODD), -2),
    (dict(ws=None), -1), (dict(nbytes=64), -1), (dict(ws=at(20) + 128), -2), (dict(dX=at(0)), -1), (dict(dX=at(3)), -1),
    (dict(dweights=at(8)), -1), (dict(dX=at(7) + 32), -1), (dict(dweights=at(7)), -1), (dict(dX=at(20)), -1),
    (dict(dweights=at(7) - 16, dweights_f32=1), -1),   # 8 slots: 32 bytes in fp32
    (dict(T=0, dY=None), 0),
])
def test_experts_backward_refusals(kw, code):
    assert experts_backward_rc(**kw) == code


def test_experts_sizes():
    L, n = w4.lib(), ctypes.c_size_t()
    for size, call in ((L.w4a16_experts_workspace_size, experts_call),
                       (L.w4a16_experts_backward_workspace_size, experts_backward)):
        assert size(ctypes.byref(call(T=0)), ctypes.byref(n)) == 0 and n.value == 0
        assert size(ctypes.byref(call()), ctypes.byref(n)) == 0 and 0 < n.value < 1 << 20
        # bounded whatever the number of tokens: at most 2^17 slots a round
        assert size(ctypes.byref(call(T=1 << 22, D=4096, N=1024)), ctypes.byref(n)) == 0
        assert n.value < (1 << 17) * (4 * 4096 + 4 * 1024 + 256) + (1 << 30)
        assert size(ctypes.byref(call(D=100)), ctypes.byref(n)) == -1
        assert size(ctypes.byref(call()), None) == -1 and size(None, ctypes.byref(n)) == -1
    assert L.w4a16_experts(None, None, 0, None) == -1 and L.w4a16_experts_backward(None, None, 0, None) == -1


def test_binding_refuses_what_is_not_a_device_tensor():
    import torch
    x = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(TypeError):
        w4.w4a16_norm_block(x, pre=w4.Norm())
    with pytest.raises(TypeError):
        w4.w4a16_norm_block(x.float(), pre=w4.Norm())
    with pytest.raises(TypeError):
        w4.w4a16_route(x, w4.Routing(2))
    with pytest.raises(TypeError):
        w4.w4a16_route(x.int(), w4.Routing(2))
    with pytest.raises(ValueError):
        w4.w4a16_norm_block_backward(None, None)
    g = torch.zeros(4, 8, requires_grad=True)
    with pytest.raises(ValueError):
        w4.w4a16_route(g, w4.Routing(2))
    with pytest.raises(ValueError):
        w4.w4a16_norm_block(g.half(), pre=w4.Norm())


def test_stacking_refuses_unlike_weights():
    a, b = w4.PackedWeight(None, None, None, 128, 128), w4.PackedWeight(None, None, None, 128, 256)
    c = w4.PackedWeight(None, None, None, 128, 128, wbits=8)
    for bad in ([], [a, b], [a, c], [c]):
        with pytest.raises(ValueError):
            w4.w4a16_stack_experts(bad)


@pytest.mark.parametrize("source", ["norm.hip", "route.hip", "experts.hip"])
def test_block_kernels_keep_everything_in_registers(source, tmp_path):
    kernels = _kernel_metadata(_device_asm(source, tmp_path))
    assert kernels
    bad = [k for k in kernels if k[1] or k[2] or k[3]]
    assert not bad, f"{source}: (kernel, private bytes, VGPR spills, SGPR spills): {bad}"


def test_gate_of_an_empty_batch():
    """A gate of one row serves all tokens, also where there are none."""
    import torch
    for shape, want in (((64,), (64,)), ((1, 64), (1, 64)), ((0, 64), (0, 64))):
        assert ex._gate_shape(torch.zeros(shape), None, 0, 64)[0] == want
    assert ex._gate_shape(torch.zeros(1, 64), 5, 0, 64)[0] == (1, 64)
    assert ex._gate_shape(torch.zeros(2, 64), 5, 0, 64)[0] == (0, 64)      # refused: two rows for no token


@pytest.mark.parametrize("rows", [4, 1 << 40, (1 << 63) - 1])
def test_one_gate_for_all_is_checked_whatever_its_rows(rows):
    """An output over the gate is refused, also where T + gate_rows would pass 64 bits."""
    for kw in (dict(h=at(2)), dict(r=at(2)), dict(h=at(2) + 64)):
        assert norm_rc(gate_rows=rows, **kw) == -1
    for kw in (dict(dx=at(4)), dict(dy=at(4) + 64), dict(dgate=at(4)), dict(dgate=at(9) + 256), dict(dgate=at(2))):
        assert norm_backward_rc(gate_rows=rows, **kw) == -1


@pytest.mark.parametrize("rows", [5, 1 << 40, 1 << 63, (1 << 64) + 1])
def test_gate_rows_reach_the_library_whole(rows):
    """Rows past 64 bits would wrap on their way (2^64 + 1 to a gate vector per token, of which one is there)."""
    import torch
    shape, n = ex._gate_shape(torch.zeros(1, 8), rows, 5, 8)
    assert shape == (1, 8) and ex.NormCallStruct(gate_rows=n).gate_rows >= 5


def test_norm_block_without_work_checks_its_arguments():
    """Without y, pre and alpha there is nothing to launch; what is refused beside them is refused here too."""
    import torch
    x = torch.zeros(4, 8, dtype=torch.float16)
    for alpha in (1.0, 0.5):
        for kw in (dict(post=w4.Norm()), dict(gate=x[0]), dict(post=w4.Norm(w4.NORM_LAYER), gate=x)):
            with pytest.raises(ValueError):
                w4.w4a16_norm_block(x, alpha=alpha, **kw)
        for bad in (x, x.float(), None):
            with pytest.raises(TypeError):
                w4.w4a16_norm_block(bad, alpha=alpha)
        with pytest.raises(ValueError):
            w4.w4a16_norm_block(x.clone().requires_grad_(), alpha=alpha)
        with pytest.raises(ValueError):
            w4.w4a16_norm_block(x[0], alpha=alpha)
