"""What the calls of the 8-bit layer refuse, on the host and before a device is
touched (addresses are never dereferenced there), and what their binding
refuses before the call."""

import ctypes as C

import pytest
import torch

from nvfp4_mixture_experts_counting_gb300 import ftmoe

from test_train_ops_cpu import A, ALIGN, ARG, B, D, DEVICE, ODD, OFF, OK, check, lib, no_gpu  # noqa: F401

E4M3 = torch.float8_e4m3fn


def check_struct(call, good, cases):
    if no_gpu():
        assert call(good) == DEVICE
    for change, status in cases:
        if status != DEVICE or no_gpu():
            assert call({**good, **change}) == status, change


ROUTE = dict(logits=A, dtype=0, T=4, E=16, ld=16, score=0, top_k=2, norm_topk_prob=1, scale=1.0, bias=None, n_groups=1,
             top_groups=1, group_best=1, topk_idx=B, topk_w=D)
ROUTE_REFUSED = [
    (dict(logits=None), ARG), (dict(dtype=3), ARG), (dict(T=-1), ARG), (dict(E=0), ARG), (dict(E=1025, ld=1025), ARG),
    (dict(ld=15), ARG), (dict(score=2), ARG), (dict(score=-1), ARG), (dict(top_k=0), ARG), (dict(top_k=17), ARG),
    (dict(E=64, ld=64, top_k=33), ARG), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(n_groups=0), ARG), (dict(n_groups=3), ARG),
    (dict(E=64, ld=64, n_groups=64), ARG), (dict(n_groups=4, top_groups=0), ARG), (dict(n_groups=4, top_groups=5), ARG),
    (dict(n_groups=8, top_groups=1, top_k=3), ARG), (dict(group_best=0), ARG), (dict(group_best=3), ARG),
    (dict(topk_idx=None), ARG), (dict(topk_w=None), ARG), (dict(logits=ODD), ALIGN), (dict(bias=0x1002), ALIGN),
    (dict(topk_idx=ODD), ALIGN), (dict(topk_w=0x1002), ALIGN), (dict(T=0, logits=None), OK),
    (dict(n_groups=4, top_groups=2, group_best=2, bias=A), DEVICE), (dict(logits=0x1002), DEVICE),
    (dict(ld=1 << 33), DEVICE)]


def test_route(lib):  # noqa: F811
    check_struct(lambda v: lib.ftmoe_route_topk(C.byref(ftmoe.RouteArgs(**v)), None), ROUTE, ROUTE_REFUSED)
    assert lib.ftmoe_route_topk(None, None) == ARG


def test_route_backward(lib):  # noqa: F811
    def call(v):
        v = dict(v)
        dw, dl, ld = v.pop("dw"), v.pop("dl"), v.pop("ld_d")
        return lib.ftmoe_route_topk_backward(C.byref(ftmoe.RouteArgs(**v)), dw, dl, ld, None)
    good = dict(ROUTE, dw=A, dl=0x9000, ld_d=16)
    wide = [({**c, "ld_d": c["E"]} if c.get("E", 0) > 16 else c, s) for c, s in ROUTE_REFUSED]
    check_struct(call, good, wide + [
        (dict(dw=None), ARG), (dict(dl=None), ARG), (dict(ld_d=15), ARG), (dict(dl=A, ld_d=17), ARG), (dict(dw=ODD), ALIGN),
        (dict(dl=0x9001), ALIGN), (dict(dl=A), DEVICE), (dict(dl=0x9002), DEVICE)])


def test_quantize(lib):  # noqa: F811
    # x dtype T K inv top_k used codes scales stream
    good = [A, 0, 4, 128, A, 2, None, B, D, None]
    check(lib, "ftmoe_fp8_quantize", good, [
        ({0: None}, ARG), ({1: 4}, ARG), ({2: -1}, ARG), ({3: 0}, ARG), ({3: 1 << 25}, ARG), ({5: 0}, ARG), ({5: 33}, ARG),
        ({4: None}, ARG), ({2: 1 << 30, 5: 2}, ARG), ({7: None}, ARG), ({8: None}, ARG), ({7: A}, ARG), ({3: 120}, ALIGN),
        ({0: OFF}, ALIGN), ({7: OFF}, ALIGN), ({8: ODD}, ALIGN), ({4: ODD}, ALIGN), ({6: ODD}, ALIGN), ({2: 0, 0: None}, OK),
        ({4: None, 5: 1}, DEVICE), ({6: A}, DEVICE), ({3: 144}, DEVICE)])


def test_quantize_weights(lib):  # noqa: F811
    # w dtype E N K codes scales stream
    good = [A, 0, 2, 130, 144, B, D, None]
    check(lib, "ftmoe_fp8_quantize_weights", good, [
        ({0: None}, ARG), ({1: -1}, ARG), ({2: -1}, ARG), ({2: 1025}, ARG), ({3: 0}, ARG), ({4: 0}, ARG),
        ({3: 1 << 24, 4: 1 << 24}, ARG), ({5: None}, ARG), ({6: None}, ARG), ({5: A}, ARG), ({4: 136}, ALIGN),
        ({0: OFF}, ALIGN), ({5: OFF}, ALIGN), ({6: ODD}, ALIGN), ({2: 0, 0: None}, OK)])


def test_matmul(lib):  # noqa: F811
    good = dict(a=A, a_scale=A, w=A, w_scale=A, offsets=A, M=8, E=4, N=256, K=128, transpose=0, swiglu=0, out_dtype=0,
                out=B, out_scale=None)
    check_struct(lambda v: lib.ftmoe_fp8_matmul(C.byref(ftmoe.Fp8MatmulArgs(**v)), None), good, [
        (dict(M=-1), ARG), (dict(M=1 << 31), ARG), (dict(E=0), ARG), (dict(E=1025), ARG), (dict(N=0), ARG), (dict(K=0), ARG),
        (dict(N=(1 << 24) + 1), ARG), (dict(offsets=None), ARG), (dict(transpose=1, swiglu=1, out_scale=D), ARG),
        (dict(out_dtype=3), ARG), (dict(a=None), ARG), (dict(a_scale=None), ARG), (dict(w=None), ARG),
        (dict(w_scale=None), ARG), (dict(out=None), ARG), (dict(out=A), ARG), (dict(swiglu=1), ARG), (dict(K=120), ALIGN),
        (dict(transpose=1, N=250), ALIGN), (dict(swiglu=1, out_scale=D, N=384), ALIGN), (dict(a=OFF), ALIGN),
        (dict(w=OFF), ALIGN), (dict(out=OFF), ALIGN), (dict(a_scale=ODD), ALIGN), (dict(w_scale=ODD), ALIGN),
        (dict(offsets=ODD), ALIGN), (dict(swiglu=1, out_scale=ODD), ALIGN), (dict(M=0, a=None), OK),
        (dict(N=333), DEVICE), (dict(transpose=1, N=144), DEVICE), (dict(swiglu=1, out_scale=D, out_dtype=9), DEVICE),
        (dict(offsets=None, E=1), DEVICE)])
    assert lib.ftmoe_fp8_matmul(None, None) == ARG


def test_matmul_strides_and_aliases(lib):  # noqa: F811
    good = dict(a=A, a_scale=A, w=A, w_scale=A, offsets=A, M=8, E=4, N=256, K=128, transpose=0, swiglu=1, out_dtype=0,
                out=B, out_scale=D)
    check_struct(lambda v: lib.ftmoe_fp8_matmul(C.byref(ftmoe.Fp8MatmulArgs(**v)), None), good, [
        (dict(N=1 << 20, K=1 << 20), ARG), (dict(N=1 << 20, K=(1 << 20) - 16), DEVICE), (dict(out_scale=A), ARG)])


def test_swiglu(lib):  # noqa: F811
    # gu dtype rows I used out scales stream
    check(lib, "ftmoe_swiglu", [A, 0, 4, 128, None, B, D, None], [
        ({0: None}, ARG), ({1: 5}, ARG), ({2: -1}, ARG), ({3: 0}, ARG), ({5: None}, ARG), ({5: A}, ARG), ({3: 120}, ALIGN),
        ({0: OFF}, ALIGN), ({5: OFF}, ALIGN), ({6: ODD}, ALIGN), ({4: ODD}, ALIGN), ({2: 0, 0: None}, OK),
        ({6: None, 3: 7}, DEVICE), ({6: None, 5: A}, ARG)])
    # dh gu dtype rows I used dgu scales stream
    check(lib, "ftmoe_swiglu_backward", [A, B, 0, 4, 128, None, D, 0x5000, None], [
        ({0: None}, ARG), ({1: None}, ARG), ({6: None}, ARG), ({6: A}, ARG), ({6: B}, ARG), ({2: 7}, ARG), ({4: 130}, ALIGN),
        ({0: OFF}, ALIGN), ({1: OFF}, ALIGN), ({6: OFF}, ALIGN), ({7: ODD}, ALIGN), ({3: 0, 0: None}, OK),
        ({7: None, 6: B}, DEVICE), ({7: None, 4: 3}, DEVICE)])


def test_packed_arguments():
    """The packed fields are the structures'."""
    for packed, struct in ((ftmoe._ROUTE, ftmoe.RouteArgs), (ftmoe._MATMUL, ftmoe.Fp8MatmulArgs)):
        fields = struct._fields_
        values = [0.5 if t is C.c_float else 3 + i for i, (_, t) in enumerate(fields)]
        args = struct()
        packed.pack_into(args, 0, *values)
        assert [getattr(args, n) for n, _ in fields] == values
        assert packed.size <= C.sizeof(struct) < packed.size + 8


def test_binding_refuses():
    """Tensors of a wrong type, shape or size never reach the library."""
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    i32 = torch.int32
    with pytest.raises(TypeError):
        ftmoe.route_args(z(4, 8, dtype=torch.float64), z(4, 2, dtype=i32), z(4, 2))
    with pytest.raises(TypeError):
        ftmoe.route_args(z(4, 8), z(4, 2, dtype=torch.int64), z(4, 2))
    with pytest.raises(ValueError):
        ftmoe.route_args(z(4, 8), z(3, 2, dtype=i32), z(3, 2))
    with pytest.raises(ValueError):
        ftmoe.route_args(z(8, 4).t(), z(4, 2, dtype=i32), z(4, 2))
    with pytest.raises(ValueError):
        ftmoe.route_args(z(4, 8), z(4, 2, dtype=i32), z(4, 2), bias=z(7))
    with pytest.raises(KeyError):
        ftmoe.route_args(z(4, 8), z(4, 2, dtype=i32), z(4, 2), score="tanh")
    args = ftmoe.route_args(z(4, 9)[:, :8], z(4, 2, dtype=i32), z(4, 2))
    assert args.ld == 9 and args.E == 8 and len(args.tensors) == 4
    with pytest.raises(TypeError):
        ftmoe.ftmoe_route_topk_backward(args, z(4, 2), z(4, 7))
    with pytest.raises(TypeError):
        ftmoe.ftmoe_route_topk_backward(args, z(4, 2), z(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ftmoe.ftmoe_route_topk_backward(args, z(4, 1), z(4, 8))
    codes, scales = z(4, 128, dtype=E4M3), z(1, 4)
    for bad in (dict(x=z(4, 127)), dict(codes=z(4, 128)), dict(codes=z(3, 128, dtype=E4M3)), dict(scales=z(1, 3)),
                dict(inv=z(3, dtype=i32)), dict(used=z(1))):
        v = {**dict(x=z(4, 128), inv=None, codes=codes, scales=scales, used=None), **bad}
        with pytest.raises((TypeError, ValueError)):
            ftmoe.ftmoe_fp8_quantize(v["x"], 4, 128, v["inv"], 1, v["codes"], v["scales"], used=v["used"])
    with pytest.raises(ValueError):
        ftmoe.ftmoe_fp8_quantize_weights(z(2, 130, 128), 2, 130, 128, z(2, 130, 128, dtype=E4M3), z(2, 1, 1))
    good = dict(a=codes, a_scale=scales, w=z(2, 256, 128, dtype=E4M3), w_scale=z(2, 2, 1), offsets=z(3, dtype=i32),
                out=z(4, 256), out_scale=None, transpose=False, swiglu=False)
    for bad in (dict(a=z(4, 128)), dict(a_scale=z(1, 3)), dict(w=z(2, 255, 128, dtype=E4M3)), dict(w_scale=z(2, 1, 1)),
                dict(offsets=z(2, dtype=i32)), dict(out=z(4, 255)), dict(out=z(4, 256, dtype=torch.float64)),
                dict(transpose=True), dict(swiglu=True), dict(swiglu=True, out=z(4, 128, dtype=E4M3), out_scale=z(1, 3))):
        v = {**good, **bad}
        with pytest.raises((TypeError, ValueError)):
            ftmoe.ftmoe_fp8_matmul(v["a"], v["a_scale"], v["w"], v["w_scale"], v["offsets"], 4, 2, 256, 128, v["out"],
                                   v["out_scale"], transpose=v["transpose"], swiglu=v["swiglu"])
    with pytest.raises(TypeError):
        ftmoe.ftmoe_swiglu(z(4, 256), 4, 128, z(4, 128), scales)
    with pytest.raises(TypeError):
        ftmoe.ftmoe_swiglu(z(4, 256), 4, 128, codes)
    with pytest.raises(ValueError):
        ftmoe.ftmoe_swiglu_backward(z(4, 128), z(4, 256), 4, 128, z(4, 256, dtype=E4M3), z(1, 4))


def test_withhold_matmul_limits(lib):  # noqa: F811
    for limit in (-1, 1_000_000_001):
        with pytest.raises(ftmoe.FtmoeError):
            ftmoe.ftmoe_test_withhold_matmul(True, limit)
    ftmoe.ftmoe_test_withhold_matmul(True, 1_000_000_000)
    ftmoe.ftmoe_test_withhold_matmul(False)
