"""What the training operators refuse, on the host and before a device is
touched.  Addresses are never dereferenced there: 0x1000 stands for an
aligned device pointer, 0x1004 and 0x1001 for misaligned ones."""

import ctypes as C

import pytest

from nvfp4_mixture_experts_counting_gb300 import build as build_mod
from nvfp4_mixture_experts_counting_gb300 import ftmoe

A, B, D, ODD, OFF = 0x1000, 0x2000, 0x3000, 0x1001, 0x1004
OK, ARG, ALIGN, DEVICE = 0, -1, -2, -9


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return ftmoe.lib()


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def check(lib, name, good, cases):
    """The refusals of `cases` ({argument place: value}, status); what is not refused reaches the device check."""
    f = getattr(lib, name)
    if no_gpu():
        assert f(*good) == DEVICE
    for change, status in cases:
        args = list(good)
        for at, value in change.items():
            args[at] = value
        if status != DEVICE or no_gpu():
            assert f(*args) == status, (name, change)


def test_dispatch(lib):
    # x dtype T H idx k E offsets perm inv xs stream
    good = [A, 0, 4, 16, A, 2, 8, A, A, A, B, None]
    check(lib, "ftmoe_dispatch", good, [
        ({1: 3}, ARG), ({1: -1}, ARG), ({2: -1}, ARG), ({3: 0}, ARG), ({3: 1 << 25}, ARG), ({5: 0}, ARG), ({5: 33}, ARG),
        ({2: 1 << 30, 5: 2}, ARG), ({6: 0}, ARG), ({6: 1025}, ARG), ({4: None}, ARG), ({7: None}, ARG), ({8: None}, ARG),
        ({9: None}, ARG), ({0: None}, ARG), ({10: None}, ARG), ({10: A}, ARG), ({0: OFF}, ALIGN), ({10: OFF}, ALIGN),
        ({4: ODD}, ALIGN), ({7: ODD}, ALIGN), ({0: None, 10: None}, DEVICE), ({2: 0}, DEVICE), ({3: 17}, DEVICE)])


def test_combine(lib):
    # ys dtype T H k inv w out stream
    good = [A, 0, 4, 16, 2, A, A, B, None]
    check(lib, "ftmoe_combine", good, [
        ({1: 9}, ARG), ({2: -1}, ARG), ({3: -3}, ARG), ({4: 40}, ARG), ({0: None}, ARG), ({5: None}, ARG), ({7: None}, ARG),
        ({7: A}, ARG), ({0: OFF}, ALIGN), ({7: OFF}, ALIGN), ({5: ODD}, ALIGN), ({6: ODD}, ALIGN), ({6: None}, DEVICE),
        ({2: 0, 0: None}, OK)])


def test_combine_backward(lib):
    # dout ys dtype T H k inv w dys dw stream
    good = [A, B, 0, 4, 16, 2, A, A, D, A, None]
    check(lib, "ftmoe_combine_backward", good, [
        ({2: 4}, ARG), ({3: -1}, ARG), ({5: 0}, ARG), ({0: None}, ARG), ({1: None}, ARG), ({6: None}, ARG), ({7: None}, ARG),
        ({8: None}, ARG), ({9: None}, ARG), ({8: A}, ARG), ({8: B}, DEVICE), ({0: OFF}, ALIGN), ({1: OFF}, ALIGN),
        ({8: OFF}, ALIGN), ({9: ODD}, ALIGN), ({3: 0}, OK)])


def test_route_backward(lib):
    # logits idx w dw T E k norm dlogits stream
    good = [A, A, A, A, 4, 8, 2, 0, B, None]
    check(lib, "ftmoe_route_backward", good, [
        ({4: -1}, ARG), ({5: 0}, ARG), ({5: 1025}, ARG), ({6: 9}, ARG), ({6: 0}, ARG), ({0: None}, ARG), ({1: None}, ARG),
        ({2: None}, ARG), ({3: None}, ARG), ({8: None}, ARG), ({0: None, 7: 1}, DEVICE), ({8: ODD}, ALIGN), ({4: 0}, OK)])


def test_embed(lib):
    # table dtype V H ids id_bytes N scale out stream
    good = [A, 0, 100, 16, A, 8, 4, 1.0, B, None]
    check(lib, "ftmoe_embed", good, [
        ({1: 7}, ARG), ({2: 0}, ARG), ({2: 1 << 31}, ARG), ({3: 0}, ARG), ({5: 2}, ARG), ({6: -1}, ARG), ({6: 1 << 31}, ARG),
        ({0: None}, ARG), ({4: None}, ARG), ({8: None}, ARG), ({8: A}, ARG), ({0: OFF}, ALIGN), ({8: OFF}, ALIGN),
        ({4: OFF}, ALIGN), ({4: OFF, 5: 4}, DEVICE), ({6: 0}, OK)])


def test_embed_backward(lib):
    # dout dtype ids id_bytes N V H scale padding dtable table_dtype accumulate ws ws_bytes stream
    need = lib.ftmoe_embed_workspace(40, 16)
    assert need >= 40 * 16 + 2 * 2 * 16 * 4
    good = [A, 0, A, 4, 40, 100, 16, 1.0, -1, B, 1, 0, D, need, None]
    check(lib, "ftmoe_embed_backward", good, [
        ({1: 5}, ARG), ({10: 2}, ARG), ({1: 1, 10: 0}, ARG), ({10: 0, 11: 1}, ARG), ({3: 3}, ARG), ({4: -2}, ARG), ({5: 0}, ARG),
        ({6: 0}, ARG), ({0: None}, ARG), ({2: None}, ARG), ({9: None}, ARG), ({9: A}, ARG), ({12: None}, ARG),
        ({13: need - 1}, ARG), ({0: OFF}, ALIGN), ({9: OFF}, ALIGN), ({12: OFF}, ALIGN), ({2: ODD}, ALIGN),
        ({4: 0, 0: None, 2: None, 12: None, 13: 0}, DEVICE), ({11: 1}, DEVICE)])
    assert lib.ftmoe_embed_workspace(-1, 16) == ARG and lib.ftmoe_embed_workspace(4, 0) == ARG
    assert lib.ftmoe_embed_workspace(0, 16) == 0


def policy(**kw):
    base = dict(logits=A, dtype=0, id_bytes=8, N=4, V=10, ld=10, targets=A, old_logp=A, ref_logp=A, advantage=A, weight=A,
                temperature=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.0, grad_scale=1.0, loss=A, row_loss=A, logp=A,
                dlogits=B, ld_d=10)
    base.update(kw)
    return ftmoe.PolicyArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), ARG), (dict(id_bytes=2), ARG), (dict(N=-1), ARG), (dict(V=0), ARG), (dict(ld=9), ARG), (dict(ld_d=9), ARG),
    (dict(temperature=0.0), ARG), (dict(temperature=float("nan")), ARG), (dict(temperature=float("inf")), ARG),
    (dict(clip_low=-0.1), ARG), (dict(clip_high=float("nan")), ARG), (dict(kl_coef=float("inf")), ARG),
    (dict(grad_scale=float("nan")), ARG), (dict(loss=None), ARG), (dict(row_loss=None), ARG), (dict(logits=None), ARG),
    (dict(targets=None), ARG), (dict(old_logp=None), ARG), (dict(advantage=None), ARG), (dict(dlogits=A, ld=12), ARG),
    (dict(logits=ODD), ALIGN), (dict(dlogits=ODD), ALIGN), (dict(targets=OFF), ALIGN), (dict(loss=ODD), ALIGN),
    (dict(dtype=1, logits=0x1002), ALIGN), (dict(dlogits=None, ld_d=0), DEVICE), (dict(ref_logp=None, weight=None), DEVICE),
    (dict(logits=0x1002), DEVICE), (dict(dlogits=A), DEVICE)])
def test_policy_loss(lib, kw, status):
    if status != DEVICE or no_gpu():
        assert lib.ftmoe_policy_loss(C.byref(policy(**kw)), None) == status


def test_policy_loss_without_arguments(lib):
    assert lib.ftmoe_policy_loss(None, None) == ARG


def adam(hp=None, **kw):
    base = dict(p=A, g=A, master=None, m=A, v=A, m_scale=None, v_scale=None, n=8, weight_decay=0.0, p_dtype=0, g_dtype=0,
                state_bits=32)
    base.update(kw)
    params = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, grad_scale=None)
    params.update(hp or {})
    return (ftmoe.AdamwTensor * 1)(ftmoe.AdamwTensor(**base)), ftmoe.AdamwParams(**params)


@pytest.mark.parametrize("hp,kw,status", [
    (dict(beta1=1.0), {}, ARG), (dict(beta2=-0.1), {}, ARG), (dict(eps=-1e-9), {}, ARG), (dict(step=0), {}, ARG),
    (dict(lr=float("nan")), {}, ARG), (dict(grad_scale=ODD), {}, ALIGN), ({}, dict(n=-1), ARG), ({}, dict(p=None), ARG),
    ({}, dict(g=None), ARG), ({}, dict(m=None), ARG), ({}, dict(v=None), ARG), ({}, dict(p_dtype=3), ARG),
    ({}, dict(g_dtype=2), ARG), ({}, dict(state_bits=16), ARG), ({}, dict(state_bits=8), ARG),
    ({}, dict(p_dtype=1, g_dtype=1, master=A), ARG), ({}, dict(weight_decay=float("inf")), ARG), ({}, dict(p=ODD), ALIGN),
    ({}, dict(m=0x1002), ALIGN), ({}, dict(master=0x1002), ALIGN), ({}, dict(p=0x1002, g=0x1002), DEVICE),
    ({}, dict(state_bits=8, m=ODD, v=ODD, m_scale=A, v_scale=A), DEVICE), ({}, dict(n=0, p=None), OK)])
def test_adamw(lib, hp, kw, status):
    tensors, params = adam(hp, **kw)
    if status != DEVICE or no_gpu():
        assert lib.ftmoe_adamw(tensors, 1, C.byref(params), None) == status


def test_adamw_lists(lib):
    tensors, params = adam()
    assert lib.ftmoe_adamw(tensors, -1, C.byref(params), None) == ARG
    assert lib.ftmoe_adamw(None, 1, C.byref(params), None) == ARG
    assert lib.ftmoe_adamw(tensors, 1, None, None) == ARG
    assert lib.ftmoe_adamw(None, 0, C.byref(params), None) == OK


def test_status_without_a_gpu(lib):
    if no_gpu():
        assert lib.ftmoe_ops_status(None) == DEVICE


def test_binding_refuses_wrong_types_and_sizes(lib):
    """Before any call: on a device the addresses would be read as what they are not."""
    torch = pytest.importorskip("torch")
    new = lambda n, dtype=torch.float32: torch.zeros(n, dtype=dtype)
    half, wide = torch.bfloat16, torch.int64
    x, idx, w = new((4, 16), half), new((4, 2), torch.int32), new((4, 2))
    tables = new(9, torch.int32), new(8, torch.int32), new(8, torch.int32)
    with pytest.raises(TypeError):
        ftmoe.ftmoe_dispatch(x, 4, 16, idx.long(), 2, 8, *tables, new((8, 16), half), stream=0)
    for inv, weights in ((tables[1].long(), w), (tables[1], w.to(half))):
        with pytest.raises(TypeError):
            ftmoe.ftmoe_combine(new((8, 16), half), 4, 16, 2, inv, weights, x, stream=0)
    with pytest.raises(TypeError):
        ftmoe.ftmoe_route_backward(new((4, 8), half), idx, w, w, 4, 8, 2, False, new((4, 8)), stream=0)
    with pytest.raises(TypeError):
        ftmoe.ftmoe_embed(x.int(), 4, 16, new(3, wide), 3, 1.0, new((3, 16), half), stream=0)

    def args(**kw):
        a = dict(logits=new((4, 10), half), targets=new(4, wide), old_logp=new(4), ref_logp=new(4), advantage=new(4),
                 weight=new(4), loss=new(1), row_loss=new(4), logp=new(4), dlogits=new((4, 10), half))
        a.update(kw)
        return ftmoe.policy_args(**a)

    assert args().N == 4 and args(ref_logp=None, weight=None, logp=None, dlogits=None).V == 10
    for kw in (dict(targets=new(3, wide)), dict(old_logp=new(3)), dict(advantage=new(4, half)), dict(weight=new(2)),
               dict(loss=new(0)), dict(row_loss=new(3)), dict(logp=new(4, torch.float64)), dict(dlogits=new((4, 10))),
               dict(dlogits=new((4, 9), half)), dict(logits=new((10, 4), half).t()), dict(ref_logp=new(8)[::2])):
        with pytest.raises((TypeError, ValueError)):
            args(**kw)

    def tensors(**kw):
        a = dict(p=new(300, half), g=new(300, half), m=new(300, torch.uint8), v=new(300, torch.uint8), m_scale=new(2),
                 v_scale=new(2))
        a.update(kw)
        return ftmoe.adamw_list([a])

    assert tensors().array[0].n == 300 and tensors().array[0].state_bits == 8
    for kw in (dict(g=new(299, half)), dict(m=new(299, torch.uint8)), dict(v=new(300)), dict(v_scale=new(1)),
               dict(m_scale=new(2, half)), dict(master=new(299)), dict(master=new(300, half)), dict(p=new(300, wide)),
               dict(p=new(600, half)[::2])):
        with pytest.raises((TypeError, ValueError)):
            tensors(**kw)
