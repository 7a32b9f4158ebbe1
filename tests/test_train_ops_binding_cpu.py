"""What the training operators' entry points and binding refuse or keep, on the host."""

import pytest

from nvfp4_mixture_experts_counting_gb300 import build as build_mod
from nvfp4_mixture_experts_counting_gb300 import ftmoe


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return ftmoe.lib()


def test_withhold_policy_limits(lib):
    for limit in (-1, 1_000_000_001):
        with pytest.raises(ftmoe.FtmoeError):
            ftmoe.ftmoe_test_withhold_policy(True, limit)
    ftmoe.ftmoe_test_withhold_policy(True, 1_000_000_000)
    ftmoe.ftmoe_test_withhold_policy(False)


def test_policy_args_keep_their_tensors():
    """The block holds addresses: what it was made of lives as long as it does."""
    torch = pytest.importorskip("torch")
    import weakref
    N, V = 4, 10
    made = dict(logits=torch.zeros(N, V), targets=torch.zeros(N, dtype=torch.int64), old_logp=torch.zeros(N),
                ref_logp=torch.zeros(N), advantage=torch.zeros(N), weight=torch.zeros(N), loss=torch.zeros(1),
                row_loss=torch.zeros(N), logp=torch.zeros(N), dlogits=torch.zeros(N, V))
    alive = {n: weakref.ref(t) for n, t in made.items()}
    args = ftmoe.policy_args(**made)
    del made
    assert [n for n, r in alive.items() if r() is None] == []
    del args
    assert [n for n, r in alive.items() if r() is not None] == []


# what each call's tensors are: name -> (values, type); the rest of its arguments; the order
CALLS = {
    "ftmoe_dispatch": (dict(x=(64, "f16"), topk_idx=(8, "i32"), offsets=(6, "i32"), perm=(8, "i32"), inv=(8, "i32"),
                            xs=(128, "f16")), dict(T=4, H=16, top_k=2, E=5)),
    "ftmoe_combine": (dict(ys=(128, "f16"), inv=(8, "i32"), w=(8, "f32"), out=(64, "f16")), dict(T=4, H=16, top_k=2)),
    "ftmoe_combine_backward": (dict(dout=(64, "f16"), ys=(128, "f16"), inv=(8, "i32"), w=(8, "f32"),
                                    dys=(128, "f16"), dw=(8, "f32")), dict(T=4, H=16, top_k=2)),
    "ftmoe_route_backward": (dict(logits=(20, "f32"), topk_idx=(8, "i32"), topk_w=(8, "f32"), dw=(8, "f32"),
                                  dlogits=(20, "f32")), dict(T=4, E=5, top_k=2, norm_topk_prob=False)),
    "ftmoe_embed": (dict(table=(160, "f16"), ids=(7, "ids"), out=(112, "f16")), dict(V=10, H=16, N=7, scale=1.0)),
    "ftmoe_embed_backward": (dict(dout=(112, "any"), ids=(7, "ids"), dtable=(160, "any")),
                             dict(V=10, H=16, N=7, scale=1.0, padding_id=-1, accumulate=False, workspace=None)),
}


def tensors(name, **changed):
    """The call's tensors: `changed` gives some a kind of fault."""
    torch = pytest.importorskip("torch")
    types = {"f16": torch.float16, "f32": torch.float32, "i32": torch.int32, "ids": torch.int64, "any": torch.float32}
    made = {}
    for key, (n, kind) in CALLS[name][0].items():
        fault, dtype = changed.get(key), types[kind]
        if fault == "short":
            made[key] = torch.zeros(n - 1, dtype=dtype)
        elif fault == "strided":
            made[key] = torch.zeros(2 * n, dtype=dtype)[::2]
        elif fault is not None:
            made[key] = torch.zeros(n, dtype=getattr(torch, fault))
        else:
            made[key] = torch.zeros(n, dtype=dtype)
    return made


def faults():
    """Every tensor of every call: too short, strided, and of types of its own width and others."""
    wrong = {"f16": ["bfloat16", "float32", "int16", "uint8"], "f32": ["int32", "float64", "bfloat16"],
             "i32": ["float32", "int64", "int16"], "ids": ["float32", "float64", "int16"],
             "any": ["float64", "int32", "uint8"]}
    for name, (takes, _) in CALLS.items():
        for key, (_, kind) in takes.items():
            for fault in ["short", "strided"] + wrong[kind]:
                yield name, key, fault


class Recorder:
    """Stands for the library: a call that gets there is a call that a GPU would run."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture()
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ftmoe, "lib", lambda: r)
    return r


@pytest.mark.parametrize("name", CALLS)
def test_right_tensors_pass(recorder, name):
    getattr(ftmoe, name)(**tensors(name), **CALLS[name][1], stream=0)
    assert recorder.calls == [name]


@pytest.mark.parametrize("name,key,fault", list(faults()))
def test_wrong_tensors_are_refused(recorder, name, key, fault):
    """On a device the kernel would read or write past the buffer's end, or values of another type."""
    made = tensors(name, **{key: fault})
    with pytest.raises((TypeError, ValueError)):
        getattr(ftmoe, name)(**made, **CALLS[name][1], stream=0)
    assert recorder.calls == []


@pytest.mark.parametrize("key", ["old_logp", "ref_logp", "advantage", "weight", "loss", "row_loss", "logp", "targets",
                                 "dlogits", "logits"])
def test_policy_args_refuse_other_types(key):
    """Of the right bytes or the right count, but not the values that the kernel reads."""
    torch = pytest.importorskip("torch")
    N, V = 4, 10
    f = lambda n: torch.zeros(n)
    made = dict(logits=torch.zeros(N, V), targets=torch.zeros(N, dtype=torch.int32), old_logp=f(N), ref_logp=f(N),
                advantage=f(N), weight=f(N), loss=f(1), row_loss=f(N), logp=f(N), dlogits=torch.zeros(N, V))
    assert ftmoe.policy_args(**made).id_bytes == 4
    n = 1 if key == "loss" else N
    if key in ("logits", "dlogits"):
        wrong = [torch.zeros(N, V, dtype=t) for t in (torch.int32, torch.float64, torch.bfloat16)]
    elif key == "targets":
        wrong = [torch.zeros(N, dtype=t) for t in (torch.float32, torch.float64, torch.int16)] + [
            torch.zeros(N - 1, dtype=torch.int64), torch.zeros(2 * N, dtype=torch.int64)[::2]]
    else:
        wrong = [torch.zeros(n, dtype=torch.int32), torch.zeros(2 * n, dtype=torch.bfloat16),
                 torch.zeros(2 * n, dtype=torch.int16), torch.zeros(n, dtype=torch.float64)]
    for t in wrong:
        with pytest.raises((TypeError, ValueError)):
            ftmoe.policy_args(**{**made, key: t})


def adam_tensors(torch, bits=32, **changed):
    n, state = 300, torch.float32 if bits == 32 else torch.uint8
    t = dict(p=torch.zeros(n, dtype=torch.bfloat16), g=torch.zeros(n, dtype=torch.bfloat16),
             m=torch.zeros(n, dtype=state), v=torch.zeros(n, dtype=state), master=torch.zeros(n),
             m_scale=torch.zeros(2), v_scale=torch.zeros(2))
    t.update(changed)
    return t


def test_adamw_refuses_other_types(recorder):
    torch = pytest.importorskip("torch")
    for bits in (8, 32):
        made = ftmoe.adamw_list([adam_tensors(torch, bits)])
        ftmoe.ftmoe_adamw(made, 1e-3, grad_scale=torch.ones(1), stream=0)
        for scale in (torch.ones(1, dtype=torch.bfloat16), torch.ones(1, dtype=torch.float64), torch.ones(0),
                      torch.ones(1, dtype=torch.int32)):
            with pytest.raises((TypeError, ValueError)):
                ftmoe.ftmoe_adamw(made, 1e-3, grad_scale=scale, stream=0)
        for key, dtype, n in (("m_scale", torch.int32, 2), ("v_scale", torch.int32, 2), ("master", torch.int32, 300),
                              ("m", torch.int32, 300), ("v", torch.int32, 300), ("p", torch.int16, 300),
                              ("g", torch.int16, 300)):
            with pytest.raises((TypeError, ValueError)):
                ftmoe.adamw_list([adam_tensors(torch, bits, **{key: torch.zeros(n, dtype=dtype)})])
    with pytest.raises((TypeError, ValueError)):  # both of a type that is neither fp32 nor codes
        ftmoe.adamw_list([adam_tensors(torch, m=torch.zeros(300, dtype=torch.int32),
                                       v=torch.zeros(300, dtype=torch.int32))])
    codes = dict(m=torch.zeros(300, dtype=torch.float8_e4m3fn), v=torch.zeros(300, dtype=torch.float8_e4m3fn))
    assert ftmoe.adamw_list([adam_tensors(torch, **codes)]).array[0].state_bits == 8
    assert recorder.calls == ["ftmoe_adamw"] * 2


def test_adamw_list_keeps_its_tensors():
    """Also where the caller puts others into the dicts that the list was made of."""
    torch = pytest.importorskip("torch")
    import weakref
    t = adam_tensors(torch, 8)
    alive = {n: weakref.ref(v) for n, v in t.items()}
    made = ftmoe.adamw_list([t])
    t.clear()
    assert [n for n, r in alive.items() if r() is None] == []
    del made
    assert [n for n, r in alive.items() if r() is not None] == []
