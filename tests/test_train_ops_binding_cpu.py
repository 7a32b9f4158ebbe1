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
