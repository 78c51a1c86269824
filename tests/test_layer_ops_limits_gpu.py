"""The layer operators at the ends of their arguments' ranges."""
import pytest
import torch

from delta_rule_linear_kla_b200 import api

pytestmark = pytest.mark.gpu


def _room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip("needs %d GB of device memory" % gigabytes)


def test_ssm_step_groups_past_32_bits():
    """A token whose rows of B and C have more than 2^31 elements (a group for
    every channel): the last channels come out as in a call of their own."""
    _room(48)
    D, N, tail = (1 << 28) + 64, 8, 4096
    gen = torch.Generator(device="cuda").manual_seed(70)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    u, dt, Bm, Cm = mk(1, D), mk(1, D), mk(1, D, N), mk(1, D, N)
    assert Bm.numel() > 1 << 31
    A = torch.rand(D, N, generator=gen, device="cuda").neg_()
    S = torch.rand(1, D, N, generator=gen, device="cuda")
    cut = [t[:, -tail:].clone() for t in (u, dt, Bm, Cm, S)]
    y = api.ssm_step(u, dt, A, Bm, Cm, S)
    want = api.ssm_step(cut[0], cut[1], A[-tail:].contiguous(), cut[2], cut[3], cut[4])
    assert torch.equal(y[:, -tail:], want) and torch.equal(S[:, -tail:], cut[4])
