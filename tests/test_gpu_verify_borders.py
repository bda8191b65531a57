"""The verification of drafted tokens where a decision is near: large noise, draws at the border of an acceptance,
residuals that nearly vanish, vocabularies at the borders of the kernels' chunks. Expected tokens follow from the
definition in 64 bits or from arithmetic stated beside the case."""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _f32(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("e", [2.0 ** 126, 1e38, 3.4e38])
def test_noise_of_the_largest_size(e):
    # token 11: score about 1 / e >= 2.9e-39; token 500: e^-70 / 1e10 < 4e-41; the others have no weight
    V = 600
    for winner, other in ((11, 500), (500, 11)):
        l = torch.full((1, V), -torch.inf, dtype=torch.bfloat16, device="cuda")
        noise = torch.ones(1, V, device="cuda")
        l[0, winner], noise[0, winner] = 0, e
        l[0, other], noise[0, other] = -70, 1e10
        t, a = moe.moe_verify_drafts(l, _i32(0), _i32(0, 1), _f32(0.5), noise)
        assert t.tolist() == [winner] and a.tolist() == [0]


def test_noise_that_is_infinite_loses_to_any_weight():
    V = 600
    l = torch.full((1, V), -torch.inf, dtype=torch.bfloat16, device="cuda")
    noise = torch.full((1, V), 3e38, device="cuda")
    l[0, 11], noise[0, 11] = 0, torch.inf
    l[0, 500] = -70
    t, _ = moe.moe_verify_drafts(l, _i32(0), _i32(0, 1), _f32(0.5), noise)
    assert t.tolist() == [500]   # e^-70 / 3e38 > 0 = 1 / inf
