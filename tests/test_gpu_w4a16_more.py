"""The W4A16 linear layer on the GPU: its workspace, and the ends of the range of its sums."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


class _Ops(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append(func.name())
        return func(*args, **(kwargs or {}))


def test_a_call_without_a_workspace_clears_none():
    x = torch.randn(3, 256, device="cuda").bfloat16()
    w = torch.randint(-2 ** 31, 2 ** 31 - 1, (40, 32), dtype=torch.int32, device="cuda")
    s = torch.rand(40, 2, device="cuda").bfloat16()
    want = moe.moe_w4a16_linear(x, w, s, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with _Ops() as ops:
        y = moe.moe_w4a16_linear(x, w, s)
    assert torch.equal(y, want)
    assert all(n.startswith("aten::empty") for n in ops.seen), ops.seen


def test_a_workspace_is_left_as_it_is():
    x = torch.randn(9, 128, device="cuda").bfloat16()
    w = torch.zeros(17, 16, dtype=torch.int32, device="cuda")
    ws = torch.full((512,), 7, dtype=torch.uint8, device="cuda")
    moe.moe_w4a16_linear(x, w, torch.ones(17, 1, device="cuda").bfloat16(), ws=ws)
    assert (ws == 7).all()


@pytest.mark.parametrize("T", [1, 9])
def test_the_largest_values_whose_sums_are_in_range(T):
    # |x| <= 2^117: a group's sum is 128 x 8 x 2^117 = 2^127 at most; scales bring it back
    K, N = 256, 24
    x = torch.full((T, K), 2.0 ** 117, device="cuda").bfloat16()
    w = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")    # every code -8
    s = torch.full((N, K // 128), 2.0 ** -120, device="cuda").bfloat16()
    assert (moe.moe_w4a16_linear(x, w, s) == -2.0 ** 8).all()
    x[:, 128:] = -x[:, 128:]
    assert (moe.moe_w4a16_linear(x, w, s) == 0).all()
    # and from the other end: values of 2^-110, scales of 2^100
    y = moe.moe_w4a16_linear(torch.full((T, K), 2.0 ** -110, device="cuda").bfloat16(), w, torch.full((N, 2), 2.0 ** 100, device="cuda").bfloat16())
    assert (y == -2.0).all()
