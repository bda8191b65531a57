"""What the binding makes itself for the attention block's calls: outputs and workspaces, on the call's stream."""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe
from test_gpu_kv4 import _filled, _gen, _randn, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("nq", [1, 40])
def test_what_a_call_makes_belongs_to_its_stream(nq, handle):
    """The call's stream is behind a long wait when the call returns, and the caller goes on: tensors that it makes then, of
    every size that the call let go of, are not written by the call's kernels, nor its results by theirs."""
    g = _gen(nq)
    Hkv, G, D, S, n = 2, 4, 128, 16, 3000
    cache = _filled(g, 200, Hkv, S, D)
    table = _tables(g, [n], S, 200)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q, x = _randn(g, nq, Hkv * G, D).bfloat16(), _randn(g, nq, Hkv, D).bfloat16()
    lens, cu, slots = i32(n), i32(0, nq), torch.arange(nq, dtype=torch.int32, device="cuda")
    pos, freq = torch.arange(nq, dtype=torch.int32, device="cuda"), torch.ones(64, device="cuda")

    def all_calls(stream):
        return (*moe.moe_qk_norm_rope(q, x, pos, freq, stream=stream), *moe.moe_kv4_read(slots, cache, stream=stream),
                *moe.moe_kv4_attention(q, cache, table, lens, cu_q=cu, max_q=nq, lse=True, stream=stream))

    want = [t.clone() for t in all_calls(None)]
    sizes = [moe.moe_kv4_workspace_size(nq, Hkv * G, Hkv, D), 256] + [t.numel() * t.element_size() for t in want]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                    # about 0.1 s
    got = all_calls(side.cuda_stream if handle else side)
    mine = [torch.full((b,), 7, dtype=torch.uint8, device="cuda") for b in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in mine)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_batch_of_no_tokens():
    cache = moe.kv4_cache(4, 2, 16, 128)
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    for ws in (None, moe.kv4_workspace(0, 8, 2, 128)):
        out, lse = moe.moe_kv4_attention(q, cache, i32(3, 4), i32(3), cu_q=i32(4), lse=True, ws=ws)
        assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
        assert moe.moe_kv4_attention(q, cache, i32(0, 4), i32(0), ws=ws).shape == (0, 8, 128)
        moe.moe_kv4_append(q[:, :2], q[:, :2], i32(0), cache, ws=ws)
        assert moe.moe_kv4_read(i32(0), cache, ws=ws)[0].shape == (0, 2, 128)


@pytest.mark.parametrize("nq", [1, 6, 140])
def test_a_workspace_of_the_calls_own(nq):
    """Only its control block is cleared: whatever lies in the rest, the results are those of a zeroed one."""
    g = _gen(nq)
    Hkv, G, D, S, n = 2, 4, 128, 16, 3000
    cache = _filled(g, 200, Hkv, S, D)
    table = _tables(g, [n], S, 200)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = _randn(g, nq, Hkv * G, D).bfloat16()
    args = (q, cache, table, i32(n), i32(0, nq), nq)
    want, lse = moe.moe_kv4_attention(*args, lse=True, ws=moe.kv4_workspace(nq, Hkv * G, Hkv, D))
    size = moe.moe_kv4_workspace_size(nq, Hkv * G, Hkv, D)
    for fill in (0xFF, 0x7F, 1):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        at = ws.data_ptr()
        del ws                                            # the call gets this memory
        got, z = moe.moe_kv4_attention(*args, lse=True)
        again = torch.empty(size, dtype=torch.uint8, device="cuda")
        assert again.data_ptr() == at and bool((again[256:512] == fill).all())
        assert torch.equal(got, want) and torch.equal(z, lse)


def test_more_work_than_a_call_counts():
    """2^31 units of work: refused on the device, and nothing is written."""
    Hkv, D, S, nq, pages = 128, 64, 1024, 1 << 15, 1024
    cache = moe.kv4_cache(1, Hkv, S, D)
    q = torch.zeros(nq, Hkv, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 3.0)
    ws = moe.kv4_workspace(nq, Hkv, Hkv, D)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    # 4096 groups of 8 rows x 8192 units x 128 heads
    moe.moe_kv4_attention(q, cache, table, i32(pages * S), cu_q=i32(0, nq), max_q=1, out=out, ws=ws)
    assert moe.moe_check_device_error(ws) == 5 and bool((out == 3).all())
    # and the workspace is as good as new
    assert bool((moe.moe_kv4_attention(q[:4], cache, table, i32(4), cu_q=i32(0, 4), max_q=4, ws=ws) == 0).all())
    assert moe.moe_check_device_error(ws) == 0
