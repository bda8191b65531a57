"""The W4A16 linear layer on the GPU, against y = x W^T in 64 bits.

Tolerances. With A = sum_c |x_c W_c| (the mass an output is made of): codes and scales enter exactly; a path through
the sums passes at most the 128 products of a group, its G = K / 128 groups and 64 partial results, each off by at most
2 u(fp32) of A (a tensor core may cut off instead of rounding: a whole step an addition), and y is rounded to bf16
once: u(bf16) of itself. u(t) = finfo(t).eps / 2.
"""
import pytest
import torch

import w4a16_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu

UB, U32 = (torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.lib()


def _inputs(T, N, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, K, generator=g, device="cuda")
    x = (x * (1 + 30 * (torch.rand(K, generator=g, device="cuda") < 0.01))).bfloat16()
    w = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s = (torch.randn(N, K // 128, generator=g, device="cuda") * 0.02).bfloat16()
    return x, w, s


def _weights(w, s):
    b = w.view(torch.uint8)
    q = torch.stack((b & 15, b >> 4), -1).flatten(1).double() - 8
    return q * s.double().repeat_interleave(128, 1)


def _near(y, x, w, s, rows=slice(None)):
    W = _weights(w[rows], s[rows])
    want, mass = x.double() @ W.T, x.double().abs() @ W.abs().T
    K = x.shape[1]
    tol = UB * want.abs() + (128 + K // 128 + 64) * 2 * U32 * mass
    off = (y[:, rows].double() - want).abs()
    assert (off <= tol).all(), (float((off - tol).max()), float(off.max()))


SIZES = [
    (1, 1, 128), (1, 16, 128), (2, 17, 256), (3, 100, 640), (8, 15, 1280), (5, 257, 2560), (1, 5120, 2560), (8, 5120, 2560),
    (7, 2560, 10240), (4, 2561, 4224), (1, 320, 10240), (8, 64, 16384), (1, 33, 65536), (6, 8200, 128), (2, 20000, 384), (8, 40, 65536),
    (9, 1, 128), (9, 16, 256), (16, 129, 384), (17, 127, 128), (33, 100, 16384), (64, 5120, 2560), (100, 10200, 2560), (127, 128, 640),
    (128, 128, 128), (129, 131, 2560), (300, 2048, 1280), (257, 320, 10240), (1000, 77, 4096), (2049, 5121, 512), (40, 40, 65536),
    (513, 20001, 128),
]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear(T, N, K):
    x, w, s = _inputs(T, N, K, T + N + K)
    ws = torch.zeros(moe.moe_w4a16_workspace_size(T, N, K), dtype=torch.uint8, device="cuda")
    y = moe.moe_w4a16_linear(x, w, s, ws=ws)
    assert moe.moe_check_device_error(ws) == 0
    _near(y, x, w, s)
    assert torch.equal(y, moe.moe_w4a16_linear(x, w, s))   # without a workspace, and the same bits again


@pytest.mark.parametrize("T", range(1, 9))
def test_small_batches_of_a_head(T):
    N, K = 248320, 2560
    x, w, s = _inputs(T, N, K, T)
    y = moe.moe_w4a16_linear(x, w, s)
    for lo in (0, 100000, N - 5000):
        _near(y, x, w, s, slice(lo, lo + 5000))


@pytest.mark.parametrize("T", [1, 8, 9, 40, 200])
def test_exact_products(T):
    # every partial sum is a whole number below 2^24: the result is exact before its one rounding
    N, K = 200, 1024
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randint(-3, 4, (T, K), generator=g, device="cuda").bfloat16()
    _, w, _ = _inputs(T, N, K, 5)
    s = (2.0 ** torch.randint(-3, 4, (N, K // 128), generator=g, device="cuda")).bfloat16()
    want = (x.double() @ _weights(w, s).T).float().bfloat16()
    assert torch.equal(moe.moe_w4a16_linear(x, w, s), want)


@pytest.mark.parametrize("T", [1, 20])
def test_every_code_at_every_place(T):
    # row r of W has code r % 16 everywhere but one place, which has code (r + 7) % 16
    N, K = 16 * 128, 128
    codes = torch.arange(N, device="cuda").remainder(16).unsqueeze(1).repeat(1, K)
    place = torch.arange(N, device="cuda") // 16
    codes[torch.arange(N), place] = (torch.arange(N, device="cuda") + 7).remainder(16)
    w = moe.moe_pack_int4((codes - 8).to(torch.int8))
    s = torch.ones(N, 1, dtype=torch.bfloat16, device="cuda")
    x = torch.arange(1, K + 1, device="cuda").float().bfloat16().repeat(T, 1)
    want = (x.double() @ (codes - 8).double().T).float().bfloat16()
    assert torch.equal(moe.moe_w4a16_linear(x, w, s), want)


@pytest.mark.parametrize("T", [3, 30])
def test_against_the_quantiser(T):
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(300, 512, generator=g, device="cuda").bfloat16()
    packed, scales = moe.moe_quantize_int4(W)
    x = torch.randn(T, 512, generator=g, device="cuda").bfloat16()
    y = moe.moe_w4a16_linear(x, packed, scales)
    _near(y, x, packed, scales)
    full = x.double() @ W.double().T   # 4 bits: a step of about amax / 7 a weight
    assert float((y.double() - full).norm() / full.norm()) < 0.15


@pytest.mark.parametrize("T", [2, 11, 150])
def test_values_that_are_not_finite_stay_in_their_rows(T):
    N, K = 100, 512
    x, w, s = _inputs(T, N, K, 3)
    x[1, 130] = float("nan")
    s[37, 2] = float("inf")
    s[38, 0] = float("nan")
    y = moe.moe_w4a16_linear(x, w, s)
    assert y[1].isnan().all()
    keep = torch.arange(T, device="cuda") != 1
    assert not y[keep][:, 37].isfinite().any() and y[keep][:, 38].isnan().all()
    fine = [i for i in range(N) if i not in (37, 38)]
    _near(y[keep][:, fine], x[keep], w[fine], s[fine])


def test_large_and_small_magnitudes():
    N, K = 64, 256
    x, w, s = _inputs(12, N, K, 9)
    for T in (4, 12):
        for f in (2.0 ** 100, 2.0 ** -100):
            a, b = (x[:T].float() * f).bfloat16(), (s.float() / f).bfloat16()
            _near(moe.moe_w4a16_linear(a, w, b), a, w, b)


def test_empty():
    x, w, s = _inputs(4, 16, 128)
    assert moe.moe_w4a16_linear(x[:0], w, s).shape == (0, 16)
    assert moe.moe_w4a16_linear(x, w[:0], s[:0]).shape == (4, 0)


def test_refuses_other_layouts():
    x, w, s = _inputs(4, 16, 256)
    for bad in (dict(x=x.float()), dict(x=x[:, :200]), dict(x=x.t()), dict(w=w[:, :31]), dict(w=w.long()), dict(s=s[:, :1]), dict(s=s[:15]),
                dict(y=torch.empty(4, 17, dtype=torch.bfloat16, device="cuda")), dict(y=torch.empty(4, 16, device="cuda")),
                dict(x=x[:, :192].contiguous())):
        a = dict(x=x, w=w, s=s, y=None)
        a.update(bad)
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_w4a16_linear(a["x"], a["w"], a["s"], y=a["y"])
    with pytest.raises(moe.MoeError) as e:
        moe.moe_w4a16_linear(x, w, s, ws=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(moe.MoeError) as e:   # a view that does not begin on 16 bytes
        moe.moe_w4a16_linear(torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device="cuda")[1:1025].view(4, 256), w, s)
    assert e.value.status == 1


@pytest.mark.parametrize("T", [1, 8, 50, 260])
def test_other_streams_graphs_and_a_shared_workspace(T):
    N, K = 2000, 1280
    x, w, s = _inputs(T, N, K, T)
    n = max(moe.moe_w4a16_workspace_size(T, N, K), moe.moe_workspace_size(4, 256, 16, 2, 128), moe.moe_kv4_workspace_size(T, 8, 2, 64))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    want = moe.moe_w4a16_linear(x, w, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = moe.moe_w4a16_linear(x, w, s, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    with torch.cuda.graph(graph):
        moe.moe_w4a16_linear(x, w, s, y=out, ws=ws)
        moe.moe_w4a16_linear(x, w, s, y=out, ws=ws)
    for seed in (50, 51):
        x.copy_(_inputs(T, N, K, seed)[0])
        graph.replay()
        assert torch.equal(out, moe.moe_w4a16_linear(x, w, s))
    # what the experts' calls need zero is zero still
    assert not ws[: 512 + 1024 * 128].any()
    assert moe.moe_check_device_error(ws) == 0


def test_nothing_behind_the_rows_is_written():
    for T, N, K in [(3, 37, 256), (20, 37, 256), (130, 131, 512)]:
        x, w, s = _inputs(T, N, K, 1)
        y = torch.full((T + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_w4a16_linear(x, w, s, y=y[:T])
        assert (y[T:] == 7).all()
        _near(y[:T], x, w, s)


@pytest.mark.parametrize("T", [2, 12])
def test_weights_past_32_bit_offsets(T):
    N, K = 1100000, 16384   # 9 GB of words
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.empty(N, K // 8, dtype=torch.int32, device="cuda")
    w.random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    s = (torch.rand(N, K // 128, generator=g, device="cuda") * 0.02).bfloat16()
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    y = moe.moe_w4a16_linear(x, w, s)
    for lo in (0, 524280, 1048570, N - 1000):
        _near(y, x, w, s, slice(lo, lo + 1000))


def test_outputs_past_32_bit_offsets():
    T, N, K = 20000, 120001, 128
    x, w, s = _inputs(T, N, K, 4)
    y = moe.moe_w4a16_linear(x, w, s)
    for t in (0, 9000, 17890, 19990):
        _near(y[t: t + 10], x[t: t + 10], w, s)
