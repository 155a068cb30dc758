"""fp8_block_linear on the GPU against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
VALUES = ref.e4m3_values()


def _inputs(M, N, K, seed=0, ints=False, pad=0):
    g = torch.Generator("cuda").manual_seed(seed)
    G = K // 128
    if ints:  # whole numbers of up to 4, scales that are powers of two: every sum is exact
        a, b = (torch.randint(-4, 5, (r, K), device="cuda", generator=g).float() for r in (M, N))
        a_s, b_s = (2.0 ** torch.randint(-2, 3, s, device="cuda", generator=g).float() for s in ((G, M), ((N + 127) // 128, G)))
    else:
        a, b = (torch.randn((r, K), device="cuda", generator=g) * 60 for r in (M, N))
        a_s, b_s = (0.001 + 0.02 * torch.rand(s, device="cuda", generator=g) for s in ((G, M), ((N + 127) // 128, G)))
    a, b = (t.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for t in (a, b))
    ld = max(4, (M + 3) // 4 * 4) + pad
    scales = torch.full((G, ld), float("nan"), device="cuda")  # what lies behind the last token is not read
    scales[:, :M] = a_s
    return a, scales, b, b_s


def _want(a, a_s, b, b_s, dtype):
    M = a.shape[0]
    return ref.block_linear(VALUES[a.cpu().numpy()], a_s[:, :M].t().double().cpu().numpy(), VALUES[b.cpu().numpy()],
                            b_s.double().cpu().numpy(), dtype)


def _check(lib, M, N, K, out="bf16", seed=0, pad=0, opad=0, shift=0):
    a, a_s, b, b_s = _inputs(M, N, K, seed, pad=pad)
    buf = torch.full((M * (N + opad) + shift,), 7.0, device="cuda").to(DT[out])
    o = buf[shift:].view(M, N + opad)[:, :N]
    assert lib.fp8_block_linear(a, a_s, b, b_s, out_dtype=DT[out], out=o) is o
    assert lib.device_error() == 0
    want, bound = _want(a, a_s, b, b_s, out)
    err = np.abs(o.double().cpu().numpy() - want)
    assert (err <= bound).all(), (err - bound).max()
    assert torch.all(buf[:shift] == 7.0) and torch.all(buf[shift:].view(M, N + opad)[:, N:] == 7.0)


SIZES = [(1, 1, 128), (1, 128, 256), (1, 1000, 1024), (3, 130, 384), (8, 512, 2048), (16, 77, 640), (17, 256, 128),
         (33, 1152, 512), (64, 384, 1536), (65, 130, 256), (100, 72, 896), (128, 512, 512), (129, 257, 384), (256, 256, 128),
         (300, 300, 256), (513, 1000, 256), (777, 1001, 512), (1025, 48, 1152), (2304, 1288, 384), (2305, 1283, 256),
         (5000, 600, 128), (390, 4100, 256)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_sizes(lib, M, N, K, out):
    _check(lib, M, N, K, out, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(1, 256, 256), (40, 300, 384), (700, 520, 256)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("pad,opad,shift", [(4, 8, 0), (0, 4, 4), (0, 3, 1), (400, 0, 2)])
def test_strides_and_starts(lib, M, N, K, out, pad, opad, shift):
    _check(lib, M, N, K, out, seed=pad, pad=pad, opad=opad, shift=shift)


CONFIGS = [(256, 1)] + [(r, p) for r in (128, 64, 32, 16) for p in (1, 2, 3, 4, 5, 8) if r < 128 or p in (1, 2, 4)]


@pytest.fixture
def config(lib, request):
    clib = lib.load()
    assert clib.w4a8_test_fp8_linear_config(*request.param) == 0
    yield request.param
    clib.w4a8_test_fp8_linear_config(0, 0)


@pytest.mark.parametrize("config", CONFIGS, indirect=True)
@pytest.mark.parametrize("M,N,K", [(1, 128, 1024), (19, 130, 1152), (96, 264, 1408), (300, 520, 1024)])
def test_every_configuration_is_exact_in_whole_numbers(lib, config, M, N, K):
    # products of up to 16 * 16, sums below 2^24: every product is there once, at its place, with its scales
    a, a_s, b, b_s = _inputs(M, N, K, seed=N, ints=True)
    got = lib.fp8_block_linear(a, a_s, b, b_s, out_dtype=torch.float32).double().cpu().numpy()
    want, _ = _want(a, a_s, b, b_s, "f32")
    assert np.array_equal(got, want)
    _check(lib, M, N, K, "bf16", seed=K)
    _check(lib, M, N, K, "f32", seed=K, opad=1)


@pytest.mark.parametrize("M,N,K", [(4, 256, 16384), (200, 256, 16384), (2048, 512, 16384)])
def test_long_sums_stay_fp32(lib, M, N, K):
    # groups are summed in fp32, rounded to nearest: 128 roundings of running sums, far below one long sum of 512 cut-off
    # additions on the tensor core; a group's own four additions are cut off by at most 2^-23 of it each
    a, a_s, b, b_s = _inputs(M, N, K, seed=5)
    got = lib.fp8_block_linear(a, a_s, b, b_s, out_dtype=torch.float32)
    x = torch.from_numpy(VALUES).cuda()[a.long()] * a_s[:, :M].t().double().repeat_interleave(128, 1)
    w = torch.from_numpy(VALUES).cuda()[b.long()] * b_s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    want = x @ w.t()
    assert (got.double() - want).norm() <= 32 * 2.0 ** -24 * want.norm()


def test_quantised_rows_through_the_quantisation_call(lib):
    # as a projection is computed: rows quantised per token and 128 columns, weights with a scale per 128 x 128
    M, N, K = 70, 384, 512
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
    q, s, _ = lib.fp8_quant_per_token_group(x)
    _, _, b, b_s = _inputs(M, N, K, seed=4)
    got = lib.fp8_block_linear(q, s, b.view(torch.float8_e4m3fn), b_s)
    want, bound = _want(q, s, b, b_s, "bf16")
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


def test_nan_codes_stay_in_their_row_and_column(lib):
    for M in (5, 300):
        a, a_s, b, b_s = _inputs(M, 260, 256)
        a[2, 9] = 0x7F
        b[131, 200] = 0xFF
        got = lib.fp8_block_linear(a, a_s, b, b_s).float()
        nan = torch.isnan(got)
        want = torch.zeros_like(nan)
        want[2], want[:, 131] = True, True
        assert torch.equal(nan, want)


def test_same_bits_again_on_another_stream_and_in_a_graph(lib):
    for M in (8, 64, 700):
        a, a_s, b, b_s = _inputs(M, 520, 2048, seed=M)
        want = lib.fp8_block_linear(a, a_s, b, b_s)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = [lib.fp8_block_linear(a, a_s, b, b_s) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(g, want) for g in got)
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.fp8_block_linear(a, a_s, b, b_s, out=out)
        b.copy_(b.flip(0))
        graph.replay()
        assert torch.equal(out, lib.fp8_block_linear(a, a_s, b, b_s))


def test_empty(lib):
    a, a_s, b, b_s = _inputs(4, 8, 128)
    assert lib.fp8_block_linear(a[:0], a_s, b, b_s).shape == (0, 8)
    assert lib.fp8_block_linear(a, a_s, b[:0], b_s[:0]).shape == (4, 0)


def test_refusals(lib):
    a, a_s, b, b_s = _inputs(4, 260, 256)
    for args, err, msg in [
            ((a.int(), a_s, b, b_s), TypeError, "A must be"), ((a, a_s, b[:, :128].contiguous(), b_s), ValueError, "B must have"),
            ((a[:, :192].contiguous(), a_s[:1], b[:, :192].contiguous(), b_s[:, :1].contiguous()), lib.W4A8Error, "K=192"),
            ((a, a_s[:1], b, b_s), ValueError, "a_scales"), ((a, a_s[:, :3], b, b_s), ValueError, "a_scales"),
            ((a, a_s.half(), b, b_s), TypeError, "a_scales"), ((a, a_s, b, b_s[:2]), ValueError, "b_scales"),
            ((a, a_s, b, b_s.t().contiguous().t()), ValueError, "contiguous"), ((a[:, ::2], a_s, b, b_s), ValueError, "contiguous"),
            ((a.cpu(), a_s, b, b_s), TypeError, "CUDA"),
            ((a.flatten()[1:513].view(2, 256), a_s, b, b_s), lib.W4A8Error, "16-byte")]:
        with pytest.raises(err, match=msg):
            lib.fp8_block_linear(*args)
    for kw, err, msg in [(dict(out_dtype=torch.float64), TypeError, "out_dtype"),
                         (dict(out=torch.empty((4, 260), device="cuda")), TypeError, "out"),
                         (dict(out=torch.empty((4, 259), device="cuda", dtype=torch.bfloat16)), ValueError, "out")]:
        with pytest.raises(err, match=msg):
            lib.fp8_block_linear(a, a_s, b, b_s, **kw)
    assert lib.device_error() == 0


@pytest.fixture
def without(lib, request):
    clib = lib.load()
    assert clib.w4a8_test_fp8_linear_without(request.param) == 0
    yield request.param
    clib.w4a8_test_fp8_linear_without(0)


@pytest.mark.parametrize("without", [256, 128, 64, 32, 16], indirect=True)
@pytest.mark.parametrize("M,N,K", [(1, 256, 128), (90, 300, 512), (700, 2600, 256)])
def test_a_configuration_that_is_not_there_leaves_the_others(lib, without, M, N, K):
    # as where a kernel was built with other registers than it needs: the rest serves the call, an error only without any
    _check(lib, M, N, K, "bf16", seed=N)
    clib = lib.load()
    assert clib.w4a8_test_fp8_linear_config(without, 1) == 0
    try:
        with pytest.raises(lib.W4A8Error, match=f"{without} rows"):
            _check(lib, M, N, K)
    finally:
        clib.w4a8_test_fp8_linear_config(0, 0)
