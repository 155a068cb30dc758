"""dense_linear on the GPU against its definition in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _mat(n, m, dt, g, pad=0, shift=0, ints=False, scale=1.0):
    """[n, m] with rows `pad` elements apart, `shift` elements into the memory; NaN around it."""
    buf = torch.full((n * (m + pad) + shift + 8,), float("nan"), dtype=DT[dt], device="cuda")
    v = buf[shift:shift + n * (m + pad)].view(n, m + pad)[:, :m]
    if ints:
        v.copy_(torch.randint(-2, 3, (n, m), device="cuda", generator=g).to(DT[dt]))
    else:
        v.copy_((torch.randn((n, m), device="cuda", generator=g) * scale).to(DT[dt]))
    return v


def _check(lib, M, N, K, dtype="bf16", out="bf16", act="none", gated=False, bias=None, residual=False, pad=0, shift=0,
           opad=0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = _mat(M, K, dtype, g, pad, shift)
    w = _mat(N, K, dtype, g, pad, shift, scale=1.5 / K ** 0.5)
    b = None if bias is None else torch.randn(N, device="cuda", generator=g).to(DT[bias])
    n_out = N // 2 if gated else N
    r = _mat(M, n_out, out, g, opad, shift) if residual else None
    obuf = torch.full((M, n_out + opad), 7.0, dtype=DT[out], device="cuda")
    o = obuf[:, :n_out]
    got = lib.dense_linear(x, w, bias=b, act=act, gated=gated, residual=r, out_dtype=DT[out], out=o)
    torch.cuda.synchronize()
    assert got is o and lib.device_error() == 0
    assert torch.all(obuf[:, n_out:] == 7.0)  # nothing beside the rows
    want, bound = ref.linear(_np(x), _np(w), _np(b), act, gated, _np(r))
    ref.check(_np(o), want, bound, out)


SIZES = [(1, 1, 1), (1, 256, 1024), (1, 33, 77), (3, 17, 64), (8, 128, 4096), (9, 40, 513), (16, 512, 2048),
         (17, 16, 96), (33, 200, 1000), (64, 256, 1536), (65, 130, 320), (100, 72, 64), (128, 384, 512),
         (129, 257, 130), (255, 64, 1024), (256, 512, 256), (300, 300, 300), (513, 1000, 200), (1025, 48, 2056),
         (2304, 1288, 320), (2305, 1283, 130), (4100, 700, 72), (520, 9000, 64),
         (700, 260, 640), (390, 1032, 1300), (8192, 40, 1088)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_sizes(lib, M, N, K, gated):
    N = 2 * N if gated else N
    _check(lib, M, N, K, gated=gated, act="silu" if gated else "none", bias="f32", residual=True, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(1, 64, 7168), (8, 256, 520), (40, 96, 3000), (130, 272, 1056), (700, 260, 1024),
                                   (2000, 520, 640), (2300, 1544, 640), (9000, 520, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_whole_numbers_are_exact(lib, M, N, K, dtype):
    # sums of whole numbers below 2^24 have no rounding: every product is there once, at its place
    g = torch.Generator("cuda").manual_seed(K)
    x, w = _mat(M, K, dtype, g, ints=True), _mat(N, K, dtype, g, ints=True)
    got = lib.dense_linear(x, w, out_dtype=torch.float32)
    want = x.cpu().double() @ w.cpu().double().t()
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("M,N,K", [(2, 64, 16384), (30, 128, 16384), (200, 512, 16384), (1300, 2000, 16384),
                                   (600, 512, 8000)])
def test_long_sums_stay_fp32(lib, M, N, K):
    # Sums on the tensor core are cut off at every addition of 16 products, to one side.  With at most 64 additions
    # (1024 products) to a sum before it is added up in fp32, each cut at most 2^-23 of its sum, the error stays below
    # 64 * 2^-23 of the result's norm; a single sum over K = 16384 would be off by about 1024 / 3 * 2^-23.
    g = torch.Generator("cuda").manual_seed(21)
    x, w = _mat(M, K, "bf16", g), _mat(N, K, "bf16", g)
    got = lib.dense_linear(x, w, out_dtype=torch.float32).double()
    want = x.double() @ w.double().t()
    assert (got - want).norm() <= 64 * 2.0 ** -23 * want.norm()


CONFIGS = [(256, 1), (256, 2), (256, 4), (128, 1), (128, 2), (128, 4), (64, 1), (64, 2), (64, 4), (64, 8), (32, 1),
           (32, 2), (32, 4), (32, 8)]


@pytest.fixture
def config(lib, request):
    clib = lib.load()
    assert clib.w4a8_test_linear_config(*request.param) == 0
    yield request.param
    clib.w4a8_test_linear_config(0, 0)


@pytest.mark.parametrize("config", CONFIGS, indirect=True)
@pytest.mark.parametrize("M,N,K", [(17, 130, 520), (96, 264, 1100), (300, 520, 832), (1000, 1288, 640)])
@pytest.mark.parametrize("gated", [False, True])
def test_every_configuration(lib, config, M, N, K, gated):
    g = torch.Generator("cuda").manual_seed(M)
    x, w = _mat(M, K, "bf16", g, ints=True), _mat(N, K, "bf16", g, ints=True)
    got = lib.dense_linear(x, w, out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), x.cpu().double() @ w.cpu().double().t())
    _check(lib, M, N, K, gated=gated, act="silu" if gated else "gelu", bias="f32", residual=True, seed=N)
    _check(lib, M, N, K, gated=gated, act="relu", out="f32", residual=True, opad=1, seed=N)
    # fp32 outputs of a long K: sums in pieces
    x, w = _mat(M, 4224, "bf16", g, ints=True), _mat(N, 4224, "bf16", g, ints=True)
    r = _mat(M, N // 2 if gated else N, "f32", g, ints=True)
    z = x.cpu().double() @ w.cpu().double().t()
    want = (z[:, :N // 2].clamp_min(0) * z[:, N // 2:] if gated else z.clamp_min(0)) + r.cpu().double()
    got = lib.dense_linear(x, w, act="relu", gated=gated, residual=r, out_dtype=torch.float32).cpu().double()
    assert torch.equal(got, want.float().double() if gated else want)


def test_configuration_that_does_not_exist(lib):
    x = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
    lib.load().w4a8_test_linear_config(96, 1)
    try:
        with pytest.raises(lib.W4A8Error, match="no configuration"):
            lib.dense_linear(x, x)
    finally:
        lib.load().w4a8_test_linear_config(0, 0)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N", [(3, 192), (50, 192), (300, 192), (1300, 2000)])
def test_activations(lib, act, gated, M, N):
    _check(lib, M, N, 256, act=act, gated=gated, out="f32", seed=11)


@pytest.mark.parametrize("dtype,out,bias", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f16", "f16", "f16"),
                                            ("f16", "f32", "f16"), ("f16", "f16", "f32")])
@pytest.mark.parametrize("M,N", [(1, 320), (20, 320), (70, 320), (400, 320), (1400, 2000)])
def test_types(lib, dtype, out, bias, M, N):
    _check(lib, M, N, 384, dtype=dtype, out=out, act="gelu", bias=bias, residual=True, seed=12)


@pytest.mark.parametrize("pad,shift,opad", [(8, 0, 8), (0, 1, 0), (3, 0, 1), (1, 8, 3), (8, 4, 4), (24, 16, 16)])
@pytest.mark.parametrize("M,N", [(2, 136), (24, 136), (90, 136), (600, 136), (1100, 2088)])
@pytest.mark.parametrize("K", [256, 333])
def test_strides_and_alignment(lib, pad, shift, opad, M, N, K):
    _check(lib, M, N, K, pad=pad, shift=shift, opad=opad, bias="f32", residual=True, seed=13)


@pytest.mark.parametrize("M", [1, 30, 77, 260, 1500])
def test_residual_in_place_and_repeatable(lib, M):
    g = torch.Generator("cuda").manual_seed(14)
    x, w = _mat(M, 2048, "bf16", g), _mat(128, 2048, "bf16", g)
    r = _mat(M, 128, "bf16", g)
    a = lib.dense_linear(x, w, residual=r)
    b = lib.dense_linear(x, w, residual=r)
    assert torch.equal(a, b)  # sums are added in a fixed order
    lib.dense_linear(x, w, residual=r, out=r)
    assert torch.equal(a, r)


def test_rows_do_not_mix(lib):
    # a NaN or an infinity in one token, or one weight row, stays in its row or column
    g = torch.Generator("cuda").manual_seed(15)
    for M in (4, 60, 300):
        x, w = _mat(M, 200, "bf16", g), _mat(96, 200, "bf16", g)
        x[1, 3] = float("nan")
        w[70, 199] = float("inf")
        y = lib.dense_linear(x, w)
        good = torch.ones_like(y, dtype=torch.bool)
        good[1] = False
        good[:, 70] = False
        assert torch.isfinite(y[good]).all() and torch.isnan(y[1]).all() and not torch.isfinite(y[:, 70]).any()


def test_empty(lib):
    x, w = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    assert lib.dense_linear(x, w).shape == (0, 32)
    assert lib.dense_linear(w, x).shape == (32, 0)


@pytest.mark.parametrize("M", [5, 64, 1024])
def test_other_stream_and_graph(lib, M):
    g = torch.Generator("cuda").manual_seed(16)
    x, w = _mat(M, 512, "bf16", g), _mat(256, 512, "bf16", g)
    want = lib.dense_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    with torch.cuda.stream(s):
        lib.dense_linear(x, w, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            lib.dense_linear(x, w, out=out)
        out.zero_()
        graph.replay()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)


def test_refusals(lib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError, match="x must be one of"):
        lib.dense_linear(x.float(), w.float())
    with pytest.raises(TypeError, match="w must be one of"):
        lib.dense_linear(x, w.half())
    with pytest.raises(ValueError, match="64 columns"):
        lib.dense_linear(x, w[:, :32])
    with pytest.raises(ValueError, match="even"):
        lib.dense_linear(x, w[:31], gated=True)
    with pytest.raises(ValueError, match="act"):
        lib.dense_linear(x, w, act="tanh")
    with pytest.raises(TypeError, match="out_dtype"):
        lib.dense_linear(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="residual"):
        lib.dense_linear(x, w, residual=torch.zeros((4, 31), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="bias"):
        lib.dense_linear(x, w, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(lib.W4A8Error, match="K=0"):
        lib.dense_linear(x[:, :0], w[:, :0])
    with pytest.raises(TypeError, match="CUDA tensor"):
        lib.dense_linear(x.cpu(), w)


@pytest.mark.parametrize("M,N,K", [(2501, 2056, 128), (2501, 2051, 128), (2500, 2048, 1600)])
@pytest.mark.parametrize("gated", [False, True])
def test_fp32_residual_in_place(lib, M, N, K, gated):
    if gated and N % 2:
        N += 1
    g = torch.Generator("cuda").manual_seed(21)
    x = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
    w = (torch.randn((N, K), device="cuda", generator=g) / K**0.5).to(torch.bfloat16)
    r = torch.randn((M, N // 2 if gated else N), device="cuda", generator=g)
    apart = lib.dense_linear(x, w, act="relu", gated=gated, residual=r, out_dtype=torch.float32)
    alone = lib.dense_linear(x, w, act="relu", gated=gated, out_dtype=torch.float32)
    assert torch.equal(apart, alone + r)  # one fp32 addition
    lib.dense_linear(x, w, act="relu", gated=gated, residual=r, out_dtype=torch.float32, out=r)
    assert torch.equal(apart, r)


@pytest.mark.parametrize("missing", [-1, 0, 3, 7])
def test_warps_that_share_a_step_give_up_together(lib, missing):
    # one warp's wait runs out (1 ms): every warp learns of it, the kernel ends, and the error word says so once
    gave_up = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.load().w4a8_test_linear_wait(missing, 1_000_000, ctypes.c_void_p(gave_up.data_ptr()), stream) == 0
    torch.cuda.synchronize()
    assert gave_up.tolist() == [(missing >= 0) | (2 if w == missing else 0) for w in range(8)]
    assert lib.device_error() == (1 if missing >= 0 else 0)
    assert lib.device_error() == 0
    # a product whose sums are taken in pieces, through the same routine
    g = torch.Generator("cuda").manual_seed(22)
    x, w = _mat(520, 4224, "bf16", g, ints=True), _mat(264, 4224, "bf16", g, ints=True)
    lib.load().w4a8_test_linear_config(256, 1)
    try:
        got = lib.dense_linear(x, w, out_dtype=torch.float32)
    finally:
        lib.load().w4a8_test_linear_config(0, 0)
    assert torch.equal(got.double(), x.double() @ w.double().t()) and lib.device_error() == 0


@pytest.mark.parametrize("M,N,K,dtype", [(8, 64, 1 << 20, "f16"), (64, 256, 1 << 20, "f16"), (300, 512, 1 << 20, "f16"),
                                         (64, 256, 131072, "f16"), (1300, 2000, 40000, "f16"), (300, 512, 1 << 20, "bf16")])
def test_long_sums_of_16_bit_outputs(lib, M, N, K, dtype):
    # Positive terms, where the cut-off of the tensor core's additions only adds up.  A sum in one accumulator may be off by
    # a sixteenth of the output's own rounding, the joining of up to 1024 pieces in fp32 by another.
    g = torch.Generator("cuda").manual_seed(23)
    x, w = (((0.5 + 0.5 * torch.rand((n, K), device="cuda", generator=g)) * 2.0 ** -5).to(DT[dtype]) for n in (M, N))
    got = lib.dense_linear(x, w).double()
    want = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for k in range(0, K, 65536):
        want += x[:, k:k + 65536].double() @ w[:, k:k + 65536].double().t()
    assert lib.device_error() == 0
    assert torch.all((got - want).abs() <= (1 + 1 / 8) * ref.U[dtype] * want)


@pytest.mark.parametrize("config,dtype,K", [((256, 1), "f16", 16520), ((256, 2), "f16", 33000), ((256, 4), "f16", 65800),
                                            ((256, 1), "bf16", 131200)], indirect=["config"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("opad", [0, 8, 3])
def test_sums_in_pieces_with_a_16_bit_residual(lib, config, dtype, K, gated, opad):
    # whole numbers: the sums are exact, and the residual is added before the one rounding to the output's type
    M, N = 300, 512
    g = torch.Generator("cuda").manual_seed(24)
    x, w = _mat(M, K, dtype, g, ints=True), _mat(N, K, dtype, g, ints=True)
    r = _mat(M, N // 2 if gated else N, dtype, g, pad=opad, ints=True)
    z = x.double() @ w.double().t()
    want = (z[:, :N // 2].clamp_min(0) * z[:, N // 2:] if gated else z.clamp_min(0)) + r.double()
    got = lib.dense_linear(x, w, act="relu", gated=gated, residual=r)
    assert lib.device_error() == 0 and torch.equal(got, want.float().to(DT[dtype]))
    lib.dense_linear(x, w, act="relu", gated=gated, residual=r, out=r)
    assert torch.equal(r, got)


# few rows: aligned weights from 12 MiB (9 to 16 rows) or 24 MiB (up to 8, gated) leave the streaming kernel for tiles of
# which most rows do not exist; just below and just above, and the same without alignment
@pytest.mark.parametrize("M,N,K,gated", [(1, 4096, 7168, True), (1, 1754, 7168, True), (5, 1756, 7168, True),
                                         (8, 4096, 7168, True), (8, 8192, 4096, False), (9, 1535, 4096, False),
                                         (9, 1536, 4096, False), (16, 2048, 4096, False), (16, 1024, 6152, True),
                                         (16, 2050, 4100, True)])
@pytest.mark.parametrize("dtype,out,residual", [("bf16", "bf16", True), ("bf16", "f32", False), ("f16", "f32", True)])
def test_few_rows_with_large_weights(lib, M, N, K, gated, dtype, out, residual):
    _check(lib, M, N, K, dtype=dtype, out=out, gated=gated, act="silu" if gated else "gelu", bias="f32", residual=residual,
           seed=25)


@pytest.mark.parametrize("config", CONFIGS, indirect=True)
@pytest.mark.parametrize("M", [1, 13])
def test_few_rows_in_every_configuration(lib, config, M):
    N, K = (1800, 7168) if M == 1 else (1544, 4160)
    g = torch.Generator("cuda").manual_seed(26)
    x, w = _mat(M, K, "bf16", g, ints=True), _mat(N, K, "bf16", g, ints=True)
    z = x.cpu().double() @ w.cpu().double().t()
    got = lib.dense_linear(x, w, act="relu", gated=True, out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), (z[:, :N // 2].clamp_min(0) * z[:, N // 2:]))
    assert lib.device_error() == 0
