"""rotary_embedding on the GPU against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _np(t):
    return t.double().cpu().numpy()


def _check(got, want, slack, dtype):
    err = np.abs(_np(got) - want)
    bound = ref.rounded(want, dtype, slack)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("T,H,D,R,start", [
    (1, 1, 2, 2, 0), (1, 72, 128, 128, 0), (3, 5, 64, 32, 32), (64, 9, 192, 64, 128), (17, 3, 80, 40, 0),
    (33, 2, 65, 20, 7), (300, 17, 96, 48, 48), (5, 1, 1024, 1024, 0), (2, 3, 1023, 1000, 11), (2000, 1, 8, 2, 6),
    (1111, 2, 256, 256, 0), (7, 300, 24, 12, 8), (130, 40, 128, 64, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(lib, T, H, D, R, start, dtype, interleaved):
    g = torch.Generator("cuda").manual_seed(T + H + D)
    x = torch.randn((T, H, D), device="cuda", generator=g).to(DT[dtype])
    pos = torch.randint(0, 200000, (T,), device="cuda", generator=g)
    f = ref.inv_freq(R)
    freqs = lib.rotary_frequencies(R)
    got = lib.rotary_embedding(x, pos, freqs, interleaved=interleaved, start=start, scale=1.25)
    want, slack = ref.rotate(_np(x), _np(pos), f, interleaved, start, 1.25)
    _check(got, want, slack, dtype)
    assert torch.equal(got[:, :, :start], x[:, :, :start]) and torch.equal(got[:, :, start + R:], x[:, :, start + R:])
    again = x.clone()
    assert lib.rotary_embedding(again, pos.int(), freqs, interleaved=interleaved, start=start, scale=1.25, out=again) is again
    assert torch.equal(again, got)


@pytest.mark.parametrize("T,H,D,R,start", [
    (3, 2, 1024, 1022, 1), (9, 3, 1022, 1020, 2), (9, 3, 1020, 508, 4), (41, 5, 90, 44, 46),
    (41, 5, 90, 44, 0), (7, 1, 6, 2, 2), (200, 3, 101, 50, 51)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_narrow_vectors(lib, T, H, D, R, start, dtype, interleaved):
    # rows that fall into vectors of 2, 4 or 8 bytes, several of them to a thread, the last thread's not all there
    test_sizes(lib, T, H, D, R, start, dtype, interleaved)


@pytest.mark.parametrize("pos", [0, 1, -1, 4095, 163839, 1 << 20, (1 << 31) - 1, -(1 << 31)])
def test_far_positions_keep_their_angle(lib, pos):
    # a float32 product of position and frequency would be off by up to 64 radians here
    R, D = 128, 128
    x = torch.randn((2, 3, D), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    p = torch.full((2,), pos, dtype=torch.int32, device="cuda")
    got = lib.rotary_embedding(x, p, lib.rotary_frequencies(R))
    # the reference's angle is rounded to 64 bits: 2^31 * 2^-53 radians, 2^-22
    want, slack = ref.rotate(_np(x), np.full(2, pos), ref.inv_freq(R))
    err = np.abs(_np(got) - want)
    assert (err <= ref.rounded(want, "f32", slack) + 4 * abs(pos) * 2.0 ** -53).all()


def test_far_positions_of_64_bits(lib):
    # one whole turn every 2^20 positions: p and p modulo 2^20 have the same angle
    freqs = torch.tensor([1 << 44], dtype=torch.int64, device="cuda")
    x = torch.randn((4, 1, 2), device="cuda")
    p = torch.tensor([5, 700001, -3, 123456], device="cuda")
    far = p + (torch.tensor([1 << 40, -(1 << 42), 1 << 33, 3 << 41], device="cuda"))
    assert torch.equal(lib.rotary_embedding(x, p, freqs), lib.rotary_embedding(x, far, freqs))


@pytest.mark.parametrize("pad,shift,dtype", [(0, 0, "bf16"), (8, 0, "bf16"), (4, 4, "f16"), (3, 1, "bf16"), (2, 2, "f32")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_starts(lib, pad, shift, dtype, interleaved):
    # queries and keys as columns of one projection's rows, heads apart, outputs likewise; nothing beside them is touched
    T, H, D, R = 37, 6, 64, 32
    g = torch.Generator("cuda").manual_seed(pad)
    step = H * (D + pad) + pad

    def view(buf):
        return buf[shift:].as_strided((T, H, D), (step, D + pad, 1), buf.storage_offset() + shift)
    src = torch.randn(T * step + 16, device="cuda", generator=g).to(DT[dtype])
    dst = torch.full((T * step + 16,), 7.0, device="cuda").to(DT[dtype])
    pos = torch.arange(T, device="cuda") * 1000
    out = view(dst)
    lib.rotary_embedding(view(src), pos, lib.rotary_frequencies(R), interleaved=interleaved, start=16, out=out)
    want, slack = ref.rotate(_np(view(src)), _np(pos), ref.inv_freq(R), interleaved, 16)
    _check(out, want, slack, dtype)
    mark = torch.zeros_like(dst)
    view(mark).fill_(1)
    assert torch.all(dst[mark == 0] == 7.0)
    one = src[:T * D].view(T, 1, D).expand(T, 1, D)
    got = lib.rotary_embedding(src[:D].view(1, 1, D).expand(T, 4, D), pos, lib.rotary_frequencies(R), interleaved=interleaved)
    want, slack = ref.rotate(_np(src[:D].view(1, 1, D).expand(T, 4, D)), _np(pos), ref.inv_freq(R), interleaved)
    _check(got, want, slack, dtype)
    assert one.shape == (T, 1, D)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(lib, interleaved):
    # the inverse is the gradient: against autograd of the formula in 64 bits, and against differences
    T, H, D, R, start = 9, 3, 48, 32, 8
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn((T, H, D), device="cuda", generator=g)
    dy = torch.randn((T, H, D), device="cuda", generator=g)
    pos = torch.randint(0, 100000, (T,), device="cuda", generator=g)
    freqs = lib.rotary_frequencies(R)
    dx = lib.rotary_embedding(dy, pos, freqs, interleaved=interleaved, start=start, scale=1.5, inverse=True)
    leaf = x.double().cpu().requires_grad_()
    t = pos.cpu().double()[:, None, None] * torch.from_numpy(ref.inv_freq(R))
    part = leaf[:, :, start:start + R]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :R // 2], part[..., R // 2:])
    p, q = 1.5 * (a * t.cos() - b * t.sin()), 1.5 * (b * t.cos() + a * t.sin())
    y = torch.stack([p, q], -1).flatten(2) if interleaved else torch.cat([p, q], -1)
    y = torch.cat([leaf[:, :, :start], y, leaf[:, :, start + R:]], 2)
    (want,) = torch.autograd.grad((y * dy.cpu().double()).sum(), leaf)
    _, slack = ref.rotate(_np(dy), _np(pos), ref.inv_freq(R), interleaved, start, 1.5, True)
    _check(dx, want.numpy(), slack, "f32")
    # differences: the operator is linear, so any step does; sums of T H D products in 64 bits
    d = torch.randn((T, H, D), device="cuda", generator=g)
    up, down = (lib.rotary_embedding(x + s * d, pos, freqs, interleaved=interleaved, start=start, scale=1.5).double()
                for s in (1.0, -1.0))
    diff = ((up - down) / 2 * dy.double()).sum().item()
    dot = (dx.double() * d.double()).sum().item()
    size = (dy.double().abs() * (up.abs() + down.abs())).sum().item() + (dx.double().abs() * d.double().abs()).sum().item()
    assert abs(diff - dot) <= 32 * ref.U * 4 * size


def test_empty_and_one(lib):
    freqs = lib.rotary_frequencies(4)
    assert lib.rotary_embedding(torch.zeros((0, 3, 4), device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                                freqs).shape == (0, 3, 4)
    assert lib.rotary_embedding(torch.zeros((3, 0, 4), device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                                freqs).shape == (3, 0, 4)


def test_graph_and_stream(lib):
    x = torch.randn((50, 4, 64), device="cuda")
    pos = torch.arange(50, device="cuda")
    freqs = lib.rotary_frequencies(64)
    want = lib.rotary_embedding(x, pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lib.rotary_embedding(x, pos, freqs)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.rotary_embedding(x, pos, freqs, out=out)
    pos += 77
    graph.replay()
    assert torch.equal(out, lib.rotary_embedding(x, pos, freqs))


def test_refusals(lib):
    x = torch.zeros((4, 2, 8), device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = lib.rotary_frequencies(8)
    for args, err, msg in [
            ((x[0], pos, f), ValueError, "x must have 3"), ((x.double(), pos, f), TypeError, "x must be"),
            ((x.transpose(1, 2), pos, f), ValueError, "contiguous heads"), ((x, pos[:3], f), ValueError, "positions"),
            ((x, pos.float(), f), TypeError, "positions"), ((x, pos, f.int()), TypeError, "freqs"),
            ((x, pos, None), TypeError, "freqs"), ((x, None, f), TypeError, "positions"), ((x, pos, f.cpu()), TypeError, "freqs"),
            ((x, pos, lib.rotary_frequencies(10)), lib.W4A8Error, "R=10"), ((x.cpu(), pos, f), TypeError, "CUDA"),
            ((x, pos, f[:0]), ValueError, "empty")]:
        with pytest.raises(err, match=msg):
            lib.rotary_embedding(*args)
    for kw, err, msg in [(dict(start=1), lib.W4A8Error, "start=1"), (dict(start=-1), lib.W4A8Error, "start=-1"),
                         (dict(scale=float("inf")), lib.W4A8Error, "finite"), (dict(out=x.half()), TypeError, "out"),
                         (dict(out=x[:3]), ValueError, "shape"),
                         (dict(out=x[:1].expand(4, 2, 8)), ValueError, "overlapping")]:
        with pytest.raises(err, match=msg):
            lib.rotary_embedding(x, pos, f, **kw)
    with pytest.raises(lib.W4A8Error, match="D=1025"):
        lib.rotary_embedding(torch.zeros((1, 1, 1025), device="cuda"), pos[:1], f)
    assert lib.device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_one_head_from_shared_rows(lib, interleaved, shift):
    # views whose strides say little: one head expanded from a row each, tokens that overlap, a token shared by all
    T, D = 37, 64
    src = torch.randn(T * D + 16, device="cuda", generator=torch.Generator("cuda").manual_seed(shift)).to(torch.bfloat16)
    pos = torch.arange(T, device="cuda") * 1000
    freqs = lib.rotary_frequencies(D)
    for x in (src[shift:shift + T * D].view(T, 1, D).expand(T, 1, D), src[shift:].as_strided((T, 1, D), (8, 0, 1), shift),
              src[shift:shift + D].view(1, 1, D).expand(T, 1, D)):
        got = lib.rotary_embedding(x, pos, freqs, interleaved=interleaved)
        want, slack = ref.rotate(_np(x), _np(pos), ref.inv_freq(D), interleaved)
        _check(got, want, slack, "bf16")
