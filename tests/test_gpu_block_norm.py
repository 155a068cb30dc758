"""The fused block norm on the GPU against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(lib, T, H, dtype="bf16", rdtype="bf16", post="rms", pre="rms", gate=None, pdtype="f32", bias=False,
           residual=True, branch=0.75, resid=1.25, eps=1e-6, pad=0, shift=0, seed=0, alias=False):
    g = torch.Generator("cuda").manual_seed(seed)

    def mat(n, m, dt, s=1.0):  # rows `pad` elements apart, starting `shift` elements into the memory
        buf = torch.full((n * (m + pad) + shift + 8,), float("nan"), dtype=DT[dt], device="cuda")
        v = buf[shift:shift + n * (m + pad)].view(n, m + pad)[:, :m]
        v.copy_((torch.randn((n, m), device="cuda", generator=g) * s + 0.3).to(DT[dt]))
        return v

    f, r = mat(T, H, dtype), mat(T, H, rdtype, 2.0) if residual else None
    par = {}
    for name, kind in (("post", post), ("pre", pre)):
        par["w_" + name] = (1 + 0.3 * torch.randn(H, device="cuda", generator=g)).to(DT[pdtype]) if kind != "none" else None
        par["b_" + name] = (0.2 * torch.randn(H, device="cuda", generator=g)).to(DT[pdtype]) if bias and kind != "none" else None
    gt = None if gate is None else mat(gate[0], gate[1], dtype)
    fn, rn = _np(f), _np(r)
    outs = dict(h=r, y=f) if alias else {}
    h, y = lib.block_norm(f, r, post=post, pre=pre, gate=gt, branch_scale=branch, residual_scale=resid, eps=eps,
                          residual_dtype=DT[rdtype], **par, **outs)
    torch.cuda.synchronize()
    assert h.dtype == DT[rdtype] and y.dtype == DT[dtype]
    b32, r32 = float(np.float32(branch)), float(np.float32(resid))
    (rh, bh), (ry, by) = ref.block_norm(fn, rn, post, _np(par["w_post"]), _np(par["b_post"]), _np(gt), b32, r32, pre,
                                        _np(par["w_pre"]), _np(par["b_pre"]), float(np.float32(eps)),
                                        T // gate[0] if gate else 1)
    ref.check(_np(h), rh, bh, rdtype, "h")
    ref.check(_np(y), ry, by, dtype, "y")


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("none", "rms"), ("rms", "none"), ("layer", "layer"),
                                      ("none", "layer"), ("layer", "none"), ("none", "none")])
@pytest.mark.parametrize("H", [1, 7, 64, 200, 1003, 4096])
def test_kinds_and_widths(lib, post, pre, H):
    _check(lib, 5, H, post=post, pre=pre, bias=True, seed=H)


@pytest.mark.parametrize("dtype,rdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"),
                                          ("f32", "f32")])
@pytest.mark.parametrize("H", [256, 1001, 7168])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full", "sample", "sample-token"])
def test_types_and_gates(lib, dtype, rdtype, H, gate):
    T = 12
    shape = {None: None, "channel": (1, H), "token": (T, 1), "full": (T, H), "sample": (3, H),
             "sample-token": (4, 1)}[gate]
    _check(lib, T, H, dtype=dtype, rdtype=rdtype, gate=shape, post="layer", pre="rms", bias=True, seed=1)


@pytest.mark.parametrize("H", [8192, 8200, 16384, 16392, 32768, 8191, 12345, 32767])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_rows(lib, H, dtype):
    _check(lib, 3, H, dtype=dtype, rdtype=dtype, pre="layer", bias=True, seed=2)


@pytest.mark.parametrize("T", [1, 2, 153, 700, 3001])
@pytest.mark.parametrize("H", [96, 1536])
def test_row_counts(lib, T, H):
    _check(lib, T, H, gate=(T, 1), seed=3)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (8, 8), (1, 5), (0, 4)])
@pytest.mark.parametrize("H", [512, 777])
def test_strides_and_alignment(lib, pad, shift, H):
    _check(lib, 9, H, pad=pad, shift=shift, gate=(9, H), seed=4)


@pytest.mark.parametrize("T", [1, 5, 1000, 4001])
@pytest.mark.parametrize("H", [8, 60, 64, 65, 128, 136, 250, 256])
def test_narrow_rows(lib, T, H):
    _check(lib, T, H, post="layer", pre="rms", gate=(T, 1), bias=True, seed=H)
    _check(lib, T, H, dtype="f32", rdtype="f32", post="rms", pre="layer", gate=(1, H), seed=H)


@pytest.mark.parametrize("T,H,pad", [(1, 13942, 0), (1, 20001, 0), (1, 777, 0), (5, 777, 7), (400, 777, 7), (3, 12345, 7),
                                     (2, 16385, 7), (2, 32767, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_aligned_rows_of_odd_width(lib, T, H, pad, dtype):
    _check(lib, T, H, dtype=dtype, rdtype="f32", post="layer", pre="layer", gate=(1, H), bias=True, pad=pad, seed=8)


def test_parameters_in_the_activations_type(lib):
    _check(lib, 6, 640, pdtype="bf16", post="layer", pre="layer", bias=True)
    _check(lib, 6, 641, dtype="f16", rdtype="f16", pdtype="f16", post="rms", pre="layer", bias=True)


def test_in_place(lib):
    _check(lib, 300, 1024, alias=True, seed=6)
    _check(lib, 300, 515, alias=True, rdtype="f32", seed=6)


def test_no_residual_and_single_outputs(lib):
    _check(lib, 7, 384, residual=False, post="none", pre="rms")
    f = torch.randn((7, 384), device="cuda").to(torch.bfloat16)
    r = torch.randn((7, 384), device="cuda").to(torch.bfloat16)
    h, y = lib.block_norm(f, r, pre="rms")
    h1, none = lib.block_norm(f, r, pre="rms", want_y=False)
    none2, y1 = lib.block_norm(f, r, pre="rms", want_h=False)
    assert none is None and none2 is None
    assert torch.equal(h, h1) and torch.equal(y, y1)
    assert torch.equal(h, (f.float() + r.float()).to(torch.bfloat16))


def test_zero_rows_constant_rows_and_no_rows(lib):
    f = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    f[1] = 3.0
    h, y = lib.block_norm(f, post="layer", pre="rms")
    assert torch.all(h[:2] == 0) and torch.all(y == 0)  # a constant row has no deviation
    h, y = lib.block_norm(f, post="rms", pre="none")
    assert torch.all(h[0] == 0) and torch.all(h[1] == 1)
    h, y = lib.block_norm(f[:0], post="rms")
    assert h.shape == (0, 256) and y.shape == (0, 256)


def test_large_mean_keeps_its_variance(lib):
    # the deviations are taken from the mean before they are squared: a mean 2^11 times larger costs no digits
    g = torch.Generator("cuda").manual_seed(7)
    f = torch.randn((4, 2048), device="cuda", generator=g) + 2048.0
    h, _ = lib.block_norm(f, post="layer", pre="none", eps=0.0)
    d = f.double() - f.double().mean(1, keepdim=True)
    want = d / d.square().mean(1, keepdim=True).sqrt()
    # |error of the mean| <= 48 * 2^-24 * 2048 (derived as for the sums), relative to a deviation of 1
    assert (h.double() - want).abs().max() <= 2 * 48 * 2.0 ** -24 * 2048


def test_non_finite_rows_stay_in_their_rows(lib):
    f = torch.ones((3, 512), dtype=torch.float16, device="cuda")
    f[1, 100] = float("inf")
    f[2, 5] = float("nan")
    h, y = lib.block_norm(f, post="rms", pre="rms")
    assert torch.isfinite(h[0]).all() and torch.isfinite(y[0]).all()
    assert torch.isnan(h[1, 100]) and torch.isnan(y[1]).all() and torch.isnan(y[2]).all()


def test_other_stream(lib):
    f = torch.randn((2048, 4096), device="cuda").to(torch.bfloat16)
    want = lib.block_norm(f, f, post="rms")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lib.block_norm(f, f, post="rms")
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_refusals(lib):
    f = torch.zeros((6, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(lib.W4A8Error, match="H=40000"):
        lib.block_norm(torch.zeros((1, 40000), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.W4A8Error, match="gate_rows=4"):
        lib.block_norm(f, gate=torch.ones((4, 1), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.W4A8Error, match="gate_cols=2"):
        lib.block_norm(f, gate=torch.ones((6, 2), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.W4A8Error, match="none"):
        lib.block_norm(f, post="none", w_post=w)
    with pytest.raises(lib.W4A8Error, match="eps"):
        lib.block_norm(f, eps=-1.0)
    with pytest.raises(lib.W4A8Error, match="nothing to compute"):
        lib.block_norm(f, want_h=False, want_y=False)
    with pytest.raises(ValueError, match="post"):
        lib.block_norm(f, post="group")
    with pytest.raises(TypeError, match="residual"):
        lib.block_norm(f, f.half())
    with pytest.raises(ValueError, match="residual"):
        lib.block_norm(f, f[:5])
    with pytest.raises(TypeError, match="one dtype"):
        lib.block_norm(f, post="rms", w_post=w, pre="rms", w_pre=w.to(torch.bfloat16))
    with pytest.raises(ValueError, match="w_pre"):
        lib.block_norm(f, w_pre=torch.ones(63, device="cuda"))


@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 1), (0, 3), (5, 2), (8, 7), (2, 4)])
@pytest.mark.parametrize("T,H", [(2, 705), (401, 705), (401, 2047), (309, 3999), (3, 7001), (330, 7680), (401, 7682),
                                 (307, 9001)])
@pytest.mark.parametrize("dtype,rdtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_rows_that_start_alike_in_every_matrix(lib, dtype, rdtype, T, H, pad, shift):
    # whole aligned vectors and the single elements beside them, for every start of a row within 16 bytes
    _check(lib, T, H, dtype=dtype, rdtype=rdtype, post="layer", pre="rms", gate=(T, H), bias=True, pad=pad, shift=shift,
           alias=True, seed=11)
    _check(lib, T, H, dtype=dtype, rdtype=rdtype, post="rms", pre="layer", gate=(T, 1), pad=pad, shift=shift, alias=True,
           seed=12)


@pytest.mark.parametrize("T,H,groups", [(400, 1003, 4), (400, 1000, 8), (2, 1003, 2)])
@pytest.mark.parametrize("pad,shift", [(5, 0), (5, 3), (0, 1)])
def test_gates_of_several_rows(lib, T, H, groups, pad, shift):
    _check(lib, T, H, gate=(groups, H), pad=pad, shift=shift, alias=True, seed=13)
    _check(lib, T, H, dtype="f16", rdtype="f32", gate=(groups, H), pad=pad, shift=shift, alias=True, seed=14)


@pytest.mark.parametrize("T,H,pad,shift", [(2, 1001, 0, 1), (401, 1001, 3, 3), (401, 771, 0, 5), (350, 5119, 2, 6)])
@pytest.mark.parametrize("dtype,rdtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_nothing_beside_the_rows_is_written_or_counted(lib, dtype, rdtype, T, H, pad, shift):
    g = torch.Generator("cuda").manual_seed(15)
    bufs, views = [], []
    for dt in (dtype, rdtype):
        buf = torch.full((T * (H + pad) + shift + 16,), float("inf"), dtype=DT[dt], device="cuda")
        v = buf[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H]
        v.copy_(torch.randn((T, H), device="cuda", generator=g).to(DT[dt]))
        bufs.append(buf)
        views.append(v)
    beside = [torch.ones_like(b, dtype=torch.bool) for b in bufs]
    for m in beside:
        m[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H] = False
    f, r = views
    h0, y0 = lib.block_norm(f.contiguous(), r.contiguous(), post="layer", pre="layer", residual_dtype=DT[rdtype])
    lib.block_norm(f, r, post="layer", pre="layer", residual_dtype=DT[rdtype], h=r, y=f)
    torch.cuda.synchronize()
    for b, m in zip(bufs, beside):
        assert torch.isinf(b[m]).all()
    assert torch.isfinite(r).all() and torch.isfinite(f).all()
    # the sums' order differs with a row's start: a few units in the last place of fp32, then each type's rounding
    eps = {"bf16": 2.0**-7, "f16": 2.0**-9, "f32": 2.0**-18}
    assert torch.all((r.double() - h0.double()).abs() <= eps[rdtype] * (1 + h0.double().abs()))
    assert torch.all((f.double() - y0.double()).abs() <= eps[dtype] * (1 + y0.double().abs()))


@pytest.mark.parametrize("H", [129, 136, 200, 248, 255, 256, 257, 300, 504, 512, 513, 704])
@pytest.mark.parametrize("dtype,rdtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_many_short_rows(lib, dtype, rdtype, H):
    # more rows than the warps of the device take in one turn
    _check(lib, 9001, H, dtype=dtype, rdtype=rdtype, post="layer", pre="rms", gate=(9001, 1), bias=True, seed=16)
    _check(lib, 7500, H, dtype=dtype, rdtype=rdtype, post="rms", pre="layer", gate=(1, H), pad=8, alias=True, seed=17)


@pytest.mark.parametrize("T,H", [(1, 4096), (64, 1003), (2048, 4096), (1500, 1003)])
def test_graph(lib, T, H):
    g = torch.Generator("cuda").manual_seed(18)
    f, r = (torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    want = lib.block_norm(f, r, post="rms", pre="layer")
    given = torch.zeros_like(f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.block_norm(given, r, post="rms", pre="layer")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = lib.block_norm(given, r, post="rms", pre="layer")
        given.copy_(f)
        graph.replay()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
