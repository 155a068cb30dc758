"""Argument checks of the operators around the routed experts at the C ABI, without a GPU: nothing is launched."""
import ctypes

import pytest

NULL = None
P16 = ctypes.c_void_p(16)  # never dereferenced: every call below is refused first
P18 = ctypes.c_void_p(18)
P17 = ctypes.c_void_p(17)
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def clib():
    from w4afp8_mixture_experts_gb300 import build
    build.build()
    import w4afp8_mixture_experts_gb300._binding as b
    return b.load()


def _route(L, logits=P16, dt=F32, ld=64, T=4, E=64, k=4, score=1, bias=NULL, G=8, keep=4, top=2, ids=P16, w=P16):
    return L.moe_route_grouped_topk(logits, dt, ld, T, E, k, score, bias, G, keep, top, 1, 1.0, ids, w, NULL)


def _norm(L, f=P16, ldf=64, dt=BF16, r=P16, ldr=64, rdt=BF16, post=1, w=NULL, gate=NULL, ldg=64, gr=1, gc=64, gd=BF16,
          pre=1, pd=F32, eps=1e-6, T=4, H=64, h=P16, ldh=64, y=P16, ldy=64):
    return L.block_norm(f, ldf, dt, r, ldr, rdt, post, w, NULL, gate, ldg, gr, gc, gd, 1.0, 1.0, pre, NULL, NULL, pd,
                        eps, T, H, h, ldh, y, ldy, NULL)


def _linear(L, x=P16, ldx=64, w=P16, ldw=64, dt=BF16, bias=NULL, bd=F32, act=0, gated=0, r=NULL, ldr=32, out=P16, ldo=32,
            od=BF16, M=4, N=32, K=64):
    return L.dense_linear(x, ldx, w, ldw, dt, bias, bd, act, gated, r, ldr, out, ldo, od, M, N, K, NULL, 0, NULL)


@pytest.mark.parametrize("call,msg", [
    (lambda L: _route(L, dt=3), b"logits_dtype=3"),
    (lambda L: _route(L, score=2), b"score=2"),
    (lambda L: _route(L, E=1025, ld=1025), b"E=1025"),
    (lambda L: _route(L, ld=63), b"ld=63"),
    (lambda L: _route(L, k=33), b"k=33"),
    (lambda L: _route(L, G=33), b"n_group=33"),
    (lambda L: _route(L, G=7), b"n_group=7"),
    (lambda L: _route(L, keep=0), b"topk_group=0"),
    (lambda L: _route(L, G=64, top=2), b"n_group=64"),
    (lambda L: _route(L, G=32, top=3), b"group_top=3"),
    (lambda L: _route(L, k=9, keep=1), b"k=9"),
    (lambda L: _route(L, T=-1), b"T=-1"),
    (lambda L: _route(L, ids=NULL), b"null"),
    (lambda L: _route(L, logits=P18), b"aligned"),
    (lambda L: _norm(L, dt=5), b"dtype=5"),
    (lambda L: _norm(L, dt=F16, rdt=BF16), b"residual_dtype"),
    (lambda L: _norm(L, dt=F16, rdt=F16, pd=BF16), b"param_dtype"),
    (lambda L: _norm(L, post=3), b"post=3"),
    (lambda L: _norm(L, H=0), b"H=0"),
    (lambda L: _norm(L, H=32769, ldf=40000, ldr=40000, ldh=40000, ldy=40000), b"H=32769"),
    (lambda L: _norm(L, ldf=63), b"leading dimensions"),
    (lambda L: _norm(L, post=0, w=P16), b"none"),
    (lambda L: _norm(L, gate=P16, gd=F16), b"gate_dtype"),
    (lambda L: _norm(L, gate=P16, gr=3), b"gate_rows=3"),
    (lambda L: _norm(L, gate=P16, gc=2), b"gate_cols=2"),
    (lambda L: _norm(L, gate=P16, ldg=63), b"ldg=63"),
    (lambda L: _norm(L, h=NULL, y=NULL), b"nothing"),
    (lambda L: _norm(L, f=NULL), b"null"),
    (lambda L: _norm(L, f=P17), b"aligned"),
    (lambda L: _norm(L, eps=-1.0), b"eps"),
    (lambda L: _linear(L, dt=F32), b"dtype=2"),
    (lambda L: _linear(L, dt=F16, od=BF16), b"out_dtype"),
    (lambda L: _linear(L, bias=P16, bd=F16), b"bias_dtype"),
    (lambda L: _linear(L, act=5), b"act=5"),
    (lambda L: _linear(L, K=0), b"K=0"),
    (lambda L: _linear(L, M=(1 << 20) + 1), b"M=1048577"),
    (lambda L: _linear(L, N=31, gated=1), b"N=31"),
    (lambda L: _linear(L, ldx=63), b"ldx=63"),
    (lambda L: _linear(L, ldo=31), b"ldo=31"),
    (lambda L: _linear(L, r=P16, ldr=31), b"ldr=31"),
    (lambda L: _linear(L, out=NULL), b"null"),
    (lambda L: _linear(L, w=P17), b"aligned"),
    (lambda L: _linear(L, od=F32, out=P18), b"aligned"),
    (lambda L: L.w4a8_moe_forward_routed(P16, P16, P16, 4, 256, 256, 8, 9, P16, P16, P16, P16, P16, P16, 1 << 30, NULL),
     b"k=9"),
    (lambda L: L.w4a8_moe_forward_routed(P16, NULL, P16, 4, 256, 256, 8, 2, P16, P16, P16, P16, P16, P16, 1 << 30, NULL),
     b"null"),
    (lambda L: L.w4a8_moe_forward_routed(P16, P16, P16, 4, 256, 256, 8, 2, P16, P16, P16, P16, P16, P16, 10, NULL),
     b"workspace too small"),
])
def test_refused_before_launch(clib, call, msg):
    assert call(clib) == 1  # W4A8_ERR_INVALID_ARG
    assert msg in clib.w4a8_last_error(), clib.w4a8_last_error()


def test_empty_calls_launch_nothing(clib):
    assert _route(clib, T=0, logits=NULL, ids=NULL, w=NULL) == 0
    assert _norm(clib, T=0) == 0
    assert _linear(clib, M=0) == 0 and _linear(clib, N=0) == 0


def test_wait_test_refuses(clib):
    assert clib.w4a8_test_linear_wait(8, 1000, P16, NULL) == 1 and b"missing=8" in clib.w4a8_last_error()
    assert clib.w4a8_test_linear_wait(0, 3_000_000_000, P16, NULL) == 1 and b"limit_ns" in clib.w4a8_last_error()
    assert clib.w4a8_test_linear_wait(0, 1000, NULL, NULL) == 1 and b"gave_up" in clib.w4a8_last_error()


def test_routed_layer_runs_on_its_tensors_device(clib, monkeypatch):
    # the device and the stream are those of x, whatever the current device; a tensor of another device is refused
    import contextlib

    import torch

    import w4afp8_mixture_experts_gb300._binding as b

    class OnDevice1(torch.Tensor):  # CPU memory that says it lies on the second device
        is_cuda = property(lambda self: True)
        device = property(lambda self: torch.device("cuda", getattr(self, "place", 1)))

    def make(*shape, dtype):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice1)

    calls = []

    class Lib:
        def w4a8_moe_forward_routed(self, *a):
            calls.append(("call", a[-1].value))
            return 0

    @contextlib.contextmanager
    def device(d):
        calls.append(("enter", d))
        yield
        calls.append(("leave", d))

    class Stream:
        def __init__(self, d):
            self.cuda_stream = 100 + (0 if d is None else torch.device(d).index)

    monkeypatch.setattr(b, "load", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(d))
    T, H, I, E, k = 4, 256, 128, 8, 2
    args = dict(x=make(T, H, dtype=torch.bfloat16), topk_ids=make(T, k, dtype=torch.int32),
                topk_w=make(T, k, dtype=torch.float32), w13=make(E, 2 * I, H // 2, dtype=torch.uint8),
                w13_s=make(E, H // 128, 2 * I, dtype=torch.float32), w2=make(E, H, I // 2, dtype=torch.uint8),
                w2_s=make(E, I // 128, H, dtype=torch.float32), ws=make(1024, dtype=torch.uint8),
                out=make(T, H, dtype=torch.bfloat16))
    b.w4a8_moe_forward_routed(**args)
    one = torch.device("cuda", 1)
    assert calls == [("enter", one), ("call", 101), ("leave", one)]
    args["w2"].place = 0
    with pytest.raises(ValueError, match="w2 must be on cuda:1"):
        b.w4a8_moe_forward_routed(**args)
