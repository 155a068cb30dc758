"""Argument checks of the attention half's operators at the C ABI, without a GPU: nothing is launched."""
import ctypes

import pytest

NULL = None
P16 = ctypes.c_void_p(16)  # never dereferenced: every call below is refused first
P17, P18, P20 = ctypes.c_void_p(17), ctypes.c_void_p(18), ctypes.c_void_p(20)
BF16, F16, F32, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def clib():
    from w4afp8_mixture_experts_gb300 import build
    build.build()
    import w4afp8_mixture_experts_gb300._binding as b
    return b.load()


def _turn(freqs=16, R=8, start=0, scale=1.0, positions=16, wide=0):
    from w4afp8_mixture_experts_gb300._binding import Rotary
    return Rotary(freqs or None, R, start, 0, 0, scale, positions or None, wide)


def _cache(k=16, v=16, dtype=BF16, pages=4, page_size=16, heads=2, D=64, table=16, table_ld=4, table_pages=4, lens=16, B=3,
           k_scale=0, v_scale=0, strides=(2048, 128, 64) * 2):
    from w4afp8_mixture_experts_gb300._binding import PagedCache
    return PagedCache(k or None, v or None, *strides, dtype, pages, page_size, heads, D, table or None, table_ld, table_pages,
                      lens or None, B, k_scale or None, v_scale or None)


def _rotary(L, x=P16, lt=64, lh=64, dt=BF16, T=4, H=1, D=64, turn=_turn, out=P16, ot=64, oh=64, **kw):
    r = turn(**kw) if turn else None
    return L.rotary_embedding(x, lt, lh, dt, T, H, D, r and ctypes.byref(r), out, ot, oh, NULL)


def _append(L, k=P16, v=P16, dt=BF16, T=3, indptr=NULL, turn=None, q=NULL, Hq=0, qo=NULL, kt=128, **kw):
    c = _cache(**kw)
    return L.paged_kv_append(k, kt, 64, v, 128, 64, dt, T, indptr, ctypes.byref(c), turn and ctypes.byref(turn), q, 64, 64, Hq,
                             qo, 64, 64, NULL)


def _attend(L, q=P16, dt=BF16, Hq=4, scale=1.0, window=0, out=P16, lse=NULL, ws=P16, ws_bytes=1 << 40, qb=256, **kw):
    c = _cache(**kw)
    return L.paged_attention_decode(q, qb, 64, dt, Hq, ctypes.byref(c), scale, window, out, 256, 64, lse, ws, ws_bytes, NULL)


def _linear(L, A=P16, s=P16, lds=4, B=P16, bs=P16, M=4, N=32, K=128, out=P16, ldo=32, od=BF16):
    return L.fp8_block_linear(A, s, lds, B, bs, M, N, K, out, ldo, od, NULL)


@pytest.mark.parametrize("call,msg", [
    (lambda L: _rotary(L, dt=3), b"dtype=3"),
    (lambda L: _rotary(L, D=0), b"D=0"),
    (lambda L: _rotary(L, D=1025), b"D=1025"),
    (lambda L: _rotary(L, T=-1), b"T=-1"),
    (lambda L: _rotary(L, T=1 << 20, H=1 << 11), b"below 2^31"),
    (lambda L: _rotary(L, lt=-64), b"strides"),
    (lambda L: _rotary(L, turn=None), b"null"),
    (lambda L: _rotary(L, freqs=0), b"null"),
    (lambda L: _rotary(L, R=7), b"R=7"),
    (lambda L: _rotary(L, R=66), b"R=66"),
    (lambda L: _rotary(L, start=57), b"start=57"),
    (lambda L: _rotary(L, start=-1), b"start=-1"),
    (lambda L: _rotary(L, scale=float("nan")), b"finite"),
    (lambda L: _rotary(L, positions=0), b"positions"),
    (lambda L: _rotary(L, positions=18), b"aligned"),
    (lambda L: _rotary(L, positions=20, wide=1), b"aligned"),
    (lambda L: _rotary(L, x=NULL), b"null"),
    (lambda L: _rotary(L, out=P17), b"aligned"),
    (lambda L: _append(L, dt=F32), b"dtype=2"),
    (lambda L: _append(L, dtype=F16), b"cache dtype=1"),
    (lambda L: _append(L, D=1025), b"D=1025"),
    (lambda L: _append(L, B=-1), b"B=-1"),
    (lambda L: _append(L, page_size=0), b"page_size=0"),
    (lambda L: _append(L, pages=1 << 31), b"pages="),
    (lambda L: _append(L, table_pages=1 << 28, table_ld=1 << 28), b"table_pages"),
    (lambda L: _append(L, table_ld=3), b"table_ld=3"),
    (lambda L: _append(L, heads=0), b"heads=0"),
    (lambda L: _append(L, strides=(2048, 128, 64, 2048, -128, 64)), b"strides"),
    (lambda L: _append(L, k_scale=16), b"scales"),
    (lambda L: _append(L, k_scale=18, dtype=E4M3), b"aligned"),
    (lambda L: _append(L, T=2), b"T=2"),
    (lambda L: _append(L, T=1 << 30, indptr=P16), b"below 2^31"),
    (lambda L: _append(L, indptr=P18), b"indptr"),
    (lambda L: _append(L, Hq=2), b"Hq=2"),
    (lambda L: _append(L, q=P16, Hq=2), b"null"),
    (lambda L: _append(L, k=NULL), b"null"),
    (lambda L: _append(L, k=P17), b"aligned"),
    (lambda L: _append(L, lens=0), b"null"),
    (lambda L: _append(L, table=0), b"page_table"),
    (lambda L: _append(L, v_scale=0, k=P16, kt=-1), b"strides"),
    (lambda L: _append(L, turn=_turn(R=9)), b"R=9"),
    (lambda L: _attend(L, dt=F32), b"dtype=2"),
    (lambda L: _attend(L, D=60), b"D=60"),
    (lambda L: _attend(L, D=264), b"D=264"),
    (lambda L: _attend(L, D=24, dtype=E4M3), b"D=24"),
    (lambda L: _attend(L, Hq=3), b"Hq=3"),
    (lambda L: _attend(L, Hq=514), b"Hq=514"),
    (lambda L: _attend(L, window=-1), b"window=-1"),
    (lambda L: _attend(L, scale=float("inf")), b"finite"),
    (lambda L: _attend(L, qb=-1), b"strides"),
    (lambda L: _attend(L, B=1 << 23), b"2^24"),
    (lambda L: _attend(L, q=P17), b"aligned"),
    (lambda L: _attend(L, lse=P18), b"aligned"),
    (lambda L: _attend(L, k=20), b"multiples of 16 bytes"),
    (lambda L: _attend(L, strides=(2048, 132, 64) * 2), b"multiples of 16 bytes"),
    (lambda L: _attend(L, table=0), b"page_table"),
    (lambda L: _attend(L, out=NULL), b"null"),
    (lambda L: _linear(L, od=3), b"out_dtype=3"),
    (lambda L: _linear(L, M=-1), b"M=-1"),
    (lambda L: _linear(L, N=(1 << 20) + 1, ldo=1 << 21), b"N=1048577"),
    (lambda L: _linear(L, K=64), b"K=64"),
    (lambda L: _linear(L, K=200), b"K=200"),
    (lambda L: _linear(L, lds=3), b"lda_s=3"),
    (lambda L: _linear(L, lds=6), b"lda_s=6"),
    (lambda L: _linear(L, ldo=31), b"ldo=31"),
    (lambda L: _linear(L, A=NULL), b"null"),
    (lambda L: _linear(L, B=P20), b"16-byte"),
    (lambda L: _linear(L, out=P18, od=F32), b"aligned"),
])
def test_refused_before_launch(clib, call, msg):
    assert call(clib) == 1  # W4A8_ERR_INVALID_ARG
    assert msg in clib.w4a8_last_error(), clib.w4a8_last_error()


def test_empty_calls_launch_nothing(clib):
    assert _rotary(clib, T=0, x=NULL, out=NULL) == 0 and _rotary(clib, H=0) == 0
    assert _append(clib, T=0, B=0, k=NULL) == 0
    assert _attend(clib, B=0, q=NULL, out=NULL) == 0
    assert _linear(clib, M=0, A=NULL, lds=0) == 0 and _linear(clib, N=0, ldo=0) == 0
    assert clib.paged_attention_workspace_bytes(0, 4, 2, 64, 0, -1) == 0


def test_sources_load_nothing_as_constant():
    # as for the other operators: programmatic launch starts these kernels while their inputs may still be written
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4afp8_mixture_experts_gb300", "csrc")
    files = glob.glob(os.path.join(csrc, "paged*")) + glob.glob(os.path.join(csrc, "fp8_linear*"))
    assert len(files) >= 7
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        assert not re.findall(r"__ldg|\.nc\b|__restrict__|__builtin_nontemporal_load", code), os.path.basename(f)


def _whole(L, B=3, T=3, k=P16, q=P16, Hq=2, qo=P16, **kw):
    c = _cache(B=B, **kw)
    return L.paged_kv_append_whole(k, 128, 64, P16, 128, 64, BF16, T, NULL, ctypes.byref(c), NULL, q, 64, 64, Hq, qo, 64, 64,
                                   NULL)


@pytest.mark.parametrize("call,msg", [
    (lambda L: _whole(L, T=2), b"T=2"),
    (lambda L: _whole(L, qo=NULL), b"null"),
    (lambda L: _whole(L, B=0, qo=NULL), b"null"),
    (lambda L: _whole(L, B=0, k=NULL), b"null"),
    (lambda L: _whole(L, lens=0), b"null"),
    (lambda L: _whole(L, table=0), b"page_table"),
    (lambda L: _whole(L, q=NULL), b"Hq=2"),
    (lambda L: _whole(L, D=0), b"D=0"),
])
def test_append_of_whole_outputs_refused_before_launch(clib, call, msg):
    assert call(clib) == 1
    assert msg in clib.w4a8_last_error(), clib.w4a8_last_error()


def test_append_of_whole_outputs_without_rows_launches_nothing(clib):
    assert _whole(clib, B=0, T=0, k=NULL, qo=NULL) == 0
    assert _whole(clib, B=0, Hq=0, q=NULL, qo=NULL) == 0
