"""paged_kv_append on the GPU against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}


def _np(t):
    return t.float().double().cpu().numpy()


def _table(lens, page, g, spare=3):
    need = [-(-max(n, 0) // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return table.cuda(), sum(need) + spare


def _cache(pages, page, H, D, dtype, layout):
    # every layout's memory is one allocation; what is not written stays 3
    if layout == "heads first":
        c = torch.full((pages, H, page, D), 3.0, device="cuda").to(DT[dtype]).permute(0, 2, 1, 3)
    elif layout == "padded":
        c = torch.full((pages, page + 1, H, D + 16), 3.0, device="cuda").to(DT[dtype])[:, :page, :, :D]
    else:
        c = torch.full((pages, page, H, D), 3.0, device="cuda").to(DT[dtype])
    return c


def _run(lib, past, new, H, D, page, dtype="bf16", cache="bf16", Hq=0, R=None, start=0, interleaved=False, padding=0,
         layout="plain", positions=None, scales=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    B, rows = len(new), sum(new) + padding
    lens = [p + n for p, n in zip(past, new)]
    table, pages = _table(lens, page, g)
    k, v = (torch.randn((rows, H, D), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    q = torch.randn((rows, Hq, D), generator=g).to(DT[dtype]).cuda() if Hq else None
    kc, vc = _cache(pages, page, H, D, cache, layout), _cache(pages, page, H, D, cache, layout)
    ks = (0.01 + 0.02 * torch.rand(H, generator=g)).cuda() if scales else None
    vs = (0.01 + 0.02 * torch.rand(H, generator=g)).cuda() if scales else None
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    one = all(n == 1 for n in new) and seed % 2 == 0
    indptr = None if one else torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
    f = ref.inv_freq(R) if R else None
    pos_t = None if positions is None else torch.tensor(positions, device="cuda")
    q_out = torch.full((rows, Hq, D), 7.0, device="cuda").to(DT[dtype]) if Hq else None
    got = lib.paged_kv_append(k, v, kc, vc, table, lens_t, indptr, freqs=lib.rotary_frequencies(R) if R else None,
                              positions=pos_t, interleaved=interleaved, start=start, scale=1.1 if R else 1.0, k_scale=ks,
                              v_scale=vs, q=q, q_out=q_out)
    assert got is q_out
    assert lib.device_error() == 0
    at = np.array([p + i for p, n in zip(past, new) for i in range(n)], dtype=np.int64)
    seq = np.array([b for b, n in enumerate(new) for _ in range(n)], dtype=np.int64)
    n = len(at)
    turn = at if positions is None else np.asarray(positions)[:n]

    def rot(x):
        if not R:
            return _np(x[:n]), np.zeros((n,) + tuple(x.shape[1:]))
        return ref.rotate(_np(x[:n]), turn, f, interleaved, start, 1.1)
    host = table.cpu().numpy()
    page_id, slot = host[seq, at // page], at % page
    for c, x, s, turned in ((kc, k, ks, True), (vc, v, vs, False)):
        want, slack = rot(x) if turned else (_np(x[:n]), np.zeros((n, H, D)))
        have = _np(c)
        mine = have[page_id, slot]
        if cache == "fp8":
            scale = np.ones(H) if s is None else _np(s)
            mine = mine * scale[None, :, None]
            want = np.clip(want, -448 * scale[None, :, None], 448 * scale[None, :, None])
            # half a step of E4M3: 2^-4 relative, 2^-10 among the smallest; before it a division rounded in fp32
            bound = (np.abs(want) * 2.0 ** -4 + 2.0 ** -10 * scale[None, :, None]) * (1 + 2.0 ** -4) + 2 * slack
            assert (np.abs(mine - want) <= bound + 4 * ref.U * np.abs(want)).all()
        elif turned:
            assert (np.abs(mine - want) <= ref.rounded(want, cache, slack)).all()
        else:
            assert np.array_equal(mine, want)
        rest = np.ones(have.shape[:2], bool)
        rest[page_id, slot] = False
        assert (have[rest] == 3.0).all()  # no other slot is touched
        if layout == "padded":
            whole = torch.as_strided(c, (pages, page + 1, H, D + 16), c.stride()[:3] + (1,)).float()
            assert torch.all(whole[:, page:] == 3.0) and torch.all(whole[:, :, :, D:] == 3.0)
    if Hq:
        want, slack = rot(q)
        assert (np.abs(_np(got)[:n] - want) <= ref.rounded(want, dtype, slack)).all()
        assert torch.all(got[n:] == 7.0)  # rows behind the last sequence
    return got


CASES = [
    dict(past=[0], new=[1], H=1, D=8, page=16),
    dict(past=[5, 0, 31, 16], new=[1, 1, 1, 1], H=8, D=128, page=16, Hq=64, R=128),
    dict(past=[7, 0, 32], new=[1, 1, 1], H=2, D=64, page=16, Hq=4, R=64, padding=5),
    dict(past=[5, 0, 31, 16], new=[1, 1, 1, 1], H=3, D=96, page=7, R=48, start=48, interleaved=True, seed=1),
    dict(past=[0, 700, 3], new=[300, 1, 77], H=5, D=64, page=64, Hq=5, R=32, padding=9, layout="heads first"),
    dict(past=[0, 0, 9, 0, 0, 2], new=[0, 40, 0, 0, 13, 0], H=2, D=72, page=1, R=24, start=8, padding=3),
    dict(past=[100] * 300, new=[i % 3 for i in range(300)], H=4, D=80, page=16, dtype="f16", cache="f16", R=80),
    dict(past=[3, 8], new=[20, 30], H=2, D=33, page=5, R=20, start=3, layout="padded"),
    dict(past=[3, 8], new=[20, 30], H=2, D=48, page=16, Hq=6, layout="padded", dtype="f16", cache="f16"),
    dict(past=[0], new=[2000], H=1, D=256, page=128, Hq=1, R=256, interleaved=True),
    dict(past=[0], new=[5], H=2, D=1024, page=3, R=1024, Hq=3),
    dict(past=[70000, 2], new=[3, 4], H=1, D=16, page=100, R=16, Hq=16),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_append(lib, case):
    _run(lib, **case)


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
@pytest.mark.parametrize("scales", [False, True])
def test_append_to_8_bits(lib, case, scales):
    _run(lib, **{**case, "cache": "fp8"}, scales=scales)


@pytest.mark.parametrize("D,R,start,H,Hq", [(90, 44, 46, 3, 5), (90, 44, 0, 2, 0), (1022, 1020, 2, 2, 1), (1023, 2, 1021, 1, 1),
                                              (6, 2, 2, 4, 8), (100, 0, 0, 2, 0), (1, 0, 0, 3, 0)])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_narrow_vectors(lib, D, R, start, H, Hq, dtype, cache, interleaved):
    _run(lib, [3, 0, 40], [20, 1, 30], H, D, 7, R=R, start=start, Hq=Hq, dtype=dtype, cache=cache, interleaved=interleaved)


def test_positions_of_their_own(lib):
    _run(lib, [4, 0], [3, 6], 2, 64, 16, R=64, Hq=2, positions=[9, 8, 7, 100000, 5, 4, 3, 2, 1])


def test_saturates_and_keeps_nan(lib):
    k = torch.tensor([1e4, -1e4, float("inf"), float("nan"), 448.0, 465.0, 2.0 ** -10, 0.0],
                     device="cuda").to(torch.bfloat16).view(1, 1, 8)
    kc, vc = (torch.zeros((1, 1, 1, 8), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    lib.paged_kv_append(k, k, kc, vc, one.view(1, 1) - 1, one)
    for c in (kc, vc):
        got = c.float().flatten().tolist()
        assert got[:3] == [448.0, -448.0, 448.0] and got[3] != got[3] and got[4:] == [448.0, 448.0, 0.0, 0.0]


@pytest.mark.parametrize("scale", [1e-41, 1e-30, 0.75, 3e4, 1e30, -0.5])
def test_scales_of_any_size(lib, scale):
    x = torch.tensor([0.0, 1.0, -3.5, 2.0 ** -20, 3e38, -1e-38, 100.0, float("inf")], device="cuda").to(torch.bfloat16)
    kc, vc = (torch.zeros((1, 1, 1, 8), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    s = torch.full((1,), scale, device="cuda")
    lib.paged_kv_append(x.view(1, 1, 8), x.view(1, 1, 8), kc, vc, one.view(1, 1) - 1, one, k_scale=s, v_scale=s)
    # the quotient rounded to fp32 once, then to E4M3, beyond 448 saturating
    q = (x.double().cpu() / s.double().cpu()).float().clamp(-448, 448)
    assert torch.equal(kc.flatten().cpu().float(), q.to(torch.float8_e4m3fn).float()) and torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))


def test_padded_decode_batch(lib):
    # sequences of length 0 in a batch of one token each: nothing is stored for them
    B, H, D = 6, 2, 64
    lens = torch.tensor([3, 0, 1, 0, 17, -4], dtype=torch.int32, device="cuda")
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2)
    k, v, q = (torch.randn((B, H, D), device="cuda").to(torch.bfloat16) for _ in range(3))
    kc, vc = (torch.full((12, 16, H, D), 3.0, device="cuda").to(torch.bfloat16) for _ in range(2))
    keep = q.clone()
    got = lib.paged_kv_append(k, v, kc, vc, table, lens, freqs=lib.rotary_frequencies(D), q=q, q_out=q)
    assert got is q
    left = [1, 3, 5]
    assert torch.equal(q[left], keep[left]) and not torch.equal(q[0], keep[0])
    assert lib.device_error() == 0
    rest = torch.ones((12, 16), dtype=torch.bool, device="cuda")
    rest[0, 2] = rest[4, 0] = rest[9, 0] = False
    assert torch.all(kc[rest] == 3.0) and torch.all(vc[rest] == 3.0)
    assert torch.equal(vc[0, 2], v[0]) and torch.equal(vc[4, 0], v[2]) and torch.equal(vc[9, 0], v[4])


def test_bad_pages_are_left_out(lib):
    # the kernel checks every page id and position before it stores: an error code, and nothing written
    k = torch.randn((4, 1, 16), device="cuda").to(torch.bfloat16)
    kc, vc = (torch.full((3, 4, 1, 16), 3.0, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[0], [3], [-1], [1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2, 2, 2, 5], dtype=torch.int32, device="cuda")  # the last is behind its only page
    lib.paged_kv_append(k, k, kc, vc, table, lens)
    assert lib.device_error() == 2 and lib.device_error() == 0
    assert torch.equal(kc[0, 1], k[0])
    kc[0, 1] = vc[0, 1] = 3.0
    assert torch.all(kc == 3.0) and torch.all(vc == 3.0)


def test_places_beyond_32_bits(lib):
    # 2.2e9 elements between two pages
    far = 2_200_000_000
    store = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda")
    kc = store.as_strided((2, 4, 2, 64), (far, 128, 64, 1))
    vc = store[1024:].as_strided((2, 4, 2, 64), (far, 128, 64, 1))
    k, v = (torch.randn((1, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    lib.paged_kv_append(k, v, kc, vc, one.view(1, 1), one * 3)
    assert torch.equal(kc[1, 2], k[0]) and torch.equal(vc[1, 2], v[0])
    assert int(torch.count_nonzero(store)) == int(torch.count_nonzero(k) + torch.count_nonzero(v))


def test_graph_follows_its_lengths(lib):
    B, H, D = 3, 2, 32
    k, v = (torch.randn((B, H, D), device="cuda").to(torch.float16) for _ in range(2))
    kc, vc = (torch.zeros((6, 8, H, D), device="cuda").half() for _ in range(2))
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    lib.paged_kv_append(k, v, kc, vc, table, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.paged_kv_append(k, v, kc, vc, table, lens)
    for i in range(2, 17):
        lens.fill_(i)
        k.normal_()
        v.normal_()
        graph.replay()
        at = (table[:, (i - 1) // 8].long(), (i - 1) % 8)
        assert torch.equal(kc[at], k) and torch.equal(vc[at], v)


def test_refusals(lib):
    B, H, D = 2, 2, 16
    k = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros((4, 8, H, D), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    n = torch.ones(B, dtype=torch.int32, device="cuda")
    f = lib.rotary_frequencies(16)
    s = torch.ones(H, device="cuda")
    base = dict(k=k, v=k, k_cache=c, v_cache=c.clone(), page_table=t, seq_lens=n)
    for change, err, msg in [
            (dict(k=k.float()), TypeError, "k must be"), (dict(v=k.half()), TypeError, "v must be"),
            (dict(v=k[:1]), ValueError, "v must have shape"), (dict(k_cache=c.half()), TypeError, "k_cache"),
            (dict(v_cache=c[:3]), ValueError, "v_cache must have"), (dict(k_cache=c[0]), ValueError, "4 dimensions"),
            (dict(k_cache=c[:, :, :1].contiguous(), v_cache=c[:, :, :1].contiguous()), ValueError, "heads"),
            (dict(k_cache=c[:1].expand(4, 8, H, D), v_cache=c), ValueError, "overlapping"),
            (dict(page_table=t.long()), TypeError, "page_table"), (dict(page_table=t[0]), ValueError, "2 dimensions"),
            (dict(seq_lens=n[:1]), ValueError, "seq_lens"), (dict(seq_lens=n.long()), TypeError, "seq_lens"),
            (dict(seq_lens=None), TypeError, "seq_lens"), (dict(indptr=n), ValueError, "indptr"),
            (dict(k=k[:1], v=k[:1]), ValueError, "without indptr"), (dict(k_scale=s), lib.W4A8Error, "scales"),
            (dict(k_scale=s.half()), TypeError, "k_scale"), (dict(freqs=f, start=2), lib.W4A8Error, "start=2"),
            (dict(positions=n), ValueError, "positions"), (dict(freqs=f, positions=n[:1]), ValueError, "positions"),
            (dict(q=k.half()), TypeError, "q must be"), (dict(q=k[:1]), ValueError, "q must have"),
            (dict(q_out=k), ValueError, "without q"), (dict(q=k, q_out=k[:, :1]), ValueError, "q_out"),
            (dict(q=k, q_out=k[:1].expand(2, H, D)), ValueError, "overlapping"),
            (dict(k_cache=c.cpu()), TypeError, "CUDA")]:
        with pytest.raises(err, match=msg):
            lib.paged_kv_append(**{**base, **change})
    assert lib.paged_kv_append(**base) is None and lib.device_error() == 0


@pytest.mark.parametrize("indptr", [False, True])
@pytest.mark.parametrize("dtype,cache,D", [("bf16", "bf16", 64), ("f16", "fp8", 64), ("bf16", "bf16", 90), ("f16", "f16", 33)])
@pytest.mark.parametrize("turned", [False, True])
def test_queries_left_out_are_zeros_in_fresh_memory(lib, indptr, dtype, cache, D, turned):
    # an empty sequence, one of negative length, rows behind the last: a tensor made by the call holds zeros there, a given
    # one what it held
    H, Hq, rows = 2, 6, 9
    lens = torch.tensor([3, 0, 1, -4, 17], dtype=torch.int32, device="cuda")
    table = torch.arange(10, dtype=torch.int32, device="cuda").view(5, 2)
    k, v = (torch.randn((rows, H, D), device="cuda").to(DT[dtype]) for _ in range(2))
    q = torch.randn((rows, Hq, D), device="cuda").to(DT[dtype])
    ends = torch.tensor([0, 2, 3, 4, 4, 6], dtype=torch.int32, device="cuda") if indptr else None
    left = [2, 6, 7, 8] if indptr else [1, 3, 5, 6, 7, 8]
    rest = [i for i in range(rows) if i not in left]
    kw = dict(freqs=lib.rotary_frequencies(D // 2 * 2)) if turned else {}
    kc, vc = (torch.full((10, 16, H, D), 3.0, device="cuda").to(DT[cache]) for _ in range(2))
    given = torch.full_like(q, 7.0)
    lib.paged_kv_append(k, v, kc, vc, table, lens, ends, q=q, q_out=given, **kw)
    assert torch.all(given[left] == 7.0)
    for _ in range(3):
        keep = kc.clone(), vc.clone()
        poison = torch.full_like(q, float("nan"))  # the memory that the call is given next, most likely
        del poison
        made = lib.paged_kv_append(k, v, kc, vc, table, lens, ends, q=q, **kw)
        assert torch.all(made[left] == 0) and torch.equal(made[rest], given[rest])
        assert torch.equal(kc.view(torch.uint8), keep[0].view(torch.uint8))
        assert torch.equal(vc.view(torch.uint8), keep[1].view(torch.uint8))
    assert lib.device_error() == 0


def test_queries_of_a_batch_without_sequences(lib):
    q = torch.randn((5, 4, 64), device="cuda").to(torch.bfloat16)
    k, c = q[:, :2], torch.full((3, 16, 2, 64), 3.0, device="cuda").to(torch.bfloat16)
    none, table = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for indptr in (None, zero):
        poison = torch.full_like(q, float("nan"))
        del poison
        made = lib.paged_kv_append(k, k, c, c.clone(), table, none, indptr, q=q)
        assert torch.all(made == 0) and torch.all(c == 3.0)
        given = torch.full_like(q, 7.0)
        lib.paged_kv_append(k, k, c, c.clone(), table, none, indptr, q=q, q_out=given)
        assert torch.all(given == 7.0)
    assert lib.paged_kv_append(k, k, c, c.clone(), table, none, None, q=q[:, :0]).shape == (5, 0, 64)
    assert lib.device_error() == 0


@pytest.mark.parametrize("length", [-(2 ** 31), -(2 ** 31) + 1, -(2 ** 31) + 2, -1])
@pytest.mark.parametrize("indptr", [False, True])
def test_the_smallest_lengths_are_left_out(lib, length, indptr):
    k = torch.randn((3, 1, 16), device="cuda").to(torch.bfloat16)
    kc, vc = (torch.full((3, 4, 1, 16), 3.0, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, 3], dtype=torch.int32, device="cuda") if indptr else None
    q = torch.full_like(k, 7.0)
    lib.paged_kv_append(k, k, kc, vc, table, lens, ends, q=k, q_out=q)
    assert lib.device_error() == 0
    assert torch.all(kc == 3.0) and torch.all(vc == 3.0) and torch.all(q == 7.0)
