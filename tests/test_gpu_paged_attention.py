"""paged_attention_decode on the GPU against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}


def _np(t):
    return t.float().double().cpu().numpy()


class Case:
    """A cache with random pages; NaN wherever no sequence has a token, -1 behind each row of the table."""

    def __init__(self, lens, Hq, Hkv, D, page, dtype="bf16", cache=None, layout="plain", seed=0, spread=1.0, scales=True):
        g = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        self.lens, self.Hq, self.Hkv, self.D, self.page, self.dtype, self.cache = lens, Hq, Hkv, D, page, dtype, cache
        need = [-(-max(n, 0) // page) for n in lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
        self.q = (torch.randn((len(lens), Hq, D), generator=g) * spread).to(DT[dtype])
        k, v = (torch.full((pages, page, Hkv, D), math.nan) for _ in range(2))
        self.k, self.v = [], []
        fp8 = cache == "fp8"
        self.ks = (0.02 + 0.02 * torch.rand(Hkv, generator=g)) if fp8 and scales else None
        self.vs = (0.02 + 0.02 * torch.rand(Hkv, generator=g)) if fp8 and scales else None
        for b, n in enumerate(lens):
            ids = [order.pop() for _ in range(need[b])]
            table[b, :need[b]] = torch.tensor(ids, dtype=torch.int32)
            rows = [(torch.randn((max(n, 0), Hkv, D), generator=g) * (30.0 if fp8 else 1.0)).to(DT[cache]) for _ in range(2)]
            at = torch.arange(max(n, 0))
            where = (table[b].long()[at // page], at % page)
            k[where], v[where] = rows[0].float(), rows[1].float()
            one = torch.ones(Hkv)
            self.k.append(_np(rows[0]) * _np(one if self.ks is None else self.ks)[None, :, None])
            self.v.append(_np(rows[1]) * _np(one if self.vs is None else self.vs)[None, :, None])

        def place(c):
            c = c.to(DT[cache])
            if layout == "heads first":
                return c.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
            if layout == "one allocation":  # keys and values of a token side by side
                both = torch.empty((pages, page, Hkv, 2, D), dtype=DT[cache], device="cuda")
                return both
            return c.cuda()
        self.kc, self.vc = place(k), place(v)
        if layout == "one allocation":
            both = self.kc
            both[:, :, :, 0].copy_(k.to(DT[cache]).cuda())
            both[:, :, :, 1].copy_(v.to(DT[cache]).cuda())
            self.kc, self.vc = both[:, :, :, 0], both[:, :, :, 1]
        self.table, self.q = table.cuda(), self.q.cuda()
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if self.ks is not None:
            self.ks, self.vs = self.ks.cuda(), self.vs.cuda()

    def call(self, lib, **kw):
        return lib.paged_attention_decode(self.q, self.kc, self.vc, self.table, self.lens_t, k_scale=self.ks, v_scale=self.vs,
                                          **kw)

    def check(self, lib, out, lse, scale=None, window=0):
        scale = self.D ** -0.5 if scale is None else scale
        # a weight in one f16, or in two 16-bit pieces: the first is cut off up to 2^-8 + 2^-7 (bf16) or 2^-10 + 2^-10 (f16)
        # below it, and the second's rounding is half a step (2^-8, 2^-11) of that
        piece = 2.0 ** -11 if self.cache == "fp8" and self.dtype == "bf16" else 2.0 ** -14 if self.dtype == "bf16" else 2.0 ** -20
        q = _np(self.q)
        for b, n in enumerate(self.lens):
            lo = max(0, n - window) if window else 0
            n = max(n, 0)
            want, bound, l, lb = ref.attend(q[b], self.k[b][lo:], self.v[b][lo:], scale, self.dtype, piece)
            err = np.abs(_np(out[b]) - want)
            assert (err <= bound).all(), (b, n, (err - bound).max())
            if lse is not None:
                got = _np(lse[b])
                assert np.array_equal(np.isneginf(got), np.isneginf(l))
                fine = np.isfinite(l)
                assert (np.abs(got[fine] - l[fine]) <= lb[fine]).all(), (b, n)
        assert lib.device_error() == 0


@pytest.fixture(params=["own choice", "list", "cluster 1", "cluster 2", "cluster 8"])
def way(lib, request):
    clib = lib.load()
    ways = {"own choice": 0, "list": 16, "cluster 1": 1, "cluster 2": 2, "cluster 8": 8}
    assert clib.w4a8_test_paged_attention_way(ways[request.param]) == 0
    yield request.param
    clib.w4a8_test_paged_attention_way(0)


LENS = [[1], [0], [17, -3, 1, 64, 65, 333, 15, 16], [5000], [130, 2000, 0, 0, 700]]


@pytest.mark.parametrize("lens", LENS, ids=["one", "none", "ragged", "long", "mixed"])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 1, 128), (12, 4, 128), (8, 8, 256), (34, 2, 64), (33, 1, 128),
                                      (64, 1, 128), (40, 1, 256), (6, 2, 80), (16, 1, 8), (7, 1, 136), (2, 2, 24)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_shapes(lib, way, lens, Hq, Hkv, D, dtype):
    c = Case(lens, Hq, Hkv, D, 16, dtype, seed=Hq + D)
    c.check(lib, *c.call(lib, return_lse=True))


@pytest.mark.parametrize("lens", LENS, ids=["one", "none", "ragged", "long", "mixed"])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 64), (8, 1, 128), (16, 1, 128), (36, 2, 128), (20, 1, 64), (9, 1, 256), (6, 2, 80),
                                      (2, 1, 16), (17, 1, 240)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_8_bit_caches(lib, way, lens, Hq, Hkv, D, dtype):
    c = Case(lens, Hq, Hkv, D, 16, dtype, "fp8", seed=Hq + D, scales=dtype == "bf16")
    c.check(lib, *c.call(lib, return_lse=True))


@pytest.mark.parametrize("page", [1, 3, 7, 16, 64, 100, 1024])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["plain", "heads first", "one allocation"])
def test_pages_and_layouts(lib, way, page, cache, layout):
    c = Case([99, 100, 1, 640, 1025], 10, 2, 128, page, "bf16", cache, layout, seed=page)
    c.check(lib, *c.call(lib, return_lse=True))


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 500, 2000])
@pytest.mark.parametrize("cache", ["f16", "fp8"])
def test_window(lib, way, window, cache):
    c = Case([1, 64, 333, 0, 1999], 6, 2, 64, 16, "f16", cache, seed=window)
    c.check(lib, *c.call(lib, return_lse=True, window=window), window=window)


@pytest.mark.parametrize("B", [2, 32, 33, 37, 130, 700, 1024, 1025, 2600])
def test_many_sequences(lib, way, B):
    c = Case([(37 * b) % 101 if B < 1000 else (37 * b) % 11 for b in range(B)], 4, 2, 64, 16, seed=B)
    c.check(lib, *c.call(lib, return_lse=True))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(lib, scale):
    c = Case([70, 3], 4, 1, 64, 16, spread=2.0)
    c.check(lib, *c.call(lib, return_lse=True, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")])
def test_sharp_rows(lib, way, dtype, cache):
    # scores of hundreds: a weight of 1 and others that vanish, maxima that rise from tile to tile
    c = Case([900, 40], 8, 1, 128, 16, dtype, cache, spread=8.0)
    c.check(lib, *c.call(lib, return_lse=True))


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_queries_of_any_size_of_exponent(lib, cache):
    # one row of the smallest, one of the largest queries
    c = Case([50], 4, 1, 64, 16, "bf16", cache)
    c.q[0, 0] *= 2.0 ** -120
    c.q[0, 1] *= 2.0 ** 60
    c.q[0, 2] *= 0
    out, lse = c.call(lib, return_lse=True, scale=1.0)
    want, bound, l, lb = ref.attend(_np(c.q)[0, [0, 2, 3]], c.k[0], c.v[0], 1.0, "bf16", 2.0 ** -11)
    rows = [0, 2, 3]
    assert (np.abs(_np(out)[0, rows] - want) <= bound).all()
    assert (np.abs(_np(lse)[0, rows] - l) <= lb).all()
    top = int(np.argmax(c.k[0][:, 0] @ _np(c.q)[0, 1]))  # scores of 2^60: one key has all the weight
    assert np.allclose(_np(out)[0, 1], c.v[0][top, 0], rtol=2.0 ** -8, atol=0)


def test_infinite_and_nan_keys(lib, way):
    c = Case([40, 40, 40, 40], 2, 1, 64, 16)
    c.q.fill_(1.0)

    def put(b, at, value):
        c.kc[c.table[b, at // 16].long(), at % 16] = value
    for t in range(40):
        put(1, t, -math.inf)  # every score is -inf: nothing is left of the row
    for t in range(20):
        put(2, t, -math.inf)  # the others have the weight
    put(3, 7, math.nan)
    out, lse = c.call(lib, return_lse=True)
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)
    want, bound, _, _ = ref.attend(_np(c.q)[2], c.k[2][20:], c.v[2][20:], 0.125, "bf16", 2.0 ** -14)
    assert (np.abs(_np(out[2]) - want) <= bound).all()
    assert torch.isnan(out[3]).all() and torch.isfinite(out[0].float()).all() and torch.isfinite(lse[0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_of_infinity_stay_in_their_column(lib, dtype):
    c = Case([33], 2, 1, 64, 16, dtype)
    c.vc[c.table[0, 1].long(), 3, 0, 5] = math.inf
    out = c.call(lib)
    assert torch.all(out[0, :, 5] == math.inf)
    keep = [i for i in range(64) if i != 5]
    assert torch.isfinite(out[0][:, keep].float()).all()


def test_strided_queries_and_outputs(lib, way):
    c = Case([100, 7, 300], 6, 2, 64, 16)
    rows = torch.randn((3, 6 * 64 + 2 * 2 * 64 + 3), device="cuda").to(torch.bfloat16)
    c.q = rows[:, 1:1 + 384].unflatten(1, (6, 64))  # part of a fused projection, no alignment
    buf = torch.full((3, 6, 70), 7.0, device="cuda").to(torch.bfloat16)
    out = buf[:, :, 3:67]
    got, lse = c.call(lib, return_lse=True, out=out)
    assert got is out
    c.check(lib, out, lse)
    assert torch.all(buf[:, :, :3] == 7.0) and torch.all(buf[:, :, 67:] == 7.0)


def test_given_workspace_holds_anything(lib, way):
    c = Case([7000, 0, 50], 16, 2, 128, 16)
    need = lib.paged_attention_workspace_bytes(3, 16, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    first = c.call(lib, ws=ws)
    c.check(lib, first, None)
    assert torch.equal(first, c.call(lib, ws=ws)) and torch.equal(first, c.call(lib))  # no atomics: the same bits
    if way in ("own choice", "list"):
        with pytest.raises(lib.W4A8Error, match="workspace"):
            c.call(lib, ws=ws[:need - 16])


def test_bad_pages_read_as_zeros(lib, way):
    # the kernel checks every page id before it reads: an error code, and outputs of the other sequences as before
    c = Case([40, 40, 100], 2, 1, 64, 16)
    want = c.call(lib)
    c.table[0, 1] = c.kc.shape[0]
    c.table[1, 0] = -7
    got = c.call(lib)
    assert lib.device_error() == 2 and lib.device_error() == 0
    assert torch.equal(got[2], want[2]) and torch.isfinite(got.float()).all()
    c.lens_t[2] = 16 * c.table.shape[1] + 1  # a position behind the table's last page
    c.table[:] = 0
    c.kc.nan_to_num_()
    c.vc.nan_to_num_()
    got = c.call(lib)
    assert lib.device_error() == 2 and torch.isfinite(got.float()).all()


def test_places_beyond_32_bits(lib):
    far = 2_200_000_000  # elements between two pages
    store = torch.zeros(far + 8192, dtype=torch.bfloat16, device="cuda")
    c = Case([30], 4, 1, 64, 16)
    for name, at in (("kc", 0), ("vc", 2048)):
        view = store[at:].as_strided((2, 16, 1, 64), (far, 64, 64, 1))
        old = getattr(c, name)
        view[1].copy_(old[c.table[0, 0].long()])
        view[0].copy_(old[c.table[0, 1].long()])
        setattr(c, name, view)
    c.table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    c.check(lib, *c.call(lib, return_lse=True))


def test_graphs_streams_and_changing_lengths(lib, way):
    # two captured graphs with a workspace each, replayed side by side, and lengths that change between replays
    cases = [Case([700, 900, 20], 8, 1, 128, 16, seed=s) for s in (1, 2)]
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.call(lib)
        out = torch.empty_like(c.q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.call(lib, out=out)
        outs.append(out)
        graphs.append(graph)
    for cut in (0, 5, 690, 699):
        for c in cases:
            c.lens = [700 - cut, max(0, 900 - 3 * cut), max(0, 20 - cut)]
            c.lens_t.copy_(torch.tensor(c.lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(5):
                    graph.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            k, v = c.k, c.v
            c.k, c.v = [x[:n] for x, n in zip(k, c.lens)], [x[:n] for x, n in zip(v, c.lens)]
            c.check(lib, out, None)
            c.k, c.v = k, v


def test_parts_join_to_the_whole(lib):
    # two halves of a context, joined by their lse, are the whole
    c = Case([640], 4, 2, 64, 16, "f16")
    whole, lse = c.call(lib, return_lse=True)
    c.lens_t.fill_(320)
    a, la = c.call(lib, return_lse=True)
    c.table = c.table[:, 20:].contiguous()
    b, lb = c.call(lib, return_lse=True)
    top = torch.maximum(la, lb)
    wa, wb = (la - top).exp(), (lb - top).exp()
    both = (a.float() * wa[..., None] + b.float() * wb[..., None]) / (wa + wb)[..., None]
    # each half is rounded to f16 (2^-11 of it), the whole too
    size = (a.float().abs() * wa[..., None] + b.float().abs() * wb[..., None]) / (wa + wb)[..., None] + whole.float().abs()
    assert torch.all((both - whole.float()).abs() <= 2.0 ** -11 * size * 1.1 + 1e-6)
    assert torch.all((top + (wa + wb).log() - lse).abs() <= 1e-5)


def test_a_table_without_pages(lib, way):
    c = Case([5, 0], 4, 2, 64, 16)
    out, lse = lib.paged_attention_decode(c.q, c.kc, c.vc, c.table[:, :0], c.lens_t, return_lse=True)
    assert lib.device_error() == 2 and torch.all(out == 0) and torch.all(lse == -math.inf)


def test_empty_batch(lib):
    c = Case([5], 4, 2, 64, 16)
    out, lse = lib.paged_attention_decode(c.q[:0], c.kc, c.vc, c.table[:0], c.lens_t[:0], return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_refusals(lib):
    c = Case([5, 6], 4, 2, 64, 16)
    base = dict(q=c.q, k_cache=c.kc, v_cache=c.vc, page_table=c.table, seq_lens=c.lens_t)
    odd = torch.zeros((4, 16, 2, 65), dtype=torch.bfloat16, device="cuda")
    f8 = torch.zeros((4, 16, 2, 24), device="cuda").to(torch.float8_e4m3fn)
    for change, err, msg in [
            (dict(q=c.q.float()), TypeError, "q must be"), (dict(q=c.q[0]), ValueError, "3 dimensions"),
            (dict(q=c.q.half()), TypeError, "k_cache"), (dict(q=c.q[:, :3]), lib.W4A8Error, "Hq=3"),
            (dict(q=c.q[:, :, :32]), ValueError, "elements"), (dict(q=c.q[:1]), ValueError, "page_table"),
            (dict(v_cache=c.vc[:1]), ValueError, "v_cache"), (dict(seq_lens=c.lens_t.long()), TypeError, "seq_lens"),
            (dict(page_table=c.table.long()), TypeError, "page_table"), (dict(window=-1), lib.W4A8Error, "window=-1"),
            (dict(scale=float("nan")), lib.W4A8Error, "finite"), (dict(k_scale=torch.ones(2, device="cuda")), lib.W4A8Error, "scales"),
            (dict(out=c.q[:1].expand(2, 4, 64)), ValueError, "overlapping"), (dict(out=c.q.half()), TypeError, "out"),
            (dict(ws=torch.empty(16, device="cuda")), TypeError, "ws"),
            (dict(k_cache=odd[..., 1:], v_cache=odd[..., 1:]), lib.W4A8Error, "multiples of 16 bytes"),
            (dict(q=c.q[:, :, :60].contiguous(), k_cache=odd[..., :60], v_cache=odd[..., :60]), lib.W4A8Error, "D=60"),
            (dict(q=c.q[:, :, :24].contiguous(), k_cache=f8, v_cache=f8), lib.W4A8Error, "D=24"),
            (dict(k_cache=c.kc.cpu()), TypeError, "CUDA")]:
        with pytest.raises(err, match=msg):
            lib.paged_attention_decode(**{**base, **change})
    assert lib.device_error() == 0


def _one_page(length, D=8, page=458766, pages=4681):
    # a table of 2^31 - 2 places, all in one page of a cache of 7 MB
    c = Case([1], 2, 1, D, 16)
    c.kc, c.vc = (torch.zeros((1, page, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    c.lens_t.fill_(length)
    return c


@pytest.mark.parametrize("length", [2 ** 31 - 2, 2 ** 31 - 3, 2 ** 31 - 18, 2 ** 31 - 34])
@pytest.mark.parametrize("window", [1, 7, 40, 5000])
def test_a_window_at_the_end_of_the_longest_table(lib, way, length, window):
    # the last tile ends behind 2^31
    c = _one_page(length)
    g = torch.Generator("cuda").manual_seed(window)
    at = torch.arange(length - window, length, device="cuda") % 458766
    for t in (c.kc, c.vc):
        t.fill_(math.nan)
        t[0, at] = torch.randn((window, 1, 8), device="cuda", generator=g).to(torch.bfloat16)
    out, lse = c.call(lib, return_lse=True, window=window)
    k, v = (_np(t)[0, at.cpu().numpy()] for t in (c.kc, c.vc))
    want, bound, l, lb = ref.attend(_np(c.q)[0], k, v, 8 ** -0.5, "bf16", 2.0 ** -14)
    assert (np.abs(_np(out)[0] - want) <= bound).all() and (np.abs(_np(lse)[0] - l) <= lb).all()
    assert lib.device_error() == 0


@pytest.mark.parametrize("length", [2 ** 31 - 2, 2 ** 31 - 20])
def test_a_sequence_as_long_as_the_longest_table(lib, length):
    # scores of 0: the sum of the weights is the length.  Each of up to 8 * 152 warps adds up whole numbers below 2^24, exact;
    # their sums are joined with a rounding each, and the logarithm is within a few units of 21.5
    c = _one_page(length)
    c.vc.fill_(1.0)
    out, lse = c.call(lib, return_lse=True)
    runs = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    assert 2 ** 31 / runs < 2 ** 24
    assert (np.abs(_np(lse) - math.log(length)) <= (runs + 64) * ref.U + 4 * 22 * ref.U).all()
    # a warp's sum of values is cut off by up to a unit (2 u) at each of two additions of 16 weights' pieces
    assert (np.abs(_np(out) - 1.0) <= 2 * (2 ** 31 / runs / 16 + 64) * 2 * ref.U + 2.0 ** -8).all()
    assert lib.device_error() == 0


def test_empty_rows_of_more_than_31_bits_of_outputs(lib):
    # 2^23 heads of 256 for one sequence, all of them zeros
    Hq, Hkv, D = 1 << 23, 1 << 15, 256
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda").expand(1, Hq, D)
    cache = torch.zeros((1, 1, Hkv, D), dtype=torch.bfloat16, device="cuda")
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 1), (1,)))
    out = torch.full((1, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = lib.paged_attention_decode(q, cache, cache, table, lens, return_lse=True, out=out)
    assert int(torch.count_nonzero(out)) == 0 and torch.all(lse == -math.inf) and lib.device_error() == 0


@pytest.mark.parametrize("window", [0, 1, 30, 57, 60, 96, 200, 2 ** 31 - 1, 2 ** 40])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_positions_behind_the_table_are_left_out(lib, way, window, cache):
    # lengths of up to 40 more than the tables have places for: what is there counts, in a window before the length
    places = 96
    c = Case([places, places, 40, places, 0], 6, 2, 64, 16, "bf16", cache, seed=5)
    over = [places + 1, places + 40, 40, places, 0]
    c.lens_t.copy_(torch.tensor(over, dtype=torch.int32))
    table = c.table[:, :places // 16].contiguous()
    out, lse = lib.paged_attention_decode(c.q, c.kc, c.vc, table, c.lens_t, k_scale=c.ks, v_scale=c.vs, window=window,
                                          return_lse=True)
    assert lib.device_error() == 2 and lib.device_error() == 0
    q, piece = _np(c.q), 2.0 ** -11 if cache == "fp8" else 2.0 ** -14
    for b, n in enumerate(over):
        lo = max(0, n - window) if window else 0
        want, bound, l, lb = ref.attend(q[b], c.k[b][lo:], c.v[b][lo:], 0.125, "bf16", piece)
        assert (np.abs(_np(out[b]) - want) <= bound).all(), b
        got, fine = _np(lse[b]), np.isfinite(l)
        assert np.array_equal(np.isneginf(got), np.isneginf(l)) and (np.abs(got[fine] - l[fine]) <= lb[fine]).all(), b


@pytest.mark.parametrize("Hq,Hkv,D", [(65, 1, 64), (100, 1, 128), (256, 1, 128), (512, 2, 64), (130, 1, 256), (256, 1, 256)])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")])
def test_up_to_256_heads_to_a_key_value_head(lib, way, Hq, Hkv, D, dtype, cache):
    c = Case([1, 700, 0, 33, 129], Hq, Hkv, D, 16, dtype, cache, seed=Hq + D)
    c.check(lib, *c.call(lib, return_lse=True))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 500, 1998, 2000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_window_over_bf16(lib, way, window, D):
    c = Case([1, 64, 333, 0, 1999], 6, 2, D, 16, "bf16", seed=window)
    c.check(lib, *c.call(lib, return_lse=True, window=window), window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [33, 400])
def test_values_of_infinity_each_way(lib, way, dtype, n):
    # one of each sign in columns of their own: infinite there, the other columns as without them
    c = Case([n, 7], 20, 1, 64, 16, dtype)
    want = c.call(lib)
    c.vc[c.table[0, 1].long(), 3, 0, 5] = math.inf
    c.vc[c.table[0, 0].long(), 9, 0, 60] = -math.inf
    out = c.call(lib)
    assert torch.all(out[0, :, 5] == math.inf) and torch.all(out[0, :, 60] == -math.inf)
    keep = [i for i in range(64) if i not in (5, 60)]
    assert torch.equal(out[0][:, keep], want[0][:, keep]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (40, 1, 128), (40, 1, 256)])
def test_outputs_over_the_queries(lib, way, dtype, cache, Hq, Hkv, D):
    c = Case([2000, 0, 1, 90, 300], Hq, Hkv, D, 16, dtype, cache, seed=D)
    want, lse = c.call(lib, return_lse=True)
    c.check(lib, want, lse)
    rows = torch.randn((5, Hq + 3, D + 8), device="cuda").to(DT[dtype])
    for q in (c.q.clone(), rows[:, 1:1 + Hq, 8:]):  # by themselves, and part of other rows
        q.copy_(c.q)
        got = lib.paged_attention_decode(q, c.kc, c.vc, c.table, c.lens_t, k_scale=c.ks, v_scale=c.vs, out=q)
        assert got is q and torch.equal(q, want)
    assert lib.device_error() == 0
