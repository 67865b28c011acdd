"""The paged cache and its attention on the GPU against the definition in 64 bits (cache_ref)."""
import gc

import pytest
import torch

import cache_ref
from titans_long_term_b200 import PagedCache, TitansError, mem

pytestmark = pytest.mark.gpu


class Pool:
    """A cache of B sequences, its pages scattered and filled, and what every position holds."""

    def __init__(self, B, H, Hkv, d, dtype, page, S, seed=0, fill=None):
        G = torch.Generator().manual_seed(seed)
        most = -(-S // page)
        self.S, self.B, self.Hkv, self.d, self.page = S, B, Hkv, d, page
        self.cache = PagedCache(d, dtype, B, H, kv_heads=Hkv, page=page, num_pages=B * most + 2, max_pages=most)
        self.pages = self.cache.new_pages()
        self.table = torch.randperm(B * most + 2, generator=G)[: B * most].to(torch.int32).reshape(B, most).cuda()
        self.k, self.v = (torch.randn(B, Hkv, S, d, generator=G).to(torch.bfloat16).cuda() for _ in range(2))
        self.q = lambda T: torch.randn(B, H, T, d, generator=G).to(torch.bfloat16).cuda()  # noqa: E731
        zero = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.cache.append(self.k, self.v, self.pages, self.table, zero)
        if dtype == "e4m3":
            self.k, self.v = cache_ref.quantise(self.k), cache_ref.quantise(self.v)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,Hkv,d,page,T", [(1, 1, 64, 16, 1), (3, 2, 128, 64, 100), (2, 5, 64, 128, 333), (4, 1, 128, 32, 31)])
def test_append_and_read(B, Hkv, d, page, T, dtype):
    p = Pool(B, Hkv, Hkv, d, dtype, page, 400, seed=T)
    before = {n: t.clone() for n, t in p.pages.items()}
    starts, counts = ints(*[7 * b for b in range(B)]), ints(*[max(0, T - 40 * b) for b in range(B)])
    G = torch.Generator().manual_seed(1)
    k, v = (torch.randn(B, Hkv, T, d, generator=G).to(torch.bfloat16).cuda() for _ in range(2))
    k[0, 0, 0] *= 1e30
    v[0, 0, 0] *= 1e-30
    k[-1, -1, 0] = 0
    k[0, 0, -1, 0] = 448 * 4  # a scale's very edge
    p.cache.append(k, v, p.pages, p.table, starts, counts=counts)
    gk, gv = p.cache.read(p.pages, p.table, starts, T, counts=counts)
    for got, x in ((gk, k), (gv, v)):
        for b in range(B):
            n = int(counts[b])
            want = x[b, :, :n].double() if dtype == "bf16" else cache_ref.quantise(x[b, :, :n])
            assert torch.equal(got[b, :, :n].double(), want)
            assert (got[b, :, n:] == 0).all()
    # nothing else moved: put the old rows back and compare the pool
    for b in range(B):
        for t in range(int(counts[b])):
            at = int(starts[b]) + t
            i = (int(p.table[b, at // page]), slice(None), at % page)
            for n in p.pages:
                new, old = (z.view(torch.uint8) if z.dtype == torch.float8_e4m3fn else z for z in (p.pages[n], before[n]))
                new[i] = old[i]
    for n in p.pages:
        new, old = (z.view(torch.uint8) if z.dtype == torch.float8_e4m3fn else z for z in (p.pages[n], before[n]))
        assert torch.equal(new, old), n
    p.cache.sync_status()


def test_quantised_specials():
    """Infinities become the largest value, NaN stays, neither sets the scale; all zeros and tiny rows are exact."""
    p = Pool(1, 1, 1, 64, "e4m3", 16, 16)
    k = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0, :3] = torch.tensor([float("inf"), -float("inf"), 2.0])
    k[0, 0, 1, :2] = torch.tensor([float("nan"), 1.0])
    k[0, 0, 3, 0] = 2.0**-126
    p.cache.append(k, k, p.pages, p.table, ints(0))
    got, _ = p.cache.read(p.pages, p.table, ints(0), 4)
    got = got[0, 0].double()
    assert got[0, 0] == 448 * 2.0**-7 and got[0, 1] == -448 * 2.0**-7 and got[0, 2] == 2
    assert got[1, 0].isnan() and got[1, 1] == 1 and (got[2] == 0).all() and got[3, 0] == 2.0**-126


def check(p, T, starts, counts=None, window=0, sinks=0, missing=None, scale=None, bad=False):
    q = p.q(T)
    o = p.cache.attend(q, p.pages, p.table, starts, counts=counts, window=window, sinks=sinks, scale=scale)
    if bad:
        with pytest.raises(TitansError):
            p.cache.sync_status()
    p.cache.sync_status()
    n = torch.full((p.B,), T) if counts is None else counts.clamp(0, T)
    want = cache_ref.attend(q, p.k, p.v, starts, n, window, sinks, scale, missing)
    assert torch.isfinite(o).all()
    off = (o.double() - want).abs() / cache_ref.bar(want, p.v)
    assert off.max() <= 1, float(off.max())
    for b in range(p.B):
        assert (o[b, :, int(n[b]):] == 0).all()
    return o


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,H,Hkv,d,page,S,T", [
    (1, 1, 1, 64, 16, 1, 1), (2, 4, 4, 128, 16, 40, 1), (3, 6, 2, 64, 32, 300, 7), (1, 4, 1, 128, 64, 700, 130),
    (2, 3, 3, 64, 128, 513, 65), (1, 8, 2, 128, 16, 257, 257), (1, 20, 1, 64, 64, 1500, 3), (1, 2, 2, 128, 64, 2100, 33),
    (2, 12, 1, 128, 16, 500, 1), (300, 4, 2, 64, 32, 150, 7), (3, 8, 2, 128, 128, 9000, 2)])
def test_attend(B, H, Hkv, d, page, S, T, dtype):
    p = Pool(B, H, Hkv, d, dtype, page, S, seed=S)
    check(p, T, ints(*[max(0, S - T - (b * (S - T)) // 3) for b in range(B)]))


@pytest.mark.parametrize("T", [1, 7, 40])
def test_attend_few_keys_of_a_long_table(T):
    """Fewer blocks of keys than the table has room for, sequences of one key, and one whose first queries stand before 0."""
    p = Pool(5, 4, 2, 64, "bf16", 32, 3000, seed=T)
    check(p, T, ints(150, 0, 33, -3, 90))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,window,sinks", [(1, 1, 0), (7, 90, 20), (6, 1, 0), (1, 100, 4), (90, 17, 0), (90, 64, 16), (200, 150, 300), (200, 1, 1), (33, 5000, 9)])
def test_attend_window(T, window, sinks, dtype):
    p = Pool(2, 4, 2, 64, dtype, 16, 400, seed=T)
    check(p, T, ints(400 - T, 5), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,window,sinks,ragged", [(64, 0, 0, True), (128, 0, 0, False), (128, 200, 20, True), (64, 300, 0, False)])
def test_attend_many_rows(d, window, sinks, ragged, dtype):
    """Enough rows for two tiles of them a CTA."""
    p = Pool(4, 12, 6, d, dtype, 32, 900, seed=d)
    check(p, 560, ints(340, 0, 100, 7), counts=ints(560, 1, 300, 0) if ragged else None, window=window, sinks=sinks)


@pytest.mark.parametrize("T", [1, 6, 50, 300])
def test_attend_padded_batch(T):
    """Counts of 0, 1, T and one beyond T; sequences that hold nothing yet."""
    p = Pool(4, 4, 2, 128, "bf16", 32, 600, seed=T)
    check(p, T, ints(0, 3, 600 - T, 250), counts=ints(0, 1, T + 5, T))


@pytest.mark.parametrize("T", [1, 140])
def test_attend_ignores_what_it_does_not_see(T):
    """NaN and infinities behind the last token, in later tokens of the chunk and before the window reach no row that
    does not see them."""
    p = Pool(2, 2, 1, 64, "bf16", 16, 500, seed=T)
    starts = ints(300, 100)
    clean_k, clean_v = p.k, p.v
    k, v = p.k.clone(), p.v.clone()
    for b, s in enumerate(starts.tolist()):
        k[b, :, s + T:], v[b, :, s + T:] = float("nan"), float("inf")
        v[b, :, : s - 64] = float("nan")  # before every row's window
        if T > 1:  # a later token of the chunk: the rows from there on see it and are NaN
            v[b, :, s + 77] = float("nan")
            k[b, :, s + 99] = float("inf")
    p.cache.append(k, v, p.pages, p.table, ints(0, 0))
    q = p.q(T)
    o = p.cache.attend(q, p.pages, p.table, starts, window=64)
    want = cache_ref.attend(q, clean_k, clean_v, starts, [T, T], 64)
    n = 77 if T > 1 else T
    off = (o.double() - want).abs()[:, :, :n] / cache_ref.bar(want, clean_v)[:, :, :n]
    assert off.max() <= 1
    if T > 1:
        assert o[:, :, 77].isnan().all()
    p.cache.sync_status()


@pytest.mark.parametrize("T", [1, 60])
def test_missing_pages(T):
    """Table entries outside the pool are recorded, seen by no row and written by no token; entries that no row's
    window needs are not looked at."""
    p = Pool(2, 2, 2, 64, "bf16", 16, 320, seed=T)
    kept = p.table.clone()
    p.table[0, 3], p.table[1, 5] = -1, 1 << 20
    missing = torch.zeros(2, 320, dtype=torch.bool, device="cuda")
    missing[0, 48:64] = missing[1, 80:96] = True
    check(p, T, ints(200, 200), missing=missing, bad=True)
    check(p, T, ints(200, 200), window=70)
    before = p.pages["k"].clone()
    x = torch.ones(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    p.cache.append(x, x, p.pages, p.table, ints(48, 80))
    with pytest.raises(TitansError) as e:
        p.cache.sync_status()
    assert e.value.status == mem.EDEVICE
    assert torch.equal(before, p.pages["k"])
    p.cache.append(x, x, p.pages, kept, ints(310, 320))  # over the table's end
    with pytest.raises(TitansError):
        p.cache.sync_status()
    k, _ = p.cache.read(p.pages, p.table, ints(40, 72), 32)
    with pytest.raises(TitansError):
        p.cache.sync_status()
    assert (k[:, :, 8:24] == 0).all() and (k[:, :, :8] != 0).any()


def test_large_scores():
    p = Pool(1, 2, 2, 64, "bf16", 16, 300, seed=2)
    check(p, 40, ints(260), scale=30.0)
    check(p, 1, ints(299), scale=-30.0)
    check(p, 40, ints(260), scale=0.0)


def test_shared_pages():
    """Two sequences on the same pages (a common prefix) read the same keys."""
    p = Pool(2, 2, 2, 64, "bf16", 16, 200, seed=3)
    p.table[1] = p.table[0]
    p.k[1], p.v[1] = p.k[0], p.v[0]
    check(p, 20, ints(180, 100))


def test_other_stream_and_graph():
    p = Pool(2, 4, 2, 128, "e4m3", 64, 700, seed=4)
    starts = ints(650, 300)
    q = p.q(50)
    o = p.cache.attend(q, p.pages, p.table, starts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o1 = p.cache.attend(q, p.pages, p.table, starts, o=torch.empty_like(q), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, o1)
    gc.collect()  # handles of other memories that are still waiting to be collected would end the capture
    graph = torch.cuda.CUDAGraph()
    z = q.clone()
    with torch.cuda.graph(graph):
        o2 = p.cache.attend(z, p.pages, p.table, starts)
    for other in (p.q(50), q):
        z.copy_(other)
        graph.replay()
        assert torch.equal(o2, p.cache.attend(other, p.pages, p.table, starts))
    starts.copy_(ints(100, 0))  # the captured call reads where the sequences stand when it runs
    graph.replay()
    assert torch.equal(o2, p.cache.attend(q, p.pages, p.table, starts))


def test_a_handle_may_go_while_a_graph_is_captured():
    p, other = (Pool(1, 2, 2, 64, "bf16", 16, 64, seed=i) for i in range(2))
    q, starts = p.q(2), ints(60)
    want = p.cache.attend(q, p.pages, p.table, starts)
    gc.collect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.cache.close()
        o = p.cache.attend(q, p.pages, p.table, starts)
    graph.replay()
    assert torch.equal(o, want)


def test_binding_refuses_tensors():
    p = Pool(2, 4, 2, 64, "e4m3", 16, 64)
    q, starts = p.q(3), ints(0, 0)
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(table=p.table.long()), dict(starts=starts.long()),
                dict(pages={**p.pages, "k": p.pages["k"].view(torch.uint8)}), dict(starts=starts.cpu()),
                dict(counts=starts[:1])):
        args = {**dict(q=q, pages=p.pages, table=p.table, starts=starts), **bad}
        with pytest.raises(ValueError):
            p.cache.attend(**args)
    for bad in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan"))):
        with pytest.raises(TitansError) as e:
            p.cache.attend(q, p.pages, p.table, starts, **bad)
        assert e.value.status == mem.EINVAL
    with pytest.raises(ValueError):
        p.cache.read(p.pages, p.table, starts, 0)


@pytest.mark.parametrize("T", [1, 40])
def test_positions_behind_the_table(T):
    """Queries that stand behind the table's last position see what it has room for, and that is recorded."""
    p = Pool(2, 4, 2, 64, "bf16", 32, 320, seed=T)
    q = p.q(T)
    o = p.cache.attend(q, p.pages, p.table, ints(310, (1 << 31) - 1))
    with pytest.raises(TitansError):
        p.cache.sync_status()
    k, v = (torch.cat([x, x.new_zeros(2, 2, 70, 64)], 2) for x in (p.k, p.v))
    missing = torch.zeros(2, 390, dtype=torch.bool, device="cuda")
    missing[:, 320:] = True
    want = cache_ref.attend(q, k, v, [310, 350], [T, T], missing=missing)
    assert ((o.double() - want).abs() / cache_ref.bar(want, p.v)).max() <= 1
    o = p.cache.attend(q, p.pages, p.table, ints((1 << 31) - 1, 0), window=50)
    with pytest.raises(TitansError):
        p.cache.sync_status()
    assert (o[0] == 0).all() and (o[1] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,H,counts", [(6, 1, [3]), (4, 4, [1]), (2, 2, [0])])
def test_attend_padded_rows_of_a_split_sequence(T, H, counts, dtype):
    """Keys of one head shared out over several CTAs, whose parts are joined: the rows behind the count are zeros still."""
    p = Pool(1, H, 1, 64, dtype, 64, 4000, seed=T)
    check(p, T, ints(4000 - T), counts=ints(*counts))


def test_attend_refuses_what_an_int_or_float_cannot_hold():
    p = Pool(1, 2, 2, 64, "bf16", 16, 64)
    q, starts = p.q(3), ints(0)
    for bad in (dict(window=1 << 31), dict(window=(1 << 32) + 5), dict(sinks=1 << 32)):
        with pytest.raises(ValueError):
            p.cache.attend(q, p.pages, p.table, starts, **bad)
    for scale in (2.0**101, -(2.0**120), float("inf")):
        with pytest.raises(TitansError) as e:
            p.cache.attend(q, p.pages, p.table, starts, scale=scale)
        assert e.value.status == mem.EINVAL
    most = (1 << 31) - 1
    check(p, 3, ints(50), window=most, sinks=most)


def test_attend_many_short_sequences():
    """More sequences than a warp has lanes, more rows than the kernel for few of them takes, of unlike lengths."""
    p = Pool(40, 2, 1, 64, "bf16", 16, 100, seed=9)
    check(p, 20, ints(*[(7 * b) % 81 for b in range(40)]), counts=ints(*[20 - b % 3 for b in range(40)]))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,window,count", [(64, 0, 256), (128, 900, 131)])
def test_attend_split_keys_of_two_tiles(d, window, count, dtype):
    """Two tiles of rows a CTA and keys shared out over several CTAs at once; rows behind the count in some of them."""
    p = Pool(1, 8, 2, d, dtype, 64, 8000, seed=d)
    check(p, 256, ints(7744), counts=ints(count), window=window, sinks=30 if window else 0)
