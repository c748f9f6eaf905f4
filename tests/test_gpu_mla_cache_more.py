"""The 4-bit cache of latents and what works on it, further: the precision of split queries, weights over missing
pages, page offsets past 2^32 bytes for the weights of either form and for eviction, and what eviction moves when it is
replayed; outputs in place and apart, calls replayed from a graph, shared queries."""
import math
import re

import pytest
import torch

import gated_delta_rule_chunk_amd as kda
from tests import mla_cache_ref as ref
from tests import mla_ref
from tests.test_gpu_mla_cache import (BF16, F32, _cache, _evict_and_check, _i32, _limits, _queries, _rows_of_queries,
                                      _weights)
from tests.test_mla_split_host import HEADER, stated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,call", [(128, "step"), (16, "step"), (128, "weigh"), (256, "weigh")])
def test_split_queries(H, call):
    """One key, 2^K in the channel of x: the score is x 2^K, with nothing to add to it. x has every significand, from
    2^-7 of the block's largest down, for largest ones at either end of their exponent."""
    exact, loss, tiny, least = stated()
    tops = [-133, -126, -120, -112, -111, -60, 0, 100]
    cases = [(t, big, d) for t in tops for big in (1.0, 1.9921875) for d in range(7, 25) if t >= -126 or big == 1.0]
    Nb, Dc, page = len(cases), 256, 16
    j = torch.arange(H, device="cuda")
    ql = torch.zeros(Nb, 1, H, Dc, dtype=BF16, device="cuda")
    codes = torch.zeros(Nb, Dc, dtype=torch.uint8)
    scales = torch.full((Nb, Dc // 32), 127, dtype=torch.uint8)
    want, bound = [], []
    for b, (t, big, d) in enumerate(cases):
        block, at = b % 8, 32 * (b % 8) + (5 * b) % 32
        L = (torch.tensor(big) * 2.0 ** t).to(BF16).item()
        sign = 1 - 2 * (j % 2).double()
        x = (sign * (1 + (j * max(1, 128 // H) % 128) / 128) * 2.0 ** max(t - d, -200)).to(BF16)
        ql[b, 0, :, 32 * block + (5 * b + 7 + b % 3) % 32] = L
        ql[b, 0, :, at] = x
        K = max(-100, min(125, d - t))
        codes[b, at] = 2
        scales[b, at // 32] = 127 + K
        v = x.double()
        off = torch.full_like(v, least) if L < tiny else torch.where(v.abs() >= exact * L, 0.0, loss * L)
        want.append(v * 2.0 ** K)
        bound.append(off * 2.0 ** K)
    want, bound = torch.stack(want), torch.stack(bound)
    cache = kda.mla_cache_mx(Nb, page, Dc, 0, BF16)
    for b in range(Nb):
        ref.put_page(cache, b, codes[b:b + 1].cuda(), scales[b:b + 1].cuda(), None)
    table, n = _i32([[b] for b in range(Nb)]), _i32([1] * Nb)
    if call == "step":
        # lse is the score in base 2 and back: three roundings, and of the scale
        o, lse = kda.mla_step_mx(ql, None, cache, table, n, 1.0)
        assert bool(((lse[:, 0].double() - want).abs() <= bound + 6 * mla_ref.H32 * want.abs() + 2.0 ** -140).all())
    else:
        # exp(x 2^K - 0), summed over the heads: one head's share is seen by giving the others an lse of infinity
        for h in range(0, H, 37):
            lse = torch.full((Nb, 1, H), math.inf, device="cuda")
            lse[:, 0, h] = 0
            w = kda.mla_weigh(ql, None, cache, table, n, lse, 1.0, torch.zeros(Nb, page, device="cuda"))[:, 0].double()
            off = bound[:, h] + 8 * mla_ref.H32 * (1 + want[:, h].abs())
            assert bool(((w - want[:, h].exp()).abs() <= want[:, h].exp() * torch.expm1(off)).all()), h


# page size, lengths, missing pages by sequence: in the first and in the second tile of a pair, whole tiles, quarters,
# one behind another, the last page, the first; past the 64 pages of a window
HOLES = [
    (16, [1100, 300, 64, 45], [[1, 4, 5, 6, 7, 20, 66], [0, 18], [3], [2]]),
    (32, [700, 190, 33], [[1, 2, 3, 21], [0, 4], [1]]),
    (64, [520, 64, 129], [[0, 3, 4], [0], [2]]),
    (128, [600, 250], [[1, 3], [0]]),
]


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,T", [(8, 1), (48, 1), (100, 1), (130, 1), (50, 3), (5, 4)])
@pytest.mark.parametrize("page,lens,holes", HOLES)
def test_weights_and_attention_over_missing_pages(mx, dtype, H, T, page, lens, holes):
    """Every number of rows of queries that has a kernel of its own: what exists gets its weight, what does not keeps
    the old one, decayed; each missing page is counted once."""
    scale = 0.07
    cache, table, rows = _cache(lens, page, 512, 64, dtype, H + T, mx=mx)
    ql, qr = _queries(len(lens), T, H, 512, 64, dtype, 9)
    bad = table.clone()
    for b, gone in enumerate(holes):
        for i, p in enumerate(gone):
            bad[b, p] = -1 if i % 2 else cache.shape[0] + i
    count = f"{sum(len(x) for x in holes)} counted"
    n = _i32(lens)
    o, lse = (kda.mla_step_mx if mx else kda.mla_step)(ql, qr, cache, bad, n, scale=scale)
    with pytest.raises(kda.KDAError, match=count):
        kda.device_check()
    g = torch.Generator(device="cuda").manual_seed(10)
    old = torch.rand((len(lens), table.shape[1] * page), generator=g, device="cuda")
    out = torch.full_like(old, 7.0)
    kda.mla_weigh(ql, qr, cache, bad, n, lse, scale, old, fresh=0, decay=0.5, out=out)
    with pytest.raises(kda.KDAError, match=count):
        kda.device_check()
    for b, L in enumerate(lens):
        j = torch.arange(L, device="cuda")
        there = ~torch.isin(j // page, torch.tensor(holes[b], device="cuda"))
        at = j[there]
        c, r = rows[b][0][at], rows[b][1][at]
        limit = (at[None] < _limits(L, T, H, L)[:, None]).sum(1)
        q = _rows_of_queries(ql, qr, b)
        res = ref.attend(q, c, r, scale, limit, dtype, mx)
        mla_ref.check(f"o[{b}]", o[b].reshape(1, T * H, 512), res["o"])
        mla_ref.check(f"lse[{b}]", lse[b].reshape(1, T * H), res["lse"])
        w = ref.gathered(q, c, r, lse[b].flatten(), scale, limit, old[b, at], 0.5, dtype, mx)
        mla_ref.check(f"weights[{b}]", out[b, at], w)
        assert torch.equal(out[b, :L][~there], 0.5 * old[b, :L][~there]) and bool((out[b, L:] == 7).all())


@pytest.mark.parametrize("mx,dtype,n_pages", [(True, BF16, 43000), (True, F32, 32500), (False, BF16, 14700), (False, F32, 7400)])
def test_weights_and_eviction_past_four_gib(mx, dtype, n_pages):
    """All pages that are used lie past 2^32 bytes: what is moved, from there to there, and what is weighed."""
    page, lens = 256, [1400, 45, 900]
    cache, table, rows = _cache(lens, page, 512, 64, dtype, 6, mx=mx, n_pages=n_pages)
    used = table[table >= 0]
    assert int(used.min()) * page * cache.shape[2] * cache.element_size() > 1 << 32
    for H in (8, 130):
        ql, qr = _queries(3, 1, H, 512, 64, dtype, 7)
        lse = (kda.mla_step_mx if mx else kda.mla_step)(ql, qr, cache, table, _i32(lens), 0.07)[1]
        w = torch.zeros(3, table.shape[1] * page, device="cuda")
        kda.mla_weigh(ql, qr, cache, table, _i32(lens), lse, 0.07, w)
        for b, (c, r) in enumerate(rows):
            q, L = _rows_of_queries(ql, qr, b), lens[b]
            mla_ref.check(f"weights[{b}]", w[b, :L], ref.gathered(q, c, r, lse[b].flatten(), 0.07, _limits(L, 1, H, L),
                                                                  torch.zeros(L, device="cuda"), 1.0, dtype, mx))
    # (NaN rows are behind the lengths and in pages that nobody has: compared as bytes)
    g = torch.Generator(device="cuda").manual_seed(8)
    _evict_and_check(cache, table, _i32(lens), _weights(g, 3, table.shape[1] * page), 300, 3, 100, True)


@pytest.mark.parametrize("form", ["mx", "rows"])
@pytest.mark.parametrize("cap", [16384, 40000])
def test_what_eviction_moves_when_replayed(cap, form):
    """Captured once, replayed with other weights, lengths and page tables: rows, page table, lengths and weights, by
    one launch that decides and by several."""
    page, N, keep, first, recent = 16, 3, 4000, 5, 100
    g = torch.Generator(device="cuda").manual_seed(78)
    pages = N * cap // page
    if form == "mx":
        make = lambda: torch.randint(0, 256, (pages, page, 136), dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    else:
        make = lambda: torch.randn((pages, page, 256), device="cuda", generator=g).to(BF16)  # noqa: E731
    shuffled = lambda: torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(N, -1)  # noqa: E731
    cache, table, n, w = make(), shuffled(), _i32([cap, 9000, 100]), _weights(g, N, cap)
    out = torch.empty_like(table), torch.empty_like(n), torch.empty_like(w)
    ws = torch.empty(kda.mla_evict_workspace_bytes(N, page, cap // page), dtype=torch.uint8, device="cuda")

    def call():
        kda.mla_evict(cache, table, n, w, keep, first=first, recent=recent, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    parts = ((0, 128), (128, 8)) if form == "mx" else ((0, 512),)       # a row's bytes in a page of 16

    def bytes_of(x):                                                     # by rows
        x = x.view(torch.uint8).view(pages, -1)
        return torch.cat([x[:, at * page:(at + k) * page].reshape(pages * page, k) for at, k in parts], 1)

    moved = 0
    for i in range(4):
        cache.copy_(make())
        table.copy_(shuffled())
        n.copy_(_i32([cap - 1000 * i, 9000 - 1700 * i, 5000 * (i % 2)]))
        w.copy_(_weights(g, N, cap))
        for x in out:
            x.fill_(-5)
        want, t0 = bytes_of(cache).clone(), table.tolist()
        before = want.clone()
        graph.replay()
        if i % 2:
            torch.cuda.synchronize()
        for b, L in enumerate(n.tolist()):
            E, a, e, moves, order = ref.evict(w[b, :L].tolist(), L, page, keep, first, recent)
            t, used = t0[b], -(-L // page)
            assert out[0][b].tolist() == (t[:e - E] + t[e:used] + t[e - E:e] + t[used:] if E else t)
            ww = torch.cat((w[b].cpu()[order], torch.zeros(E * page), w[b, L:].cpu()))
            assert out[1][b].item() == L - E * page and torch.equal(out[2][b].cpu(), ww)
            if moves:
                to, src = (torch.tensor([t[j // page] * page + j % page for j in x], device="cuda") for x in zip(*moves))
                want[to] = before[src]
                moved += len(moves)
        assert torch.equal(bytes_of(cache), want)
        assert table.tolist() == t0
    assert moved > 10000


@pytest.mark.parametrize("apart", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 0, 1), (1, 1, 0)])
@pytest.mark.parametrize("cap", [16384, 40000])
def test_evict_some_in_place_some_apart(cap, apart):
    """Page table, lengths and weights, each in place or apart, give what all in place give."""
    page, lens = 16, [12000, 700, -3, 4097, cap]
    g = torch.Generator(device="cuda").manual_seed(79)
    pages = len(lens) * cap // page
    cache = torch.randint(0, 256, (pages, page, 136), dtype=torch.uint8, device="cuda", generator=g)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(len(lens), -1)
    state = table, _i32(lens), _weights(g, len(lens), cap)
    first, mine = cache.clone(), [x.clone() for x in state]
    want = kda.mla_evict(first, *mine, 3000, first=20, recent=500)
    out = tuple(torch.full_like(x, -9) if a else x for x, a in zip(state, apart))
    kept = [x.clone() for x in state]
    got = kda.mla_evict(cache, *state, 3000, first=20, recent=500, out=out)
    assert torch.equal(cache, first)
    for x, y, o, s, k, a in zip(got, want, out, state, kept, apart):
        assert x is o and torch.equal(x, y)
        assert not a or torch.equal(s, k)


@pytest.mark.parametrize("mx,dtype,Dc,H,T", [(True, BF16, 512, 12, 1), (True, BF16, 512, 40, 4), (False, BF16, 256, 40, 4),
                                             (False, BF16, 512, 100, 1), (True, F32, 256, 12, 1), (False, F32, 512, 40, 2)])
def test_write_read_attention_and_weights_replayed(mx, dtype, Dc, H, T):
    """Captured once, replayed with other lengths, queries and new rows: what the same calls give eagerly."""
    page, N, room = 16, 3, 30
    g = torch.Generator(device="cuda").manual_seed(95)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    table = torch.randperm(N * room, generator=g, device="cuda").to(torch.int32).view(N, room)
    cache = kda.mla_cache_mx(N * room, page, Dc, 64, dtype) if mx else torch.zeros((N * room, page, Dc + 64), dtype=dtype, device="cuda")
    append, step = (kda.mla_cache_append_mx, kda.mla_step_mx) if mx else (kda.mla_cache_append, kda.mla_step)
    append(rand(N, 400, Dc), rand(N, 400, 64), cache, table, _i32([0] * N))
    s = {"cache": cache, "n": _i32([0] * N), "c": rand(N, T, Dc), "r": rand(N, T, 64), "ql": rand(N, T, H, Dc),
         "qr": rand(N, T, H, 64), "w": torch.zeros(N, room * page, device="cuda")}
    cu = _i32([0, 30, 30, 75])

    def call(s):
        append(s["c"], s["r"], s["cache"], table, s["n"])
        s["n"].add_(T)
        o, lse = step(s["ql"], s["qr"], s["cache"], table, s["n"], 0.07)
        w = kda.mla_weigh(s["ql"], s["qr"], s["cache"], table, s["n"], lse, 0.07, s["w"], decay=0.9)
        return (o, lse, w) + (kda.mla_cache_read_mx(s["cache"], table, cu, 80, Dc, dtype, starts=s["n"]) if mx else ())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(s)
    for i, lens in enumerate(([100, 7, 300], [0, 64, 399], [33, -9, 200], [1, 2, 63])):
        for k in ("c", "r", "ql", "qr"):
            s[k].copy_(rand(*s[k].shape))
        s["n"].copy_(_i32(lens))
        s["w"].copy_(_weights(g, *s["w"].shape))
        twin = {k: v.clone() for k, v in s.items()}
        graph.replay()
        if i % 2:
            torch.cuda.synchronize()
        want = call(twin)
        for x, y in zip(out, want):
            assert torch.equal(x, y), lens
        assert torch.equal(s["cache"], twin["cache"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mx", [True, False])
def test_queries_that_heads_or_tokens_share(mx, dtype):
    """Strides of zero: one query for all heads, and one for all tokens."""
    lens, T, H = [70, 5, 200], 3, 44
    cache, table, _ = _cache(lens, 32, 512, 64, dtype, 96, mx=mx)
    n, old = _i32(lens), torch.zeros(3, table.shape[1] * 32, device="cuda")
    step = kda.mla_step_mx if mx else kda.mla_step
    for shape in ((3, T, 1), (3, 1, H), (1, T, H)):
        g = torch.Generator(device="cuda").manual_seed(97)
        q = [torch.randn((*shape, D), generator=g, device="cuda").to(dtype).expand(3, T, H, D) for D in (512, 64)]
        o, lse = step(*q, cache, table, n, 0.07)
        w = kda.mla_weigh(*q, cache, table, n, lse, 0.07, old, out=old.clone())
        q = [x.contiguous() for x in q]
        want = step(*q, cache, table, n, 0.07)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(w, kda.mla_weigh(*q, cache, table, n, lse, 0.07, old, out=old.clone()))


@pytest.mark.parametrize("H,pages", [(8, 4), (16, 4096), (32, 4096), (64, 4096), (96, 4096)])
def test_weights_times_scales_next_to_nothing(H, pages):
    """A block that only rows of small weight have, of values that float32 can just hold: weight times scale passes
    2^-126 on the way. Each row's part is off by no more than the header says, whatever the number of sets."""
    Dc, page = 256, 64
    codes = torch.zeros(2 + 40, Dc, dtype=torch.uint8)
    scales = torch.full((42, Dc // 32), 127, dtype=torch.uint8)
    codes[:2, 0] = 2                                             # two rows of a score of 0, with zeros in block 5
    for k in range(40):                                          # the others: scores below 0, values 1 to 6 2^e
        codes[2 + k, 160:192] = torch.arange(32) % 6 + 2
        scales[2 + k, 5] = 25 + k % 3
        codes[2 + k, 32] = 4
        codes[2 + k, 64:67] = torch.tensor([2, 2, 2]) if k % 2 else torch.tensor([0, 0, 0])
    values = ref.values(codes, scales).cuda()
    cache = kda.mla_cache_mx(1, page, Dc, 0, BF16)
    ref.put_page(cache, 0, codes.cuda(), scales.cuda(), None)
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    ql = torch.zeros(1, 1, H, Dc, dtype=BF16, device="cuda")
    ql[..., 32] = -(torch.arange(H, device="cuda") % 12).to(BF16)        # weights down to e^-23
    ql[..., 64:67] = -0.5
    o, lse = kda.mla_step_mx(ql, None, cache, table, _i32([42]), 1.0)
    q = ql[0, 0].double()
    p = torch.softmax(q @ values.t(), -1)
    want = p @ values
    m = re.search(r"may count as 0: (\d) \* 2\^-(\d+) a row at most", re.sub(r"\n \* *", " ", open(HEADER).read()))
    least = int(m.group(1)) * 2.0 ** -int(m.group(2))
    for h in range(H):
        # weights and result rounded to bf16, scores of up to 24 as the float32 they are
        got = o[0, 0, h].double()
        off = (2.0 ** -7 + 2.0 ** -13) * (p[h] @ values.abs()) + 42 * least
        assert bool(((got - want[h]).abs() <= off).all()), h
    assert bool((want[:, 160:] > 0).any())
