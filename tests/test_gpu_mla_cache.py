"""The 4-bit cache of latents, attention over it, gathered weights and eviction on the GPU, against
tests/mla_cache_ref.py (64 bits; rounding and eviction exactly), their edges, and the calls run together."""
import math
import random

import pytest
import torch

import gated_delta_rule_chunk_amd as kda
from tests import mla_cache_ref as ref
from tests import mla_ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
DIMS = [(512, 64), (512, 0), (256, 64), (256, 0)]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rand(g, dtype, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _table(lens, page, g, spare, n_pages=None):
    need = [-(-max(n, 0) // page) for n in lens]
    total = sum(need) + spare if n_pages is None else n_pages
    order = torch.randperm(total, generator=g, device="cuda").cpu()
    if n_pages is not None:
        order = order.sort(descending=True).values
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k].int()
        at += k
    return table, total


def _cache(lens, page, Dc, Dr, dtype, seed, mx=True, spare=2, n_pages=None, wide=False):
    """A cache of either form with `lens` rows per sequence in pages in random order, every other byte such that a
    read of it is a NaN. Returns cache, page table, rows [(latent in float64, shared part or None)]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table, total = _table(lens, page, g, spare, n_pages)
    if mx:
        cache = torch.full((total, page, kda.mla_mx_row_bytes(Dc, Dr, dtype)), 255, dtype=torch.uint8, device="cuda")
    else:
        cache = torch.full((total, page, Dc + Dr), math.nan, dtype=dtype, device="cuda")
    rows = []
    for i, n in enumerate(lens):
        n = max(n, 0)
        r = _rand(g, dtype, n, Dr) if Dr else None
        if mx:
            c, s = ref.encode(_rand(g, F32, n, Dc, std=0.8) * torch.exp2(2 * torch.randn((1, Dc), generator=g, device="cuda"))
                              if wide else _rand(g, F32, n, Dc))
            rows.append((ref.values(c, s), r))
            for k in range(0, n, page):
                ref.put_page(cache, table[i, k // page].item(), c[k:k + page], s[k:k + page], None if r is None else r[k:k + page])
        else:
            x = _rand(g, dtype, n, Dc)
            rows.append((x.double(), r))
            for k in range(0, n, page):
                part = x[k:k + page] if r is None else torch.cat((x[k:k + page], r[k:k + page]), -1)
                cache[table[i, k // page].item(), :part.shape[0]] = part
    return cache, table.cuda(), rows


def _queries(Nb, T, H, Dc, Dr, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ql = _rand(g, dtype, H, Nb, T, Dc, std=0.7).permute(1, 2, 0, 3)          # head-major
    qr = _rand(g, dtype, Nb, T, H, 128 + Dr)[..., 128:] if Dr else None      # a slice of wider heads
    return ql, qr


def _rows_of_queries(ql, qr, b):
    x = ql[b] if qr is None else torch.cat((ql[b], qr[b]), -1)
    return x.flatten(0, 1)


def _limits(n, T, H, have):
    t = torch.arange(T, device="cuda").repeat_interleave(H)
    return (n - T + t + 1).clamp(0, have)


def _check_step(ql, qr, rows, o, lse, scale, lens, mx=True):
    Nb, T, H, Dc = ql.shape
    for b in range(Nb):
        c, r = rows[b]
        res = ref.attend(_rows_of_queries(ql, qr, b), c, r, scale, _limits(max(lens[b], 0), T, H, c.shape[0]), ql.dtype, mx)
        mla_ref.check(f"o[{b}]", o[b].reshape(1, T * H, Dc), res["o"])
        mla_ref.check(f"lse[{b}]", lse[b].reshape(1, T * H), res["lse"])


# ---- rows to and from the cache --------------------------------------------------------------------------------------


def _special(dtype):
    """Rows of 256 channels whose blocks are the edges of the rounding."""
    b = []
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)
    for x in (ties, -ties, ties * 2.0 ** -60, torch.tensor([7.0] + [0.0] * 31), torch.tensor([7.0078125] + [1.0] * 31),
              torch.tensor([-1.75, 1.0, 0.875] + [2.0 ** -9] * 29), torch.zeros(32), -torch.zeros(32),
              torch.full((32,), 2.0 ** -100), torch.full((32,), 2.0 ** -101), torch.full((32,), 3e38), torch.full((32,), 2.0 ** 127),
              torch.tensor([3.3e38, -1e38] + [2.0 ** 120] * 30), torch.full((32,), 1e-40),
              torch.tensor([math.nan] + [1.0] * 31), torch.tensor([1.0] * 31 + [-math.inf])):
        b.append(x)
    return torch.stack(b).view(2, 256).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dc,Dr", DIMS)
@pytest.mark.parametrize("page,packed", [(16, True), (64, False), (32, True)])
def test_append_and_read(dtype, Dc, Dr, page, packed):
    before = [0, 15, -1, 16, 63, 100]
    new = [3, 1, 2, 0, 70, 17] if packed else [3] * 6
    total = [max(a, 0) + b for a, b in zip(before, new)]
    cache, table, rows = _cache([max(a, 0) for a in before], page, Dc, Dr, dtype, 10, spare=12)
    g = torch.Generator(device="cuda").manual_seed(11)
    free = sorted(set(range(cache.shape[0])) - set(table.flatten().tolist()))
    table = torch.cat((table, torch.full((6, 8), -1, dtype=torch.int32, device="cuda")), 1)
    for i, n in enumerate(total):
        for k in range(-(-n // page)):
            if table[i, k] < 0:
                table[i, k] = free.pop()
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    shape = (1, cu[-1] + 4) if packed else (6, 3)                # packed: four tokens behind the last sequence
    lat = _rand(g, dtype, *shape, Dc + 64)[..., 32:32 + Dc]      # a slice
    sp = _special(dtype).cuda()
    if packed:
        lat[0, cu[4] + 5:cu[4] + 7, Dc - 256:] = sp
    else:
        lat[4, 1:3, Dc - 256:] = sp
    kr = _rand(g, dtype, *shape, 2 * Dr)[..., Dr:] if Dr else None
    want = cache.clone()
    flat = [(lat[0, cu[n]:cu[n + 1]], None if kr is None else kr[0, cu[n]:cu[n + 1]]) if packed else
            (lat[n], None if kr is None else kr[n]) for n in range(6)]
    for n, (x, r) in enumerate(flat):
        c, s = ref.encode(x)
        for t in range(x.shape[0] if before[n] >= 0 else 0):
            p = before[n] + t
            pg = table[n, p // page].item()
            one = torch.full_like(want[pg], 0)[None]             # the row alone, by way of a page of its own
            ref.put_page(one, 0, c[t:t + 1].expand(page, -1), s[t:t + 1].expand(page, -1),
                         None if r is None else r[t:t + 1].expand(page, -1))
            mask = torch.zeros_like(one)
            f = mask.view(-1)
            a0, a1 = page * Dc // 2, page * (Dc // 2 + Dc // 32)
            i = p % page
            f[i * Dc // 2:(i + 1) * Dc // 2] = 1
            f[a0 + i * Dc // 32:a0 + (i + 1) * Dc // 32] = 1
            es = Dr * torch.finfo(dtype).bits // 8
            f[a1 + i * es:a1 + (i + 1) * es] = 1
            want[pg] = torch.where(mask[0] == 1, one[0], want[pg])
    lens = _i32(before)
    kda.mla_cache_append_mx(lat, kr, cache, table, lens, cu_seqlens=_i32(cu) if packed else None)
    assert torch.equal(cache, want)
    # back: the whole of each sequence, then parts
    live = [n if b >= 0 else 0 for n, b in zip(total, before)]
    for starts, counts in ((None, live), ([5, 0, 0, 3, 60, 7], [max(0, n - s) for n, s in zip(live, [5, 0, 0, 3, 60, 7])])):
        cb = [sum(counts[:i]) for i in range(7)]
        x, r = kda.mla_cache_read_mx(cache, table, _i32(cb), cb[-1] + 3, Dc, dtype, starts=None if starts is None else _i32(starts))
        for n in range(6):
            c, rr = ref.get_rows(want, table[n], live[n], Dc, Dr, dtype)
            s0 = 0 if starts is None else starts[n]
            got = x[0, cb[n]:cb[n + 1]].double()
            w = c[s0:s0 + counts[n]]
            assert torch.equal(torch.nan_to_num(got, nan=9e99), torch.nan_to_num(w.to(dtype).double(), nan=9e99)), n
            if Dr:
                assert torch.equal(r[0, cb[n]:cb[n + 1]], rr[s0:s0 + counts[n]])
        assert not x[0, cb[-1]:].any() and (r is None or not r[0, cb[-1]:].any())
    assert (r is None) == (Dr == 0)
    out = (torch.full_like(x, 7), None if r is None else torch.full_like(r, 7))
    kda.mla_cache_read_mx(cache, table, _i32(cb), cb[-1] + 3, Dc, dtype, starts=_i32(starts), out=out)
    assert bool((out[0][0, cb[-1]:] == 7).all()) and torch.equal(torch.nan_to_num(out[0][0, :cb[-1]]), torch.nan_to_num(x[0, :cb[-1]]))


def test_rows_that_do_not_exist_are_reported():
    cache, table, rows = _cache([40, 20], 16, 256, 64, BF16, 12)
    want = cache.clone()
    bad = table.clone()
    bad[0, 1] = cache.shape[0]
    new = _rand(torch.Generator(device="cuda").manual_seed(1), BF16, 2, 1, 256), torch.ones(2, 1, 64, dtype=BF16, device="cuda")
    kda.mla_cache_append_mx(*new, cache, bad, _i32([20, 48]))    # a missing page, one past the table
    with pytest.raises(kda.KDAError, match="2 counted"):
        kda.device_check()
    assert torch.equal(cache, want)
    x, r = kda.mla_cache_read_mx(cache, bad, _i32([0, 40, 45]), 45, 256, BF16, starts=_i32([0, -2]))
    with pytest.raises(kda.KDAError, match="18 counted"):
        kda.device_check()
    assert not x[0, 16:32].any() and not r[0, 16:32].any() and not x[0, 40:42].any()
    assert torch.equal(x[0, :16].double(), rows[0][0][:16]) and torch.equal(x[0, 42:].double(), rows[1][0][:3])
    assert torch.equal(r[0, 32:40], rows[0][1][32:40])


# ---- attention -------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dc,Dr", DIMS)
@pytest.mark.parametrize("H,T,page", [(1, 1, 16), (33, 1, 64), (96, 1, 32), (130, 1, 128), (16, 5, 16), (40, 3, 64)])
def test_step(dtype, Dc, Dr, H, T, page):
    lens = [0, 1, 31, 32, 33, -1, 130, 257, 16, 2]
    cache, table, rows = _cache(lens, page, Dc, Dr, dtype, H + T)
    ql, qr = _queries(len(lens), T, H, Dc, Dr, dtype, 2)
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.06)
    _check_step(ql, qr, rows, o, lse, 0.06, lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [12, 64, 96, 128])
@pytest.mark.parametrize("lens", [[5000], [700, 3000, 33, 0, 1201], [100] * 90])
def test_step_split_over_the_cache(dtype, H, lens):
    cache, table, rows = _cache(lens, 64, 512, 64, dtype, 4)
    ql, qr = _queries(len(lens), 1, H, 512, 64, dtype, 5)
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    _check_step(ql, qr, rows, o, lse, 0.07, lens)
    again = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_step_queries_of_very_different_sizes():
    """Channels of a block of 32 from 2^-30 of the largest on, blocks of zeros, and latents that differ as much."""
    lens, H = [70, 300], 40
    cache, table, rows = _cache(lens, 32, 512, 64, BF16, 31, wide=True)
    ql, qr = _queries(2, 1, H, 512, 64, BF16, 32)
    g = torch.Generator(device="cuda").manual_seed(33)
    ql = (ql.float() * torch.exp2(-torch.randint(0, 31, ql.shape, generator=g, device="cuda").float())).to(BF16)
    ql[:, :, ::7, 64:96] = 0
    ql[:, :, 1, :] *= 2.0 ** 40
    ql[:, :, 2, :] *= 2.0 ** -60
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.05)
    _check_step(ql, qr, rows, o, lse, 0.05, lens)


def test_step_large_scores():
    lens = [900]
    cache, table, rows = _cache(lens, 64, 512, 64, BF16, 14)
    ql, qr = _queries(1, 1, 96, 512, 64, BF16, 15)
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=5.0)
    _check_step(ql, qr, rows, o, lse, 5.0, lens)


@pytest.mark.parametrize("H", [8, 24, 96])
@pytest.mark.parametrize("std", [0.7, 40.0])
def test_step_latents_of_all_magnitudes(H, std):
    """Blocks from 2^-97 to 2^100, keys of one block up to 2^40 apart, weights spread and on a few keys."""
    lens, Dc, page = [200, 33, 1], 256, 16
    g = torch.Generator(device="cuda").manual_seed(26)
    table, total = _table(lens, page, g, 1)
    cache = torch.zeros((total, page, kda.mla_mx_row_bytes(Dc, 0, BF16)), dtype=torch.uint8, device="cuda")
    powers = torch.tensor([-97.0, -60.0, 0.0, 0.0, 0.0, 20.0, 60.0, 98.0], device="cuda").repeat_interleave(32)
    rows = []
    for i, n in enumerate(lens):
        spread = torch.zeros(n, 8, device="cuda")
        spread[:, 4] = torch.randint(-20, 21, (n,), generator=g, device="cuda").float()
        x = _rand(g, F32, n, Dc).double() * ref.power((powers + spread.repeat_interleave(32, 1)).long())
        c, s = ref.encode(x.float())
        rows.append((ref.values(c, s), None))
        for k in range(0, n, page):
            ref.put_page(cache, table[i, k // page].item(), c[k:k + page], s[k:k + page], None)
    ql, _ = _queries(len(lens), 1, H, Dc, 0, BF16, 27)
    ql = (ql / 0.7 * std).to(BF16)
    ql[..., :64] = 0                                             # scores by the two blocks of 2^0
    ql[..., 128:] = 0
    o, lse = kda.mla_step_mx(ql, None, cache, table.cuda(), _i32(lens), scale=0.06)
    _check_step(ql, None, rows, o, lse, 0.06, lens)


@pytest.mark.parametrize("Dc,Dr", DIMS)
@pytest.mark.parametrize("H,lens", [(12, [40000, 0, 3]), (24, [33000, 700]), (8, [300] * 130)])
def test_step_of_few_rows_over_many_parts(Dc, Dr, H, lens):
    """Two workgroups a compute unit: up to 512 parts, of one sequence or of many."""
    cache, table, rows = _cache(lens, 64, Dc, Dr, BF16, 24)
    ql, qr = _queries(len(lens), 1, H, Dc, Dr, BF16, 25)
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    _check_step(ql, qr, rows, o, lse, 0.07, lens)
    again = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_parts_of_more_pages_than_lanes(dtype):
    """One sequence in 16-row pages, parts of over 64 pages."""
    lens = [40000, 17]
    cache, table, rows = _cache(lens, 16, 256, 0, dtype, 19)
    ql, qr = _queries(2, 1, 8 if dtype == F32 else 1024, 256, 0, dtype, 20)    # 1024 rows: 32 parts
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    _check_step(ql, qr, rows, o, lse, 0.07, lens)


def test_step_nan_stays_in_its_sequence():
    lens = [100, 40, 300]
    cache, table, rows = _cache(lens, 16, 512, 64, BF16, 40)
    ql, qr = _queries(3, 2, 20, 512, 64, BF16, 41)
    want = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    flat = cache[table[1, 1].item()].view(-1)
    flat[16 * 256 + 3 * 16 + 5] = 255                            # block 5 of row 19 of sequence 1
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    for b in (0, 2):
        assert torch.equal(o[b], want[0][b]) and torch.equal(lse[b], want[1][b])
    assert bool(o[1, ..., 160:192].isnan().all()) and bool(lse[1].isnan().all())


def test_offsets_past_four_gib():
    """Page offsets past 2^32 bytes: write, read, attention, weights, eviction."""
    lens = [300, 45]
    cache, table, rows = _cache(lens, 256, 512, 64, BF16, 6, n_pages=43000)
    assert int(table.min()) * 256 * 400 > 1 << 32 or int(table.max()) * 256 * 400 > 1 << 32
    ql, qr = _queries(2, 1, 8, 512, 64, BF16, 7)
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    _check_step(ql, qr, rows, o, lse, 0.07, lens)
    w = torch.zeros(2, 512, device="cuda")
    kda.mla_weigh(ql, qr, cache, table, _i32(lens), lse, 0.07, w)
    _check_weights(w, ql, qr, rows, lse, 0.07, lens, torch.zeros_like(w), 1, 1.0, True)
    x, r = kda.mla_cache_read_mx(cache, table, _i32([0, 300, 345]), 345, 512, BF16)
    assert torch.equal(x[0].double(), torch.cat((rows[0][0], rows[1][0])))
    new = torch.full((2, 1, 576), 1.5, dtype=BF16, device="cuda")
    kda.mla_cache_append_mx(new[..., :512], new[..., 512:], cache, table, _i32([299, 44]))
    x, r = kda.mla_cache_read_mx(cache, table, _i32([0, 1, 2]), 2, 512, BF16, starts=_i32([299, 44]))
    assert bool((x == 1.5).all()) and bool((r == 1.5).all())


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_missing_pages_are_reported(page, dtype):
    lens = [100, 70, 40]
    cache, table, rows = _cache(lens, page, 512, 64, dtype, 8)
    ql, qr = _queries(3, 1, 8, 512, 64, dtype, 9)
    bad = table.clone()
    bad[0, 1] = cache.shape[0]
    bad[1, 0] = -1
    o, lse = kda.mla_step_mx(ql, qr, cache, bad, _i32(lens), scale=0.07)
    with pytest.raises(kda.KDAError, match="2 counted"):
        kda.device_check()
    cut = lambda x, i: None if x is None else torch.cat((x[:i * page], x[(i + 1) * page:]))  # noqa: E731
    keep = [tuple(cut(x, 1) for x in rows[0]), tuple(cut(x, 0) for x in rows[1]), rows[2]]
    _check_step(ql, qr, keep, o, lse, 0.07, [x[0].shape[0] for x in keep])
    w = torch.full((3, table.shape[1] * page), 2.0, device="cuda")
    kda.mla_weigh(ql, qr, cache, bad, _i32(lens), lse, 0.07, w, fresh=0)
    with pytest.raises(kda.KDAError, match="2 counted"):
        kda.device_check()
    assert bool((w[0, page:2 * page] == 2).all()) and bool((w[1, :page] == 2).all()) and bool((w[2, 40:] == 2).all())
    kda.mla_step_mx(ql, qr, cache, table, _i32([100, 70, 10 ** 6]), scale=0.07)
    with pytest.raises(kda.KDAError, match="page table"):
        kda.device_check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,page", [(4, 16), (3, 32)])
def test_length_past_the_page_table_hides_its_rows_only(dtype, T, page):
    cap, H = 3 * page, 7
    lens = [cap, cap + 1, cap + T - 1, cap + 50, 10 ** 9, cap - 1]
    cache, table, rows = _cache([cap] * len(lens), page, 256, 64, dtype, 22)
    ql, qr = _queries(len(lens), T, H, 256, 64, dtype, 23)
    o, lse = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), scale=0.07)
    with pytest.raises(kda.KDAError, match="4 counted"):
        kda.device_check()
    _check_step(ql, qr, rows, o, lse, 0.07, lens)
    w = torch.zeros(len(lens), cap, device="cuda")
    kda.mla_weigh(ql, qr, cache, table, _i32(lens), lse, 0.07, w)
    with pytest.raises(kda.KDAError, match="4 counted"):
        kda.device_check()
    _check_weights(w, ql, qr, rows, lse, 0.07, lens, torch.zeros_like(w), T, 1.0, True)


# ---- gathered weights ------------------------------------------------------------------------------------------------


def _check_weights(w, ql, qr, rows, lse, scale, lens, old, fresh, decay, mx):
    Nb, T, H, _ = ql.shape
    for b in range(Nb):
        c, r = rows[b]
        n = c.shape[0]
        base = old[b, :n].clone()
        base[max(0, max(lens[b], 0) - fresh):] = 0
        if decay == 0:
            base[:] = 0
        res = ref.gathered(_rows_of_queries(ql, qr, b), c, r, lse[b].flatten(), scale, _limits(max(lens[b], 0), T, H, n), base,
                           decay, ql.dtype, mx)
        mla_ref.check(f"weights[{b}]", w[b, :n], res)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("Dc,Dr", DIMS)
@pytest.mark.parametrize("H,T,page,fresh,decay", [(1, 1, 16, None, 1.0), (33, 1, 64, 0, 0.5), (96, 1, 32, None, 1.0),
                                                  (130, 1, 128, 40, 1.0), (16, 5, 16, None, 0.9), (40, 9, 64, 10 ** 10, 1.0),
                                                  (64, 2, 32, 3, 0.0)])
def test_weigh(dtype, mx, Dc, Dr, H, T, page, fresh, decay):
    lens = [0, 1, 31, 32, 33, -1, 130, 257, 16, 2, 700]
    cache, table, rows = _cache(lens, page, Dc, Dr, dtype, H + T, mx=mx)
    ql, qr = _queries(len(lens), T, H, Dc, Dr, dtype, 2)
    n = _i32(lens)
    lse = (kda.mla_step_mx if mx else kda.mla_step)(ql, qr, cache, table, n, scale=0.06)[1]
    g = torch.Generator(device="cuda").manual_seed(3)
    old = torch.rand((len(lens), table.shape[1] * page), generator=g, device="cuda")
    # weights that are not to be read
    f = T if fresh is None else fresh
    poisoned = old.clone()
    for b, m in enumerate(lens):
        m = max(m, 0)
        poisoned[b, m:] = math.nan
        poisoned[b, (0 if decay == 0 else max(0, m - f)):m] = math.nan
    out = torch.full_like(old, 7.0)
    got = kda.mla_weigh(ql, qr, cache, table, n, lse, 0.06, poisoned, fresh=fresh, decay=decay, out=out)
    assert got is out
    _check_weights(out, ql, qr, rows, lse, 0.06, lens, old, f, decay, mx)
    for b, m in enumerate(lens):
        assert bool((out[b, max(m, 0):] == 7).all())
    # in place: the same bits, and what lies behind the rows is left
    w = poisoned.clone()
    assert kda.mla_weigh(ql, qr, cache, table, n, lse, 0.06, w, fresh=fresh, decay=decay) is w
    for b, m in enumerate(lens):
        m = max(m, 0)
        assert torch.equal(w[b, :m], out[b, :m]) and bool(w[b, m:].isnan().all())


@pytest.mark.parametrize("dtype,mx,H,T,lens", [(BF16, True, 96, 1, [9000, 2500, 40]), (BF16, False, 96, 1, [9000, 2500, 40]),
                                               (BF16, True, 24, 40, [1500, 31, 300]), (F32, False, 24, 20, [1500, 31, 300]),
                                               (F32, True, 12, 1, [70] * 100), (BF16, True, 1, 1, [1] * 300)])
def test_weigh_larger(dtype, mx, H, T, lens):
    cache, table, rows = _cache(lens, 64, 512, 64, dtype, 50, mx=mx)
    ql, qr = _queries(len(lens), T, H, 512, 64, dtype, 51)
    n = _i32(lens)
    lse = (kda.mla_step_mx if mx else kda.mla_step)(ql, qr, cache, table, n, scale=0.07)[1]
    old = torch.rand((len(lens), table.shape[1] * 64), device="cuda")
    out = torch.zeros_like(old)
    kda.mla_weigh(ql, qr, cache, table, n, lse, 0.07, old, out=out)
    _check_weights(out, ql, qr, rows, lse, 0.07, lens, old, T, 1.0, mx)
    again = torch.zeros_like(old)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kda.mla_weigh(ql, qr, cache, table, n, lse, 0.07, old, out=again)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, again)
    # each token and head hands out a weight of 1
    fresh = kda.mla_weigh(ql, qr, cache, table, n, lse, 0.07, torch.zeros_like(old), fresh=10 ** 6)
    for b, m in enumerate(lens):
        seen = sum(1 for t in range(T) if m - T + t + 1 > 0) * H
        assert abs(fresh[b, :m].double().sum().item() - seen) <= 1e-4 * seen


def test_weigh_nan_stays_in_its_row():
    lens = [100, 300]
    cache, table, rows = _cache(lens, 16, 512, 64, BF16, 60)
    ql, qr = _queries(2, 1, 20, 512, 64, BF16, 61)
    n = _i32(lens)
    lse = kda.mla_step_mx(ql, qr, cache, table, n, scale=0.07)[1]
    want = kda.mla_weigh(ql, qr, cache, table, n, lse, 0.07, torch.zeros(2, table.shape[1] * 16, device="cuda"))
    cache[table[1, 1].item()].view(-1)[16 * 256 + 3 * 16 + 5] = 255
    got = kda.mla_weigh(ql, qr, cache, table, n, lse, 0.07, torch.zeros_like(want))
    assert got[1, 19].isnan()
    got[1, 19] = want[1, 19]
    assert torch.equal(got, want)


# ---- eviction --------------------------------------------------------------------------------------------------------


def _evict_and_check(cache, table, n, w, keep, first, recent, in_place):
    """Calls mla_evict and compares everything with the rule, bit for bit."""
    page, lens = cache.shape[1], n.tolist()
    before, t0, w0 = cache.clone(), table.cpu().clone(), w.cpu().clone()
    out = None if in_place else (torch.full_like(table, -9), torch.full_like(n, -9), torch.full_like(w, -9.0))
    t1, n1, w1 = kda.mla_evict(cache, table, n, w, keep, first=first, recent=recent, out=out)
    if in_place:
        assert t1 is table and n1 is n and w1 is w
    else:
        assert torch.equal(table.cpu(), t0) and n.tolist() == lens
        assert torch.equal(torch.nan_to_num(w.cpu(), nan=-5.0), torch.nan_to_num(w0, nan=-5.0))
    mx = cache.dtype == torch.uint8
    if mx:
        sizes = {136: (128, 8, 0), 264: (128, 8, 128), 392: (128, 8, 256), 272: (256, 16, 0), 400: (256, 16, 128),
                 528: (256, 16, 256)}[cache.shape[2]]

    def row(c, p):                                               # a row's bytes in either form
        pg, i = c[p // page], p % page
        if not mx:
            return pg[i].view(torch.uint8)
        flat, at, out = pg.view(-1), 0, []
        for s in sizes:
            out.append(flat[at + i * s:at + (i + 1) * s])
            at += page * s
        return torch.cat(out)

    changed = {}
    for b, L in enumerate(lens):
        L = max(L, 0)
        E, a, e, moves, order = ref.evict(w0[b, :L].tolist(), L, page, keep, first, recent)
        used = -(-L // page)
        t = t0[b].tolist()
        assert t1[b].tolist() == (t[:e - E] + t[e:used] + t[e - E:e] + t[used:] if E else t)
        assert n1[b].item() == (L - E * page if L else lens[b])
        ww = torch.cat((w0[b, order], torch.zeros(E * page), w0[b, L:]))
        assert torch.equal(torch.nan_to_num(w1[b].cpu(), nan=-5.0), torch.nan_to_num(ww, nan=-5.0))
        for d, s in moves:
            changed[t[d // page] * page + d % page] = t[s // page] * page + s % page
    # the cache: moved rows, and nothing else
    want = before.clone()
    if mx:
        view = torch.cat([want.view(want.shape[0], -1)[:, o0 * page:(o0 + s) * page].reshape(want.shape[0], page, s)
                          for o0, s in zip((0, sizes[0], sizes[0] + sizes[1]), sizes)], 2).flatten(0, 1)
        got = torch.cat([cache.view(want.shape[0], -1)[:, o0 * page:(o0 + s) * page].reshape(want.shape[0], page, s)
                         for o0, s in zip((0, sizes[0], sizes[0] + sizes[1]), sizes)], 2).flatten(0, 1)
    else:
        view, got = want.flatten(0, 1).view(torch.uint8), cache.flatten(0, 1).view(torch.uint8)
    if changed:
        d, s = torch.tensor(list(changed), device="cuda"), torch.tensor(list(changed.values()), device="cuda")
        view[d] = view[s].clone()
    assert torch.equal(got, view)
    return t1, n1, w1


def _weights(g, *shape):
    w = torch.exp(2 * torch.randn(shape, generator=g, device="cuda"))
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.2, 0.0, w)


@pytest.mark.parametrize("mx,dtype,Dc,Dr", [(True, BF16, 512, 64), (True, F32, 512, 64), (True, BF16, 256, 0), (True, F32, 256, 64),
                                            (False, BF16, 512, 64), (False, F32, 256, 0), (True, BF16, 512, 0),
                                            (True, BF16, 256, 64), (False, F32, 512, 64)])
@pytest.mark.parametrize("page,keep,first,recent,in_place", [(16, 100, 0, 0, True), (64, 200, 4, 70, False), (32, 0, 0, 33, True),
                                                             (16, 90, 40, 2000, False), (16, 17, 1, 1, True)])
def test_evict(mx, dtype, Dc, Dr, page, keep, first, recent, in_place):
    lens = [0, 1, 31, -1, keep, keep + page, keep + page - 1, 300, 257, 1111, 640]
    cache, table, rows = _cache(lens, page, Dc, Dr, dtype, keep + page, mx=mx)
    g = torch.Generator(device="cuda").manual_seed(5)
    w = _weights(g, len(lens), table.shape[1] * page)
    _evict_and_check(cache, table, _i32(lens), w, keep, first, recent, in_place)


@pytest.mark.parametrize("kind", ["equal", "two", "zeros", "odd", "falling", "rising"])
def test_evict_ties_and_odd_weights(kind):
    lens, page = [700, 333, 64], 16
    cache, table, _ = _cache(lens, page, 256, 0, BF16, 70)
    N = table.shape[1] * page
    j = torch.arange(N, device="cuda").float().expand(3, -1)
    g = torch.Generator(device="cuda").manual_seed(6)
    u = torch.randint(0, 6, (3, N), generator=g, device="cuda")
    odd = torch.tensor([math.nan, math.inf, -0.0, 0.0, -1.0, 1e-42], device="cuda")[u]
    w = {"equal": torch.ones_like(j), "two": 1.0 + (u % 2), "zeros": torch.where(u % 2 == 0, 0.0, -0.0), "odd": odd,
         "falling": 1000 - j, "rising": 1 + j / 7}[kind].contiguous()
    _evict_and_check(cache, table, _i32(lens), w, 150, 20, 40, True)


def test_evict_long_sequences_and_many():
    page = 64
    for lens, keep in (([100001, 5000], 50000), ([500 + i % 7 for i in range(300)], 256)):
        g = torch.Generator(device="cuda").manual_seed(72)
        table, total = _table(lens, page, g, 2)
        table = table.cuda()
        cache = torch.randint(0, 255, (total, page, 136), dtype=torch.uint8, device="cuda", generator=g)
        w = _weights(g, len(lens), table.shape[1] * page)
        _evict_and_check(cache, table, _i32(lens), w, keep, 0, 64, True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["equal", "two", "odd", "falling", "rising", "any"])
@pytest.mark.parametrize("cap", [16384, 16400, 1 << 21, (1 << 21) + 4096])
def test_evict_of_page_tables_of_any_room(cap, kind, in_place):
    lens, page = [16384, 40001, 700, 0, 4097, -1], 16
    lens[1] = min(lens[1], cap)
    g = torch.Generator(device="cuda").manual_seed(75)
    table, total = _table(lens, page, g, 1)
    wide = torch.full((len(lens), cap // page), -7, dtype=torch.int32)
    m = min(table.shape[1], wide.shape[1])
    wide[:, :m] = table[:, :m]
    cache = torch.randint(0, 255, (total, page, 136), dtype=torch.uint8, device="cuda", generator=g)
    N = 40016
    j = torch.arange(N, device="cuda").float().expand(len(lens), -1)
    u = torch.randint(0, 6, (len(lens), N), generator=g, device="cuda")
    odd = torch.tensor([math.nan, math.inf, -0.0, 0.0, -1.0, 1e-42], device="cuda")[u]
    some = {"equal": torch.ones_like(j), "two": 1.0 + (u % 2), "odd": odd, "falling": 1e5 - j, "rising": 1 + j / 7,
            "any": _weights(g, len(lens), N)}[kind]
    w = torch.full((len(lens), cap), 3.0, device="cuda")
    w[:, :min(N, cap)] = some[:, :cap]
    _evict_and_check(cache, wide.cuda(), _i32(lens), w, 3000, 20, 40, in_place)


def test_evict_keeps_the_order_of_many_recent_rows():
    lens, page = [30000, 9000], 16
    g = torch.Generator(device="cuda").manual_seed(76)
    table, total = _table(lens, page, g, 1)
    cache = torch.randint(0, 255, (total, page, 136), dtype=torch.uint8, device="cuda", generator=g)
    w = _weights(g, 2, table.shape[1] * page)
    _evict_and_check(cache, table.cuda(), _i32(lens), w, 1000, 100, 8500, True)


def test_evict_refuses_sequences_with_missing_pages():
    lens, page = [200, 200, 90, 5000], 16
    cache, table, _ = _cache([200, 200, 90, 208], page, 512, 64, BF16, 73)
    bad = table.clone()
    bad[0, 3] = cache.shape[0]
    bad[1, 12] = -1                                              # among the recent ones: not looked at
    g = torch.Generator(device="cuda").manual_seed(74)
    w = _weights(g, 4, table.shape[1] * page)
    before, n = cache.clone(), _i32(lens)
    t1, n1, w1 = kda.mla_evict(cache, bad, n, w, 100, recent=20, out=(torch.empty_like(bad), torch.empty_like(n), torch.empty_like(w)))
    with pytest.raises(kda.KDAError, match="2 counted"):
        kda.device_check()
    assert n1.tolist() == [200, 200 - 96, 90, 5000]
    for b in (0, 2, 3):
        assert torch.equal(t1[b], bad[b]) and torch.equal(w1[b], w[b])
    mine = table[1].tolist()
    others = [p for p in range(cache.shape[0]) if p not in mine]
    assert torch.equal(cache[others], before[others])


# ---- together --------------------------------------------------------------------------------------------------------


def test_weigh_many_rows_on_two_streams():
    """Over 128 rows of queries: calls at once with a workspace each give what they give alone; a short one is refused."""
    lens, H, T = [700, 33, 0, 400], 20, 9
    cache, table, rows = _cache(lens, 64, 512, 64, BF16, 52)
    n, old = _i32(lens), torch.zeros(4, table.shape[1] * 64, device="cuda")
    need = kda.mla_weigh_workspace_bytes(4, T, H, 512, 64, BF16, 1)
    calls, want = [], []
    for k in range(2):
        ql, qr = _queries(4, T, H, 512, 64, BF16, 53 + k)
        lse = kda.mla_step_mx(ql, qr, cache, table, n, scale=0.06)[1]
        calls.append((ql, qr, lse, torch.empty(need, dtype=torch.uint8, device="cuda"), old.clone()))
        want.append(kda.mla_weigh(ql, qr, cache, table, n, lse, 0.06, old, out=old.clone()))
        _check_weights(want[k], ql, qr, rows, lse, 0.06, lens, old, T, 1.0, True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for s, (ql, qr, lse, ws, out) in zip(streams, calls):
            with torch.cuda.stream(s):
                kda.mla_weigh(ql, qr, cache, table, n, lse, 0.06, old, out=out, workspace=ws)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c[4], w)
    ql, qr, lse, ws, out = calls[0]
    with pytest.raises(kda.KDAError, match="workspace"):
        kda.mla_weigh(ql, qr, cache, table, n, lse, 0.06, old, out=out, workspace=ws[:need - 16])


@pytest.mark.parametrize("cap", [16384, 40000])
def test_evict_in_a_graph(cap):
    """Captured once, replayed with other weights and lengths: one launch that decides, and several."""
    page, N = 16, 3
    g = torch.Generator(device="cuda").manual_seed(77)
    table = torch.randperm(N * cap // page, generator=g, device="cuda").to(torch.int32).view(N, -1)
    cache = torch.zeros(N * cap // page, page, 136, dtype=torch.uint8, device="cuda")
    n, w = _i32([cap, 9000, 100]), _weights(g, N, cap)
    out = torch.empty_like(table), torch.empty_like(n), torch.empty_like(w)
    ws = torch.empty(kda.mla_evict_workspace_bytes(N, page, cap // page), dtype=torch.uint8, device="cuda")

    def call():
        kda.mla_evict(cache, table, n, w, 4000, first=5, recent=100, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        n.copy_(_i32([cap - 1000 * i, 9000 - 1700 * i, 5000 * (i % 2)]))
        w.copy_(_weights(g, N, cap))
        for o in out:
            o.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        for b, L in enumerate(n.tolist()):
            E, a, e, moves, order = ref.evict(w[b, :L].tolist(), L, page, 4000, 5, 100)
            ww = torch.cat((w[b].cpu()[order], torch.zeros(E * page), w[b, L:].cpu()))
            assert out[1][b].item() == L - E * page and torch.equal(out[2][b].cpu(), ww)


@pytest.mark.parametrize("mx,dtype", [(True, BF16), (False, BF16), (True, F32)])
def test_serving_run(mx, dtype):
    """A prompt, its weights, and generated tokens with an eviction every few steps; attention against the rows that the
    rule keeps, tracked on the host."""
    H, Dc, Dr, N, page, keep = 12, 512, 64, 3, 16, 64
    g = torch.Generator(device="cuda").manual_seed(80)
    prompts = [90, 40, 130]
    cap = 12 * page
    table = torch.randperm(N * 12, generator=g, device="cuda").to(torch.int32).view(N, 12)
    cache = kda.mla_cache_mx(N * 12, page, Dc, Dr, dtype) if mx else torch.zeros((N * 12, page, Dc + Dr), dtype=dtype, device="cuda")
    append = kda.mla_cache_append_mx if mx else kda.mla_cache_append
    step = kda.mla_step_mx if mx else kda.mla_step
    host = [(torch.zeros(0, Dc, dtype=torch.float64, device="cuda"), torch.zeros(0, Dr, dtype=dtype, device="cuda"))
            for _ in range(N)]

    def write(lat, kr, counts, n):
        cu = _i32([sum(counts[:i]) for i in range(N + 1)])
        append(lat, kr, cache, table, n, cu_seqlens=cu)
        for b in range(N):
            x = lat[0, cu[b]:cu[b + 1]]
            x = ref.values(*ref.encode(x)) if mx else x.double()
            host[b] = torch.cat((host[b][0], x)), torch.cat((host[b][1], kr[0, cu[b]:cu[b + 1]]))

    n = _i32([0] * N)
    write(_rand(g, dtype, 1, sum(prompts), Dc), _rand(g, dtype, 1, sum(prompts), Dr), prompts, n)
    n += _i32(prompts)
    w = torch.zeros(N, cap, device="cuda")
    ql, qr = _queries(N, 8, H, Dc, Dr, dtype, 81)                # the prompts' last tokens
    o, lse = step(ql, qr, cache, table, n, 0.07)
    kda.mla_weigh(ql, qr, cache, table, n, lse, 0.07, w, fresh=10 ** 6)
    _check_weights(w, ql, qr, host, lse, 0.07, n.tolist(), w, 10 ** 6, 1.0, mx)
    for i in range(9):
        if i % 4 == 0:
            lens, w0 = n.tolist(), w.cpu()
            kda.mla_evict(cache, table, n, w, keep, first=4, recent=20)
            for b in range(N):
                E, *_, order = ref.evict(w0[b, :lens[b]].tolist(), lens[b], page, keep, 4, 20)
                assert n[b].item() == lens[b] - E * page
                host[b] = host[b][0][order], host[b][1][order]
        write(_rand(g, dtype, 1, N, Dc), _rand(g, dtype, 1, N, Dr), [1] * N, n)
        n += 1
        ql, qr = _queries(N, 1, H, Dc, Dr, dtype, 90 + i)
        o, lse = step(ql, qr, cache, table, n, 0.07)
        _check_step(ql, qr, host, o, lse, 0.07, n.tolist(), mx)
        old = w.clone()
        kda.mla_weigh(ql, qr, cache, table, n, lse, 0.07, w, decay=0.9)
        _check_weights(w, ql, qr, host, lse, 0.07, n.tolist(), old, 1, 0.9, mx)
    assert max(n.tolist()) < 90


def test_prefix_read_back_for_the_expanded_form():
    """Rows read back, up-projected, and attended to by the expanded form, equal the absorbed form over the cache."""
    H, Dn, Dc, Dr, scale = 4, 128, 512, 64, 0.07
    lens = [70, 33]
    cache, table, rows = _cache(lens, 32, Dc, Dr, F32, 82)
    g = torch.Generator(device="cuda").manual_seed(83)
    up_k, up_v = _rand(g, F32, H, Dn, Dc, std=0.05), _rand(g, F32, H, Dn, Dc, std=0.05)
    q = _rand(g, F32, 2, 1, H, Dn + Dr)
    cu = _i32([0, 70, 103])
    lat, kr = kda.mla_cache_read_mx(cache, table, cu, 103, Dc, F32)
    kv = torch.cat((torch.einsum("tc,hdc->thd", lat[0].double(), up_k.double()),
                    torch.einsum("tc,hdc->thd", lat[0].double(), up_v.double())), -1).float()[None]
    o1, lse1 = kda.mla_fwd(q.view(1, 2, H, Dn + Dr), kv, kr, cu_seqlens_q=_i32([0, 1, 2]), cu_seqlens_k=cu, scale=scale)
    ql = torch.einsum("nthd,hdc->nthc", q[..., :Dn].double(), up_k.double()).float().contiguous()
    o2, lse2 = kda.mla_step_mx(ql, q[..., Dn:], cache, table, _i32(lens), scale)
    o2 = torch.einsum("nthc,hdc->nthd", o2.double(), up_v.double())
    # both are a float32 attention of inputs rounded to float32 once (a few 2^-24 each, over 512 channels)
    assert torch.allclose(o1[0].double(), o2[:, 0], atol=2e-4, rtol=0)
    assert torch.allclose(lse1[0].t(), lse2[:, 0], atol=2e-4, rtol=0)


def test_decode_in_a_graph():
    """Write, attention, weights and eviction captured once, replayed as lengths grow and shrink, with eager work and
    synchronizations between; a second graph of another batch shares no workspace."""
    H, Dc, Dr, N, page = 12, 512, 64, 4, 16
    g = torch.Generator(device="cuda").manual_seed(84)
    state = []
    for k in range(2):
        cache, table, _ = _cache([80, 100, 0, 33], page, Dc, Dr, BF16, 85 + k, spare=30)
        full = torch.randperm(cache.shape[0], generator=g, device="cuda").to(torch.int32)[:N * 8].view(N, 8).contiguous()
        cache = kda.mla_cache_mx(cache.shape[0], page, Dc, Dr, BF16)
        x = _rand(g, BF16, 1, 213, Dc), _rand(g, BF16, 1, 213, Dr)
        kda.mla_cache_append_mx(*x, cache, full, _i32([0] * N), cu_seqlens=_i32([0, 80, 180, 180, 213]))
        s = {"cache": cache, "table": full, "n": _i32([80, 100, 0, 33]), "w": _weights(g, N, 8 * page),
             "c": _rand(g, BF16, N, 1, Dc), "r": _rand(g, BF16, N, 1, Dr)}
        s["ql"], s["qr"] = _queries(N, 1, H, Dc, Dr, BF16, 86 + k)
        s["out"], s["lse"] = torch.empty(N, 1, H, Dc, dtype=BF16, device="cuda"), torch.empty(N, 1, H, device="cuda")
        s["ws"] = torch.empty(kda.mla_step_mx_workspace_bytes(N, 1, H, Dc, page, 8, BF16), dtype=torch.uint8, device="cuda")
        s["we"] = torch.empty(kda.mla_evict_workspace_bytes(N, page, 8), dtype=torch.uint8, device="cuda")
        state.append(s)

    def step(s):
        kda.mla_evict(s["cache"], s["table"], s["n"], s["w"], 60, first=3, recent=10, workspace=s["we"])
        kda.mla_cache_append_mx(s["c"], s["r"], s["cache"], s["table"], s["n"])
        s["n"].add_(1)
        kda.mla_step_mx(s["ql"], s["qr"], s["cache"], s["table"], s["n"], 0.07, out=s["out"], lse=s["lse"], workspace=s["ws"])
        kda.mla_weigh(s["ql"], s["qr"], s["cache"], s["table"], s["n"], s["lse"], 0.07, s["w"])

    graphs = []
    for s in state:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(s)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(s)
        graphs.append(graph)
    for i in range(20):
        s = state[i % 2]
        s["c"].copy_(_rand(g, BF16, N, 1, Dc))
        s["ql"].copy_(_rand(g, BF16, N, 1, H, Dc, std=0.7))
        twin = {k: v.clone() for k, v in s.items()}
        graphs[i % 2].replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        step(twin)
        for k in ("cache", "table", "n", "out", "lse", "w"):
            assert torch.equal(s[k], twin[k]), (i, k)


def test_calls_on_two_streams_at_once():
    lens = [400, 90]
    cache, table, rows = _cache(lens, 32, 512, 64, BF16, 90)
    ql, qr = _queries(2, 1, 96, 512, 64, BF16, 91)
    want = kda.mla_step_mx(ql, qr, cache, table, _i32(lens), 0.07)
    n = _i32(lens)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(kda.mla_step_mx(ql, qr, cache, table, n, 0.07))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_binding_refuses_wrong_tensors():
    lens = [40]
    cache, table, _ = _cache(lens, 16, 512, 64, BF16, 92)
    ql, qr = _queries(1, 1, 4, 512, 64, BF16, 93)
    n, w = _i32(lens), torch.zeros(1, table.shape[1] * 16, device="cuda")
    lse = torch.zeros(1, 1, 4, device="cuda")
    with pytest.raises(ValueError, match="bytes"):
        kda.mla_step_mx(ql, None, cache, table, n, 0.1)
    with pytest.raises(TypeError, match="cache has dtype"):
        kda.mla_step_mx(ql, qr, cache.float(), table, n, 0.1)
    with pytest.raises(TypeError, match="cache has dtype"):
        kda.mla_step(ql, qr, cache, table, n, 0.1)
    with pytest.raises(ValueError, match="weights has shape"):
        kda.mla_weigh(ql, qr, cache, table, n, lse, 0.1, w[:, 1:])
    with pytest.raises(ValueError, match="lse has shape"):
        kda.mla_weigh(ql, qr, cache, table, n, lse[0], 0.1, w)
    with pytest.raises(kda.KDAError, match="decay"):
        kda.mla_weigh(ql, qr, cache, table, n, lse, 0.1, w, decay=2.0)
    with pytest.raises(kda.KDAError, match="keep"):
        kda.mla_evict(cache, table, n, w, -1)
    with pytest.raises(ValueError, match="not those of a 4-bit cache"):
        kda.mla_evict(cache[..., :300].contiguous(), table, n, w, 1)
    with pytest.raises(TypeError, match="out\\[1\\]"):
        kda.mla_evict(cache, table, n, w, 1, out=(table.clone(), n.float(), w.clone()))
    with pytest.raises(ValueError, match="bytes"):
        kda.mla_cache_read_mx(cache, table, _i32([0, 1]), 1, 256, BF16)
    with pytest.raises(ValueError, match="workspace"):
        kda.mla_evict(cache, table, n, w, 1, workspace=torch.empty(8, device="cuda"))
