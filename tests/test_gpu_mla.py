"""Latent attention on the GPU against 64 bits (tests/mla_ref.py, whose bounds
follow from the kernels' roundings), its edges, and its pieces run together."""
import math

import pytest
import torch

import gated_delta_rule_chunk_amd as kda
from gated_delta_rule_chunk_amd import autograd
from tests import mla_ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
DIMS = [(128, 64), (128, 0), (64, 64), (64, 0)]


def _rand(g, dtype, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _make(lens, H, Dn, Dr, dtype, seed, tail=0, grad=False):
    """Packed inputs of sequences of (Lq, Lk) rows, `tail` rows behind them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    Tq, Tk = sum(a for a, _ in lens) + tail, sum(b for _, b in lens) + tail
    q, kv = _rand(g, dtype, 1, Tq, H, Dn + Dr), _rand(g, dtype, 1, Tk, H, 2 * Dn)
    kr = _rand(g, dtype, 1, Tk, 3 * Dr)[..., Dr:2 * Dr] if Dr else None      # a slice of wider rows
    d_o = _rand(g, dtype, 1, Tq, H, Dn) if grad else None
    cu = [torch.tensor([0] + [sum(x[w] for x in lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32,
                       device="cuda") for w in (0, 1)]
    return q, kv, kr, d_o, cu[0], cu[1]


def _both(q, kv, kr, d_o, cuq, cuk, lens, causal, scale=None):
    """Forward and backward, checked; returns the outputs."""
    o, lse = kda.mla_fwd(q, kv, kr, cuq, cuk, causal=causal, scale=scale)
    dq, dkv, dkr = kda.mla_bwd(q, kv, kr, o, lse, d_o, cuq, cuk, causal=causal, scale=scale)
    ref = mla_ref.expanded(q, kv, kr, lens, causal, scale or q.shape[-1] ** -0.5, d_o)
    got = {"o": o, "lse": lse, "dq": dq, "dkv": dkv}
    if kr is not None:
        got["dk_rope"] = dkr
    for name, x in got.items():
        mla_ref.check(name, x, ref[name])
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dn,Dr", DIMS)
@pytest.mark.parametrize("Lq,Lk,causal", [(1, 1, True), (1, 65, True), (33, 33, True), (64, 64, False), (130, 257, True),
                                          (200, 129, True), (129, 40, False), (31, 0, True), (300, 300, True)])
def test_one_sequence(dtype, Dn, Dr, Lq, Lk, causal):
    lens = [(Lq, Lk)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 3, Dn, Dr, dtype, 1 + Lq, grad=True)
    packed = _both(q, kv, kr, d_o, cuq, cuk, lens, causal)
    dense = _both(q, kv, kr, d_o, None, None, lens, causal)
    for name in packed:
        assert torch.equal(packed[name], dense[name]), name


@pytest.mark.parametrize("dtype,H,Dn,Dr", [(BF16, 5, 128, 64), (BF16, 96, 64, 0), (F32, 2, 128, 64)])
def test_packed_ragged(dtype, H, Dn, Dr):
    lens = [(0, 0), (1, 1), (65, 65), (0, 9), (127, 300), (7, 0), (128, 128), (64, 20), (0, 0), (257, 257)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, H, Dn, Dr, dtype, 7, grad=True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, False, scale=0.3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dn,Dr", DIMS)
def test_many_heads(dtype, Dn, Dr):
    """Enough workgroups that the tiles are shared by a workgroup's waves (the
    tests of few heads run the split kernels)."""
    lens = [(130, 257), (100, 60), (1, 1), (64, 64), (0, 3)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 61, Dn, Dr, dtype, 15, tail=3, grad=True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, False)


def test_many_short_sequences():
    """More sequences than a wave's lanes: the tile search takes several steps."""
    lens = [(i % 5, i % 5 + i % 3) for i in range(200)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 2, 128, 64, BF16, 8, grad=True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dense_batch(dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    B, Tq, Tk, H = 3, 70, 150, 4
    q, kv, d_o = _rand(g, dtype, B, Tq, H, 192), _rand(g, dtype, B, Tk, H, 256), _rand(g, dtype, B, Tq, H, 128)
    kr = _rand(g, dtype, B, Tk + 2, 128)[:, 1:-1, 64:]           # strided over batches too
    o, lse = kda.mla_fwd(q, kv, kr)
    grads = kda.mla_bwd(q, kv, kr, o, lse, d_o)
    for b in range(B):
        s = slice(b, b + 1)
        ref = mla_ref.expanded(q[s], kv[s], kr[s], [(Tq, Tk)], True, 192 ** -0.5, d_o[s])
        for name, x in zip(("o", "lse", "dq", "dkv", "dk_rope"), (o, lse) + grads):
            mla_ref.check(name, x[s], ref[name])


def test_large_scores_and_long_rows():
    """Scores of several hundred (every other exponential underflows) and a row of 5000 keys."""
    lens = [(40, 5000), (3, 3)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 2, 128, 64, BF16, 5, grad=True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, True, scale=20.0)
    lens = [(300, 300)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 2, 128, 64, F32, 6, grad=True)
    _both(q, kv, kr, d_o, cuq, cuk, lens, True, scale=2.0)


def test_rows_behind_the_last_sequence():
    lens = [(60, 60), (0, 0), (75, 75)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 4, 128, 64, BF16, 9, tail=140, grad=True)
    n = 135
    for t in (q, kv, d_o):
        t[:, n:] = float("nan")
    kr[:, n:] = float("inf")
    got = _both(q, kv, kr, d_o, cuq, cuk, lens, True)            # fresh outputs: zeros there
    assert all(int(got[x][:, n:].count_nonzero()) == 0 for x in ("o", "dq", "dkv", "dk_rope"))
    out, lse = torch.full_like(got["o"], 7.0), torch.full_like(got["lse"], 7.0)
    kda.mla_fwd(q, kv, kr, cuq, cuk, out=out, lse=lse)
    assert torch.equal(out[:, :n], got["o"][:, :n]) and bool((out[:, n:] == 7).all())
    assert torch.equal(lse[..., :n], got["lse"][..., :n]) and bool((lse[..., n:] == 7).all())
    grads = [torch.full_like(got[x], 7.0) for x in ("dq", "dkv", "dk_rope")]
    kda.mla_bwd(q, kv, kr, out, lse, d_o, cuq, cuk, dq=grads[0], dkv=grads[1], dk_rope=grads[2])
    for x, y in zip(grads, (got["dq"], got["dkv"], got["dk_rope"])):
        assert torch.equal(x[:, :n], y[:, :n]) and bool((x[:, n:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dn,Dr", DIMS)
def test_backward_in_parts(dtype, Dn, Dr):
    """Few workgroups and long walks: several workgroups share a block, and their results are summed."""
    lens = [(1100, 1100), (0, 0), (40, 650), (33, 20)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 1, Dn, Dr, dtype, 19, tail=70, grad=True)
    nq, nk = 1173, 1770
    for t, n in ((q, nq), (d_o, nq), (kv, nk)) + (((kr, nk),) if Dr else ()):
        t[:, n:] = float("nan")
    got = _both(q, kv, kr, d_o, cuq, cuk, lens, True)
    names = ["dq", "dkv"] + (["dk_rope"] if Dr else [])
    o, lse = kda.mla_fwd(q, kv, kr, cuq, cuk)
    grads = {x: torch.full_like(got[x], 7.0) for x in names}
    kda.mla_bwd(q, kv, kr, o, lse, d_o, cuq, cuk, **grads)
    for x in names:
        n = nq if x == "dq" else nk
        assert int(got[x][:, n:].count_nonzero()) == 0
        assert torch.equal(grads[x][:, :n], got[x][:, :n]) and bool((grads[x][:, n:] == 7).all())
    lens = [(1100, 1100)]
    _both(q[:, :1100].clone(), kv[:, :1100].clone(), None if kr is None else kr[:, :1100], d_o[:, :1100].clone(), None,
          None, lens, False)


def _gradients_with_exact_d(q, k, v, d_o, scale, limit):
    """dq, dk of one head in 64 bits, and how far they may be off where D_i = sum_j p_ij dp_ij carries no rounding
    to bf16: mla_ref.attend's bounds without the term of the rounded o, and with the float32 roundings of D's
    own terms and sum instead."""
    f, h, u = torch.float64, mla_ref.H32, mla_ref.half_step(BF16)
    q, k, v, d = q.to(f), k.to(f), v.to(f), d_o.to(f)
    E, n = v.shape[-1], (q.shape[0] + k.shape[0] + 8) * h
    seen = torch.arange(k.shape[0], device=q.device)[None] < limit[:, None]
    s = (q @ k.t() * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - lse)
    mag = (q.abs() @ k.abs().t()) * scale
    err = torch.where(seen, (q.shape[-1] + 4) * h * mag + 4 * h * s.abs(), 0.0)
    rel = err.amax(-1, keepdim=True) + 4 * h * lse.abs() + 8 * h
    dp, dpm = d @ v.t(), d.abs() @ v.abs().t()
    delta = (p * dp).sum(-1, keepdim=True)
    size = dp.abs() + 2 * delta.abs()
    term = (4 * rel + 4 * h) * size + (E + 4) * h * dpm
    be = (p * (term + n * size)).sum(-1, keepdim=True) * 2
    ds = p * (dp - delta)
    bds = (p * (term + be) * (1 + 4 * rel) + u * ds.abs()) * (1 + u)
    dq, dk, dsa = scale * (ds @ k), scale * (ds.t() @ q), ds.abs() + bds
    return {"dq": (dq, scale * (bds @ k.abs() + n * (dsa @ k.abs())) + u * dq.abs()),
            "dk": (dk, scale * (bds.t() @ q.abs() + n * (dsa.t() @ q.abs())) + u * dk.abs())}


@pytest.mark.parametrize("Dn,Dr", DIMS)
@pytest.mark.parametrize("H,lens,scale", [(3, [(2, 2), (33, 33), (128, 128), (60, 128), (7, 3), (100, 120)], 0.5),
                                          (61, [(2, 2), (65, 65), (128, 128), (130, 130), (1, 90)], 0.5),
                                          (3, [(300, 300), (129, 400)], 0.7), (61, [(300, 300), (129, 400)], 0.7)])
def test_backward_forms_d_itself(Dn, Dr, H, lens, scale):
    """Where one key has nearly all of a row's weight, the row's gradient is small beside its D, and D from o as
    it was rounded to bf16 would be off by as much as the gradient. dk (and dk_rope with one head) never goes by
    it, dq does not in tiles of up to 128 keys."""
    q, kv, kr, d_o, cuq, cuk = _make(lens, H, Dn, Dr, BF16, 30, grad=True)
    o, lse = kda.mla_fwd(q, kv, kr, cuq, cuk, scale=scale)
    dq, dkv, _ = kda.mla_bwd(q, kv, kr, o, lse, d_o, cuq, cuk, scale=scale)
    a = b = 0
    for Lq, Lk in lens:
        rq, rk = slice(a, a + Lq), slice(b, b + Lk)
        i = torch.arange(max(0, Lq - Lk), Lq, device="cuda")          # rows before see nothing
        for h in (0, H - 1):
            k = kv[0, rk, h, :Dn] if kr is None else torch.cat((kv[0, rk, h, :Dn], kr[0, rk]), -1)
            ref = _gradients_with_exact_d(q[0, rq, h][i], k, kv[0, rk, h, Dn:], d_o[0, rq, h][i], scale,
                                          i + Lk - Lq + 1)
            if Lk <= 128:
                mla_ref.check(f"dq {Lq} {Lk} {h}", dq[0, rq, h][i], ref["dq"])
            mla_ref.check(f"dk {Lq} {Lk} {h}", dkv[0, rk, h, :Dn], tuple(x[:, :Dn] for x in ref["dk"]))
        a, b = a + Lq, b + Lk


def test_nan_in_a_hidden_key_stays_hidden():
    lens = [(100, 100)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 2, 128, 64, BF16, 10, grad=True)
    o, lse = kda.mla_fwd(q, kv, kr)
    kv[:, 70, :, :128] = float("nan")
    kr[:, 71] = float("inf")
    o2, lse2 = kda.mla_fwd(q, kv, kr)
    assert torch.equal(o[:, :70], o2[:, :70]) and torch.equal(lse[..., :70], lse2[..., :70])
    assert bool(torch.isnan(o2[:, 70:]).all())


def test_same_bits_again_and_on_another_stream():
    lens = [(500, 500), (77, 90)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 6, 128, 64, BF16, 11, grad=True)
    one = _both(q, kv, kr, d_o, cuq, cuk, lens, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = kda.mla_fwd(q, kv, kr, cuq, cuk)
        grads = kda.mla_bwd(q, kv, kr, o, lse, d_o, cuq, cuk)
    s.synchronize()
    for name, x in zip(("o", "lse", "dq", "dkv", "dk_rope"), (o, lse) + grads):
        assert torch.equal(one[name], x), name


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_autograd_equals_the_calls(dtype):
    lens = [(50, 80), (33, 33)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 3, 128, 64, dtype, 12, tail=5, grad=True)
    o, lse = kda.mla_fwd(q, kv, kr, cuq, cuk)
    want = kda.mla_bwd(q, kv, kr, o, lse, d_o, cuq, cuk)
    leaves = [x.detach().requires_grad_() for x in (q, kv, kr)]
    y = autograd.mla(*leaves, cu_seqlens_q=cuq, cu_seqlens_k=cuk)
    # an incoming gradient that is not contiguous
    wide = torch.stack((d_o, d_o), -1)
    got = torch.autograd.grad(y, leaves, wide[..., 0])
    assert torch.equal(y.detach(), o)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """Central differences of the 64-bit forward along random directions. The
    float32 gradient is within its bound of the true one, so its product with a
    direction is within the bound's product with the direction's magnitude; the
    difference quotient adds a term of third order in the step."""
    lens = [(40, 60)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 2, 64, 64, F32, 13, grad=True)
    o, lse = kda.mla_fwd(q, kv, kr)
    grads = kda.mla_bwd(q, kv, kr, o, lse, d_o)
    ref = mla_ref.expanded(q, kv, kr, lens, True, 128 ** -0.5, d_o)

    def loss(x, y, z):
        return (mla_ref.expanded(x, y, z, lens, True, 128 ** -0.5)["o"][0] * d_o.double()).sum().item()

    at = [x.double() for x in (q, kv, kr)]
    g = torch.Generator(device="cuda").manual_seed(14)
    for i, name in enumerate(("dq", "dkv", "dk_rope")):
        d = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        quot = []
        for h in (1e-4, 2e-4):
            lo, hi = list(at), list(at)
            lo[i], hi[i] = at[i] - h * d, at[i] + h * d
            quot.append((loss(*hi) - loss(*lo)) / (2 * h))
        slack = abs(quot[1] - quot[0]) + 1e-9 * sum(abs(x) for x in quot)     # a third of it is the error of the first
        have = (grads[i].double() * d).sum().item()
        assert abs(have - quot[0]) <= slack + (ref[name][1] * d.abs()).sum().item(), name


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_past_31_bits_and_largest_strides(dtype):
    """q, kv and their gradients of over 2^31 elements, with the most heads and the widest rows of k_rope that
    are supported. The first and the last head against 64 bits; the incoming gradient of the others is zero, so
    that the sum over the heads is these two's."""
    H, Tq, Tk, row = 4096, 2800, 2200, 1 << 22
    g = torch.Generator(device="cuda").manual_seed(24)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    q, kv = rand(1, Tq, H, 192), rand(1, Tk, H, 256)
    assert q.numel() > 1 << 31 and kv.numel() > 1 << 31
    kr = torch.empty((Tk - 1) * row + 64, dtype=dtype, device="cuda").as_strided((1, Tk, 64), (row * Tk, row, 1))
    kr.copy_(rand(1, Tk, 64))
    ends = [0, H - 1]
    d_o = torch.zeros(1, Tq, H, 128, dtype=dtype, device="cuda")
    d_o[:, :, ends] = rand(1, Tq, 2, 128)
    o, lse = kda.mla_fwd(q, kv, kr)
    dq, dkv, dkr = kda.mla_bwd(q, kv, kr, o, lse, d_o)
    ref = mla_ref.expanded(q[:, :, ends], kv[:, :, ends], kr, [(Tq, Tk)], True, 192 ** -0.5, d_o[:, :, ends])
    for name, x in (("o", o[:, :, ends]), ("lse", lse[:, ends]), ("dq", dq[:, :, ends]), ("dkv", dkv[:, :, ends]),
                    ("dk_rope", dkr)):
        mla_ref.check(name, x, ref[name])
    assert int(dq[:, :, 1:-1].count_nonzero()) == 0 and int(dkv[:, :, 1:-1].count_nonzero()) == 0
    del q, kv, kr, d_o, o, lse, dq, dkv, dkr, ref
    torch.cuda.empty_cache()


# ---- cache ------------------------------------------------------------------------------------------------------


def _cache(lens, page, Dc, Dr, dtype, seed, spare=2, n_pages=None):
    """A cache of pages in random order that holds `lens` rows per sequence, everything else NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    total = sum(need) + spare if n_pages is None else n_pages
    cache = torch.full((total, page, Dc + Dr), float("nan"), dtype=dtype, device="cuda")
    order = torch.randperm(total, generator=g, device="cuda").cpu()
    if n_pages is not None:
        order = order.sort(descending=True).values
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    rows = []
    for i, n in enumerate(lens):
        table[i, :need[i]] = order[at:at + need[i]].int()
        x = _rand(g, dtype, max(n, 0), Dc + Dr)
        for k in range(need[i]):
            part = x[k * page:(k + 1) * page]
            cache[order[at + k], :part.shape[0]] = part
        at += need[i]
        rows.append(x)
    return cache, table.cuda(), rows


def _check_step(q_lat, q_rope, rows, o, lse, scale, lens, seen=None):
    Nb, T, H, Dc = q_lat.shape
    for b in range(Nb):
        n = max(lens[b], 0)
        x = q_lat[b] if q_rope is None else torch.cat((q_lat[b], q_rope[b]), -1)
        t = torch.arange(T, device="cuda").repeat_interleave(H)
        limit = (n - T + t + 1).clamp(0, n)
        k = rows[b][None]
        r = mla_ref.attend(x.reshape(1, T * H, -1), k, k[..., :Dc], scale, limit, dtype=q_lat.dtype)
        mla_ref.check(f"o[{b}]", o[b].reshape(1, T * H, Dc), r["o"])
        mla_ref.check(f"lse[{b}]", lse[b].reshape(1, T * H), r["lse"])


def _queries(Nb, T, H, Dc, Dr, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ql = _rand(g, dtype, H, Nb, T, Dc, std=0.7).permute(1, 2, 0, 3)          # head-major
    qr = _rand(g, dtype, Nb, T, H, 128 + Dr)[..., 128:] if Dr else None      # a slice of wider heads
    return ql, qr


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dc,Dr", [(512, 64), (512, 0), (256, 64), (256, 0)])
@pytest.mark.parametrize("H,T,page", [(1, 1, 16), (33, 1, 64), (96, 1, 32), (130, 1, 128), (16, 5, 16), (40, 3, 64)])
def test_step(dtype, Dc, Dr, H, T, page):
    lens = [0, 1, 31, 32, 33, -1, 130, 257, 16, 2]
    cache, table, rows = _cache(lens, page, Dc, Dr, dtype, H + T)
    ql, qr = _queries(len(lens), T, H, Dc, Dr, dtype, 2)
    o, lse = kda.mla_step(ql, qr, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=0.06)
    _check_step(ql, qr, rows, o, lse, 0.06, lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[5000], [700, 3000, 33, 0, 1201], [100] * 90])
def test_step_split_over_the_cache(dtype, lens):
    cache, table, rows = _cache(lens, 64, 512, 64, dtype, 4)
    ql, qr = _queries(len(lens), 1, 12, 512, 64, dtype, 5)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = kda.mla_step(ql, qr, cache, table, n, scale=0.07)
    _check_step(ql, qr, rows, o, lse, 0.07, lens)
    again = kda.mla_step(ql, qr, cache, table, n, scale=0.07)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dc,Dr", [(512, 64), (512, 0), (256, 64), (256, 0)])
@pytest.mark.parametrize("H", [64, 96, 128])
def test_step_wide_workgroups(dtype, Dc, Dr, H):
    """A cache long enough that all rows of queries that fit share a workgroup: four, six and eight waves."""
    lens = [2900, 31, 1000]
    cache, table, rows = _cache(lens, 64, Dc, Dr, dtype, H)
    ql, qr = _queries(3, 1, H, Dc, Dr, dtype, 3)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = kda.mla_step(ql, qr, cache, table, n, scale=0.06)
    _check_step(ql, qr, rows, o, lse, 0.06, lens)


@pytest.mark.parametrize("H,tiles", [(4, 8), (4, 9), (96, 8), (96, 9)])
def test_step_few_and_many_parts(H, tiles):
    """Sequences of one tile a part: joined by a wave each up to eight parts, by four together beyond."""
    lens = [32 * tiles, 32 * tiles - 31]
    cache, table, rows = _cache(lens, 32, 512, 64, BF16, tiles)
    ql, qr = _queries(2, 1, H, 512, 64, BF16, 8)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = kda.mla_step(ql, qr, cache, table, n, scale=0.07)
    _check_step(ql, qr, rows, o, lse, 0.07, lens)


def test_step_parts_of_more_pages_than_lanes():
    """Parts of over 64 pages of 16 rows read the page table in pieces; a page that does not exist in any
    of them is hidden and counted once."""
    lens = [6500 + 41 * i for i in range(40)]
    cache, table, rows = _cache(lens, 16, 256, 64, BF16, 20)
    assert sum(-(-n // 32) for n in lens) > 256 * 32
    ql, qr = _queries(len(lens), 1, 3, 256, 64, BF16, 21)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = kda.mla_step(ql, qr, cache, table, n, scale=0.08)
    _check_step(ql, qr, rows, o, lse, 0.08, lens)
    bad = table.clone()
    bad[::2, 63], bad[1::2, 64], bad[:, 300] = -1, cache.shape[0], -7
    o, lse = kda.mla_step(ql, qr, cache, bad, n, scale=0.08)
    with pytest.raises(kda.KDAError, match="80 counted"):
        kda.device_check()
    hidden = torch.zeros(max(lens), dtype=torch.bool, device="cuda")
    hidden[4800:4816] = True
    for b, x in enumerate(rows):
        gone = hidden[:lens[b]].clone()
        gone[(63 + b % 2) * 16:(64 + b % 2) * 16] = True
        _check_step(ql[b:b + 1], qr[b:b + 1], [x[~gone]], o[b:b + 1], lse[b:b + 1], 0.08, [int((~gone).sum())])


def test_step_large_scores():
    lens = [900]
    cache, table, rows = _cache(lens, 64, 512, 64, BF16, 14)
    ql, qr = _queries(1, 1, 96, 512, 64, BF16, 15)
    o, lse = kda.mla_step(ql, qr, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=5.0)
    _check_step(ql, qr, rows, o, lse, 5.0, lens)


def test_step_cache_past_four_gib():
    """Page offsets past 2^32 bytes."""
    lens = [300, 45]
    cache, table, rows = _cache(lens, 256, 512, 64, BF16, 6, n_pages=16000)
    assert int(table.max()) * 256 * 576 * 2 > 1 << 32
    ql, qr = _queries(2, 1, 8, 512, 64, BF16, 7)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = kda.mla_step(ql, qr, cache, table, n, scale=0.07)
    _check_step(ql, qr, rows, o, lse, 0.07, lens)
    new = torch.ones(2, 1, 576, dtype=BF16, device="cuda")
    kda.mla_cache_append(new[..., :512], new[..., 512:], cache, table, n - 1)
    for b in range(2):
        assert bool((cache[table[b, (lens[b] - 1) // 256].item(), (lens[b] - 1) % 256] == 1).all())


@pytest.mark.parametrize("page", [16, 32])
def test_missing_pages_are_reported(page):
    lens = [100, 70, 40]
    cache, table, rows = _cache(lens, page, 512, 64, BF16, 8)
    ql, qr = _queries(3, 1, 8, 512, 64, BF16, 9)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bad = table.clone()
    bad[0, 1] = cache.shape[0]
    bad[1, 0] = -1
    o, lse = kda.mla_step(ql, qr, cache, bad, n, scale=0.07)
    with pytest.raises(kda.KDAError, match="2 counted"):
        kda.device_check()
    kda.device_check()
    # the rest of the sequence is attended to
    keep = [torch.cat((rows[0][:page], rows[0][2 * page:])), rows[1][page:], rows[2]]
    _check_step(ql, qr, keep, o, lse, 0.07, [x.shape[0] for x in keep])
    # a length past the page table: what the table holds
    o, lse = kda.mla_step(ql, qr, cache, table, torch.tensor([100, 70, 10 ** 6], dtype=torch.int32, device="cuda"),
                          scale=0.07)
    with pytest.raises(kda.KDAError, match="page table"):
        kda.device_check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,page", [(4, 16), (3, 32), (5, 64)])
def test_length_past_the_page_table_hides_its_rows_only(dtype, T, page):
    """Each token sees what it sees by the length given, of the rows that the table holds."""
    cap, H = 3 * page, 7
    lens = [cap, cap + 1, cap + T - 1, cap + 50, 10 ** 9, cap - 1]
    cache, table, rows = _cache([cap] * len(lens), page, 256, 64, dtype, 22)
    ql, qr = _queries(len(lens), T, H, 256, 64, dtype, 23)
    o, lse = kda.mla_step(ql, qr, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=0.07)
    with pytest.raises(kda.KDAError, match="4 counted"):
        kda.device_check()
    t = torch.arange(T, device="cuda").repeat_interleave(H)
    for b, n in enumerate(lens):
        k = rows[b][None]
        r = mla_ref.attend(torch.cat((ql[b], qr[b]), -1).reshape(1, T * H, -1), k, k[..., :256], 0.07,
                           (n - T + t + 1).clamp(0, cap), dtype=dtype)
        mla_ref.check(f"o[{b}]", o[b].reshape(1, T * H, 256), r["o"])
        mla_ref.check(f"lse[{b}]", lse[b].reshape(1, T * H), r["lse"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dc,Dr,page", [(512, 64, 16), (256, 0, 64)])
@pytest.mark.parametrize("packed", [False, True])
def test_append(dtype, Dc, Dr, page, packed):
    before = [0, 15, -1, 16, 63, 100]
    new = [3, 1, 2, 0, 70, 17] if packed else [3] * 6
    total = [max(a, 0) + b for a, b in zip(before, new)]
    cache, table, _ = _cache(total, page, Dc, Dr, dtype, 10)
    want = cache.clone()
    g = torch.Generator(device="cuda").manual_seed(11)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    shape = (1, cu[-1] + 4) if packed else (6, 3)                # packed: four tokens behind the last sequence
    lat = _rand(g, dtype, *shape, Dc + 64)[..., 32:32 + Dc]
    kr = _rand(g, dtype, *shape, 2 * Dr)[..., Dr:] if Dr else None
    lens = torch.tensor(before, dtype=torch.int32, device="cuda")
    kda.mla_cache_append(lat, kr, cache, table, lens,
                         cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None)
    for n in range(6):
        for t in range(new[n] if before[n] >= 0 else 0):
            at = (0, cu[n] + t) if packed else (n, t)
            row = lat[at] if kr is None else torch.cat((lat[at], kr[at]))
            p = before[n] + t
            want[table[n, p // page].item(), p % page] = row
    assert torch.equal(torch.nan_to_num(cache.float(), nan=9e9), torch.nan_to_num(want.float(), nan=9e9))


def test_append_past_the_table_is_reported():
    cache, table, _ = _cache([32, 32], 16, 256, 0, BF16, 12)
    want = cache.clone()
    new = torch.ones(2, 1, 256, dtype=BF16, device="cuda")
    table[1, 1] = cache.shape[0]
    kda.mla_cache_append(new, None, cache, table, torch.tensor([32, 20], dtype=torch.int32, device="cuda"))
    with pytest.raises(kda.KDAError, match="2 counted"):
        kda.device_check()
    assert torch.equal(torch.nan_to_num(cache.float(), nan=9e9), torch.nan_to_num(want.float(), nan=9e9))


def test_prefill_then_decode_equals_the_expanded_form():
    """Prompts through mla_fwd with their latents appended, then tokens one by
    one through the absorbed form; a whole pass of mla_fwd over all tokens says
    what they should be. float32, where the two forms differ by the rounding of
    the absorbing products only: sums of at most 512 terms of magnitude about
    as large as their result, so 1e-4 of the outputs' size is wide."""
    H, Dn, Dr, Dc, page = 8, 128, 64, 512, 16
    g = torch.Generator(device="cuda").manual_seed(20)
    prompts, steps = [37, 1, 90], 5
    N = len(prompts)
    w_uk = _rand(g, F32, H, Dn, Dc, std=Dc ** -0.5)              # k = w_uk c
    w_uv = _rand(g, F32, H, Dc, Dn, std=Dc ** -0.5)              # v = c w_uv
    total = [p + steps for p in prompts]
    c = [_rand(g, F32, n, Dc) for n in total]
    r = [_rand(g, F32, n, Dr) for n in total]
    q = [_rand(g, F32, n, H, Dn + Dr) for n in total]
    scale = (Dn + Dr) ** -0.5

    def kv_of(x):
        k = torch.matmul(x[None], w_uk.transpose(1, 2).contiguous()).transpose(0, 1)
        return torch.cat((k, torch.matmul(x[None], w_uv).transpose(0, 1)), -1).contiguous()

    cu = torch.tensor([0] + [sum(total[:i + 1]) for i in range(N)], dtype=torch.int32, device="cuda")
    want, _ = kda.mla_fwd(torch.cat(q)[None], torch.cat([kv_of(x) for x in c])[None].contiguous(), torch.cat(r)[None],
                          cu, cu)
    # prefill
    cu = torch.tensor([0] + [sum(prompts[:i + 1]) for i in range(N)], dtype=torch.int32, device="cuda")
    cut = lambda xs: torch.cat([x[:p] for x, p in zip(xs, prompts)])[None]  # noqa: E731
    o, _ = kda.mla_fwd(cut(q), torch.cat([kv_of(x[:p]) for x, p in zip(c, prompts)])[None].contiguous(), cut(r), cu, cu)
    cache = torch.full((20, page, Dc + Dr), float("nan"), device="cuda")
    table = torch.randperm(20, generator=g, device="cuda")[:18].int().view(3, 6).contiguous()
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")
    kda.mla_cache_append(cut(c), cut(r), cache, table, lens, cu_seqlens=cu)
    lens += torch.tensor(prompts, dtype=torch.int32, device="cuda")
    got = [[o[0, cu[n]:cu[n + 1]]] for n in range(N)]
    for t in range(steps):
        at = lambda xs: torch.stack([x[p + t] for x, p in zip(xs, prompts)])[:, None]  # noqa: E731
        kda.mla_cache_append(at(c), at(r), cache, table, lens)
        lens += 1
        qt = at(q)
        ql = torch.matmul(qt[:, 0, :, :Dn].transpose(0, 1).contiguous(), w_uk)              # [H,N,Dc]
        ol, _ = kda.mla_step(ql.transpose(0, 1)[:, None], qt[..., Dn:], cache, table, lens, scale)
        ov = torch.matmul(ol[:, 0].transpose(0, 1).contiguous(), w_uv).transpose(0, 1)      # [N,H,Dn]
        for n in range(N):
            got[n].append(ov[n:n + 1])
    got = torch.cat([torch.cat(x) for x in got])
    err = (got - want[0]).abs().max().item()
    assert err <= 1e-4 * want.abs().max().item(), err


def test_decode_in_a_graph():
    """Cache write and attention captured once, replayed as the lengths grow, eager work in between."""
    H, Dc, Dr, N = 16, 512, 64, 4
    lens = [5, 64, 0, 130]
    cache, table, _ = _cache([n + 8 for n in lens], 32, Dc, Dr, BF16, 16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c, r = torch.zeros(N, 1, Dc, dtype=BF16, device="cuda"), torch.zeros(N, 1, Dr, dtype=BF16, device="cuda")
    ql, qr = _queries(N, 1, H, Dc, Dr, BF16, 17)
    out = torch.empty(N, 1, H, Dc, dtype=BF16, device="cuda")
    lse = torch.empty(N, 1, H, device="cuda")
    ws = torch.empty(kda.mla_step_workspace_bytes(N, 1, H, Dc, 32, table.shape[1], BF16), dtype=torch.uint8, device="cuda")

    def step():
        kda.mla_cache_append(c, r, cache, table, n)
        n.add_(1)
        kda.mla_step(ql, qr, cache, table, n, 0.07, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(18)
    for _ in range(4):
        c.copy_(_rand(g, BF16, N, 1, Dc))
        r.copy_(_rand(g, BF16, N, 1, Dr))
        ql.copy_(_rand(g, BF16, N, 1, H, Dc, std=0.7))
        old, now = cache.clone(), n.clone()
        graph.replay()
        torch.cuda.synchronize()
        kda.mla_cache_append(c, r, old, table, now)
        want = kda.mla_step(ql, qr, old, table, now + 1, 0.07)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(n, now + 1)
        assert torch.equal(torch.nan_to_num(old.float()), torch.nan_to_num(cache.float()))


def test_training_calls_in_a_graph():
    lens = [(130, 130), (20, 20)]
    q, kv, kr, d_o, cuq, cuk = _make(lens, 4, 128, 64, BF16, 19, grad=True)
    out, lse = torch.empty(1, 150, 4, 128, dtype=BF16, device="cuda"), torch.empty(1, 4, 150, device="cuda")
    grads = [torch.empty_like(q), torch.empty_like(kv), torch.empty(1, 150, 64, dtype=BF16, device="cuda")]
    ws = torch.empty(kda.mla_bwd_workspace_bytes(1, 150, 150, 4, 64), dtype=torch.uint8, device="cuda")

    def both():
        kda.mla_fwd(q, kv, kr, cuq, cuk, out=out, lse=lse)
        kda.mla_bwd(q, kv, kr, out, lse, d_o, cuq, cuk, dq=grads[0], dkv=grads[1], dk_rope=grads[2], workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    g = torch.Generator(device="cuda").manual_seed(21)
    for _ in range(3):
        q.copy_(_rand(g, BF16, *q.shape))
        d_o.copy_(_rand(g, BF16, *d_o.shape))
        graph.replay()
        torch.cuda.synchronize()
        o, l = kda.mla_fwd(q, kv, kr, cuq, cuk)
        want = kda.mla_bwd(q, kv, kr, o, l, d_o, cuq, cuk)
        assert torch.equal(out, o) and torch.equal(lse, l)
        assert all(torch.equal(x, y) for x, y in zip(grads, want))


def test_binding_refuses_wrong_tensors():
    q, kv, kr = (torch.zeros(1, 8, 2, d, dtype=BF16, device="cuda") for d in (192, 256, 64))
    kr = kr[:, :, 0]
    with pytest.raises(TypeError, match="kv has dtype"):
        kda.mla_fwd(q, kv.float(), kr)
    with pytest.raises(ValueError, match="kv has shape"):
        kda.mla_fwd(q, kv[:, :, :1].contiguous(), kr)
    with pytest.raises(ValueError, match="q must be contiguous"):
        kda.mla_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), kv, kr)
    with pytest.raises(ValueError, match="last dimension"):
        kda.mla_fwd(q, kv, torch.zeros(1, 64, 8, dtype=BF16, device="cuda").transpose(1, 2))
    with pytest.raises(kda.KDAError, match="16 bytes"):
        kda.mla_fwd(q, kv, torch.zeros(1, 8, 65, dtype=BF16, device="cuda")[..., :64])
    with pytest.raises(kda.KDAError, match="aligned"):
        kda.mla_fwd(q, kv, torch.zeros(1, 8, 72, dtype=BF16, device="cuda")[..., 4:68])
    with pytest.raises(ValueError, match="together"):
        kda.mla_fwd(q, kv, kr, cu_seqlens_q=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="together"):
        kda.mla_fwd(q, kv, kr, out=torch.zeros(1, 8, 2, 128, dtype=BF16, device="cuda"))
    with pytest.raises(TypeError, match="unsupported dtype"):
        kda.mla_fwd(q.half(), kv.half(), kr.half())
    cache, table = torch.zeros(2, 16, 576, dtype=BF16, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    ql = torch.zeros(1, 1, 2, 512, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="channels"):
        kda.mla_step(ql, None, cache, table, lens, 0.1)
    with pytest.raises(TypeError, match="page_table has dtype"):
        kda.mla_step(ql, kr[:, :1, None].expand(1, 1, 2, 64), cache, table.long(), lens, 0.1)
    with pytest.raises(ValueError, match="workspace"):
        kda.mla_step(ql, kr[:, :1, None].expand(1, 1, 2, 64), cache, table, lens, 0.1,
                     workspace=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="channels"):
        kda.mla_cache_append(ql[:, 0, :1], None, cache, table, lens)
    assert math.isfinite(kda.mla_step(ql, kr[:, :1, None].expand(1, 1, 2, 64), cache, table, lens, 0.1)[1].sum().item())
