"""The 4-bit cache of latents, gathered weights and eviction in 64 bits (or exactly), written from the definitions
of include/kda_mla_cache.h, with elementwise bounds on what the kernels may be off.

Besides what tests/mla_ref.py derives, the bf16 scores over 4-bit latents take the query as two 8-bit floats of 4
significant bits, scaled for each 32 channels: channels above 2^-14 of the block's largest are exact, the others
are off by at most 2^-21 of it, so a score by at most SPLIT * scale * sum over blocks of max|q| * sum|c|."""
import math

import torch

from tests import mla_ref
from tests.mla_ref import H32

SPLIT = 2.0 ** -21
GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def power(e):
    """2^e for integers e, exactly (a device's pow need not be)."""
    t = torch.tensor([math.ldexp(1.0, k) for k in range(-200, 200)], dtype=torch.float64, device=e.device)
    return t[e.long() + 200]


def encode(x):
    """[R,Dc] to (codes [R,Dc], scale bytes [R,Dc/32]), by searching the exponents and the nearest multiples."""
    x = x.double().unflatten(1, (-1, 32))
    a = x.abs().amax(-1)
    e = torch.full_like(a, 125)
    for k in range(124, -130, -1):
        e = torch.where(a <= 7 * math.ldexp(1.0, k), torch.full_like(a, k), e)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    d = ((x / power(e)[..., None]).abs()[..., None] - grid).abs()
    near = d == d.amin(-1, keepdim=True)
    pick = torch.where(near, torch.arange(8, device=x.device) % 2, 2).argmin(-1)       # of two as near the even code
    code = pick + 8 * torch.signbit(x)
    bad, none = ~torch.isfinite(a), a < 2.0 ** -100
    code = torch.where((bad | none)[..., None], 0, code)
    return code.flatten(1).to(torch.uint8), torch.where(bad, 255, torch.where(none, 0, e + 127)).to(torch.uint8)


def values(codes, scales):
    """float64 values of codes [R,Dc] and scale bytes [R,Dc/32]."""
    v = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64, device=codes.device)[codes.long()]
    s = scales.double()[..., None]
    f = torch.where(s == 255, float("nan"), torch.where(s == 0, 0.0, power(s - 127)))
    return (v.unflatten(1, (-1, 32)) * f).flatten(1)


def put_page(cache, page, codes, scales, rope):
    """Writes the first rows of a page: codes [R,Dc], scale bytes [R,Dc/32], shared parts [R,Dr] or None."""
    ps, flat, R, Dc = cache.shape[1], cache[page].view(-1), codes.shape[0], codes.shape[1]
    flat[:ps * Dc // 2].view(ps, Dc // 2)[:R] = codes[:, ::2] + 16 * codes[:, 1::2]
    flat[ps * Dc // 2:ps * (Dc // 2 + Dc // 32)].view(ps, Dc // 32)[:R] = scales
    if rope is not None:
        flat[ps * (Dc // 2 + Dc // 32):].view(rope.dtype).view(ps, -1)[:R] = rope


def get_rows(cache, table_row, n, Dc, Dr, dtype):
    """A sequence's first n rows: latents in float64 and shared parts (or None)."""
    ps = cache.shape[1]
    flat = cache[table_row[:-(-n // ps)].long()].flatten(1)
    b = flat[:, :ps * Dc // 2].reshape(-1, Dc // 2)[:n]
    s = flat[:, ps * Dc // 2:ps * (Dc // 2 + Dc // 32)].reshape(-1, Dc // 32)[:n]
    r = flat[:, ps * (Dc // 2 + Dc // 32):].reshape(-1).view(dtype).view(-1, Dr)[:n] if Dr else None
    return values(torch.stack((b % 16, b // 16), -1).flatten(1), s), r


def _split_error(q, k, Dc, scale):
    """[M,n]: what the split of bf16 queries may cost each score."""
    m = q.double()[:, :Dc].unflatten(1, (-1, 32)).abs().amax(-1)
    return SPLIT * scale * m @ k.double()[:, :Dc].unflatten(1, (-1, 32)).abs().sum(-1).t()


def attend(q, c, r, scale, limit, dtype, mx):
    """q [M,D] over rows c [n,Dc], r [n,Dr] or None: {"o", "lse"} as (value, bound)."""
    k = c.double() if r is None else torch.cat((c.double(), r.double()), -1)
    res = mla_ref.attend(q[None], k[None], c.double()[None], scale, limit, dtype=dtype)
    if not mx or dtype != torch.bfloat16 or not k.shape[0]:
        return res
    seen = torch.arange(k.shape[0], device=q.device)[None] < limit[:, None]
    x = 2 * torch.where(seen, _split_error(q, k, c.shape[1], scale), 0.0).amax(-1)
    p = torch.softmax((q.double() @ k.t() * scale).masked_fill(~seen, -1e300), -1) * seen
    o, lse = res["o"], res["lse"]
    return {"o": (o[0], o[1] + 2 * x[None, :, None] * (p @ c.double().abs())[None]), "lse": (lse[0], lse[1] + x[None])}


def gathered(q, c, r, lse, scale, limit, old, decay, dtype, mx):
    """New weights [n] of rows c, r: (value, bound). q [M,D], lse [M], old [n] (0 where it is not read)."""
    k = c.double() if r is None else torch.cat((c.double(), r.double()), -1)
    M, D, n = q.shape[0], q.shape[1], k.shape[0]
    x = q.double()
    s = x @ k.t() * scale
    seen = torch.arange(n, device=q.device)[None] < limit[:, None]
    z = lse.double()[:, None]
    p = torch.where(seen, torch.exp(s - z), 0.0)
    err = (D + 4) * H32 * (x.abs() @ k.abs().t() * scale) + 4 * H32 * (s.abs() + z.abs()) + 8 * H32
    if mx and dtype == torch.bfloat16:
        err = err + _split_error(q, k, c.shape[1], scale)
    err = torch.where(seen, err, 0.0)
    new = p.sum(0)
    kept = decay * old.double()
    return kept + new, (p * torch.expm1(err)).sum(0) + (M + 8) * H32 * new + 3 * H32 * (kept.abs() + new)


def evict(weights, n, page_size, keep, first, recent):
    """What happens to a sequence of n rows: (E, a, b, moves [(to, from)], new order of rows as a list)."""
    ps = page_size
    a, b = -(-first // ps), max(n - recent, 0) // ps
    E = max(0, min((n - keep) // ps if n > keep else 0, b - a))
    if not E:
        return 0, a, b, [], list(range(n))
    key = [float("inf") if w != w else w for w in weights]
    nan = [w != w for w in weights]
    rank = sorted(range(a * ps, b * ps), key=lambda j: (not nan[j], -key[j], j))
    stays = set(rank[:(b - a - E) * ps])
    src = [j for j in range((b - E) * ps, b * ps) if j in stays]
    dst = [j for j in range(a * ps, (b - E) * ps) if j not in stays]
    assert len(src) == len(dst)
    order = list(range(n))
    for d, s in zip(dst, src):
        order[d] = s
    return E, a, b, list(zip(dst, src)), order[:(b - E) * ps] + order[b * ps:]
