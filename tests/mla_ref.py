"""Latent attention in 64 bits, with elementwise bounds on what the kernels may be off.

The bounds follow the kernels' arithmetic. With u = half a step of bf16 (2^-8
relative) or 0 for float32, and h = 2^-24 (half a step of float32):

- a score is a float32 sum of D products, scaled: |error| <= e_ij = (D + 4) h
  scale sum |q||k|, and the exponent's own roundings (argument, maximum or lse)
  add 4 h (|s| + |row maximum|) + 8 h; so p_ij is off by a factor 1 + E with
  E = max_j of these, twice that after division by a sum of such terms;
- p and ds are rounded once more as operands (u);
- sums of n float32 terms add n h times the sum of their magnitudes;
- outputs are rounded once (u, or h).
"""
import math

import torch

H32 = 2.0 ** -24


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 0.0


def attend(q, k, v, scale, limit, d_o=None, dtype=torch.float32):
    """One sequence: q [H,Lq,D], k [H,Lk,D], v [H,Lk,E] (any type), row i sees
    the keys j < limit[i]. Returns {name: (value, bound)} in float64: o, lse and,
    with d_o [H,Lq,E], dq, dk, dv."""
    f = torch.float64
    q, k, v = q.to(f), k.to(f), v.to(f)
    u, D, E, Lq, Lk = half_step(dtype), q.shape[-1], v.shape[-1], q.shape[1], k.shape[1]
    out = u if u else H32
    seen = torch.arange(Lk, device=q.device)[None] < limit[:, None]
    some = seen.any(1)[:, None]
    s = (q @ k.transpose(1, 2)) * scale
    mag = (q.abs() @ k.abs().transpose(1, 2)) * scale
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    safe = torch.where(torch.isfinite(lse), lse, 0.0)[..., None]
    p = torch.where(seen, torch.exp(s - safe), 0.0)
    sa = torch.where(seen, s, 0.0).abs()
    err = torch.where(seen, (D + 4) * H32 * mag + 4 * H32 * sa, 0.0)
    rel = (err.amax(-1, keepdim=True) if Lk else err.sum(-1, keepdim=True)) + \
        4 * H32 * safe.abs() + 8 * H32                                    # E
    o = p @ v
    pv = p @ v.abs()
    bo = (u + 2 * rel + (Lk + 8) * H32) * pv + out * o.abs()
    res = {"o": (o, bo), "lse": (lse, (2 * rel + (Lk + 8) * H32)[..., 0] + 2 * H32 * safe[..., 0].abs())}
    if d_o is None:
        return res
    d = d_o.to(f)
    dp = d @ v.transpose(1, 2)
    dpm = d.abs() @ v.abs().transpose(1, 2)
    delta = (d * o).sum(-1, keepdim=True)
    dm = (d.abs() * o.abs()).sum(-1, keepdim=True)
    # D_i goes through the rounded o: as far off as o's own bound lets it be
    be = (d.abs() * bo).sum(-1, keepdim=True) + (E + 4) * H32 * dm
    ds = p * (dp - delta)
    # p has the rounding of its exponent only here (lse is the forward's float32 value)
    bds = p * (4 * rel + 4 * H32) * (dp.abs() + delta.abs()) + p * ((E + 4) * H32 * dpm + be) * (1 + 4 * rel) + u * ds.abs()
    bds = bds * (1 + u)
    bp = p * (4 * rel + u)
    pd = p.transpose(1, 2) @ d.abs()
    dq, dk, dv = scale * (ds @ k), scale * (ds.transpose(1, 2) @ q), p.transpose(1, 2) @ d
    n = (Lq + Lk + 8) * H32
    dsa = ds.abs() + bds
    res["dq"] = (dq, scale * (bds @ k.abs() + n * (dsa @ k.abs())) + out * dq.abs())
    res["dk"] = (dk, scale * (bds.transpose(1, 2) @ q.abs() + n * (dsa.transpose(1, 2) @ q.abs())) + out * dk.abs())
    res["dv"] = (dv, bp.transpose(1, 2) @ d.abs() + n * pd + out * dv.abs())
    del some
    return res


def expanded(q, kv, k_rope, lens, causal, scale, d_o=None):
    """mla_fwd's (and mla_bwd's) outputs for sequences of (Lq, Lk) rows, one
    after the other in the packed [1,T,...] layout, with their bounds."""
    dtype, H = q.dtype, q.shape[2]
    Dn = kv.shape[-1] // 2
    Dr = 0 if k_rope is None else k_rope.shape[-1]
    f = torch.float64
    new = lambda *s: (torch.zeros(s, dtype=f, device=q.device), torch.zeros(s, dtype=f, device=q.device))  # noqa: E731
    Tq, Tk = q.shape[1], kv.shape[1]
    res = {"o": new(1, Tq, H, Dn), "lse": new(1, H, Tq)}
    res["lse"][0].fill_(-math.inf)
    if d_o is not None:
        res.update(dq=new(1, Tq, H, Dn + Dr), dkv=new(1, Tk, H, 2 * Dn))
        if Dr:
            res["dk_rope"] = new(1, Tk, Dr)
    a = b = 0
    for Lq, Lk in lens:
        rq, rk = slice(a, a + Lq), slice(b, b + Lk)
        x = q[0, rq].transpose(0, 1)
        y = kv[0, rk, :, :Dn].transpose(0, 1)
        if Dr:
            y = torch.cat((y, k_rope[0, rk][None].expand(H, -1, -1)), -1)
        i = torch.arange(Lq, device=q.device)
        limit = (i + Lk - Lq + 1).clamp(0, Lk) if causal else torch.full_like(i, Lk)
        r = attend(x, y, kv[0, rk, :, Dn:].transpose(0, 1), scale, limit,
                   None if d_o is None else d_o[0, rq].transpose(0, 1), dtype)
        for w in (0, 1):
            res["o"][w][0, rq] = r["o"][w].transpose(0, 1)
            res["lse"][w][0, :, rq] = r["lse"][w]
            if d_o is not None:
                res["dq"][w][0, rq] = r["dq"][w].transpose(0, 1)
                res["dkv"][w][0, rk] = torch.cat((r["dk"][w][..., :Dn], r["dv"][w]), -1).transpose(0, 1)
                if Dr:
                    # the sum over the heads: its terms' bounds, and its own roundings
                    z = r["dk"][w][..., Dn:].sum(0)
                    if w:
                        z = z + H * H32 * r["dk"][0][..., Dn:].abs().sum(0)
                    res["dk_rope"][w][0, rk] = z
        a, b = a + Lq, b + Lk
    return res


def check(name, x, ref, floor=1e-30):
    """Every element of x within its bound; infinities (lse of empty rows) equal."""
    value, bound = ref
    assert tuple(x.shape) == tuple(value.shape), (name, x.shape, value.shape)
    x = x.to(torch.float64)
    fin = torch.isfinite(value)
    assert torch.equal(x[~fin], value[~fin]), f"{name}: rows without keys"
    off = (x - value).abs()[fin] - bound[fin] - floor
    if not off.numel():
        return
    worst = off.max().item()
    assert worst <= 0, f"{name}: {int((off > 0).sum())} of {off.numel()} elements past their bound, by up to {worst:.3g}"
