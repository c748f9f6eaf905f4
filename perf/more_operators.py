"""What is measured of the operators that make the latent cache smaller, each
beside its plain form.

A cache row is a token's latent c and, in rotary models, a key part r that the
heads share. Five operators: the write of new rows into a cache that holds the
latents in 4 bits (``mla_cache_append_mx``) and the read of rows back from it
(``mla_cache_read_mx``), measured together; the absorbed attention of new tokens
over that cache (``mla_step_mx``); the accumulated attention weight of cached
rows (``mla_weigh``); and the eviction of the rows of least weight
(``mla_evict``).

4 bits: 32 consecutive channels share a power of two 2^e and are rounded to
multiples of it of {0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign, ties to the even
code. A page holds the codes of all its rows, then their scale bytes (e + 127),
then their shared key parts. The sizes follow the K3 head shape (96 heads of
128 channels, a latent of 512), one rank's share of it and smaller generic ones.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    k3 = {"heads": 96, "rope": 64, "latent": 512, "page": 64, "dtype": "bf16"}
    return [
        # one decode step of a serving batch writes its new rows, which are read back (latency)
        {"name": "store_b128_new1", "kind": "store", "batch": 128, "ctx": 600, "new": 1, **k3},
        # chunked prefill: ragged new chunks are written, then whole prefixes read back for the expanded attention
        {"name": "store_prefill_16k", "kind": "store", "batch": 7, "ctx": 2000, "new": 8192, **k3},
        # one interactive stream: the smallest decode call, where latency counts
        {"name": "step_b1_ctx1000", "kind": "step", "batch": 1, "ctx": 1000, "new": 1, **k3},
        # one stream with a very long context: the split over the long axis
        {"name": "step_b1_ctx100k", "kind": "step", "batch": 1, "ctx": 100001, "new": 1, **k3},
        # a serving batch of ragged contexts with a padding row, all heads: bound by the products
        {"name": "step_b128_ctx8k", "kind": "step", "batch": 128, "ctx": 8192, "new": 1, **k3},
        # one rank's share of the heads, no shared key part, longer contexts: bound by the cache's bytes
        {"name": "step_b64_ctx16k_h12", "kind": "step", "batch": 64, "ctx": 16384, "new": 1, **k3, "heads": 12,
         "rope": 0},
        # three speculated tokens a row, few heads, small pages, float32
        {"name": "step_f32_b8_new3", "kind": "step", "batch": 8, "ctx": 2047, "new": 3, "heads": 16, "rope": 64,
         "latent": 256, "page": 16, "dtype": "f32"},
        # the weights that one decode step of a short interactive stream adds, 4-bit cache (latency)
        {"name": "weigh_q4_b1_ctx1000", "kind": "weigh", "form": "q4", "batch": 1, "ctx": 1000, "new": 1, **k3},
        # the same of a serving batch over the unquantised cache: bound by its bytes
        {"name": "weigh_b128_ctx8k", "kind": "weigh", "form": "rows", "batch": 128, "ctx": 8192, "new": 1, **k3},
        # the last 24 tokens of four prompts weigh them whole, before their first eviction: bound by the products
        {"name": "weigh_q4_window24", "kind": "weigh", "form": "q4", "batch": 4, "ctx": 8192, "new": 24, **k3},
        # a serving batch cut back to 4096 rows each
        {"name": "evict_b128_ctx8k", "kind": "evict", "batch": 128, "ctx": 8192, "keep": 4096, "first": 4,
         "recent": 512, **k3},
        # one very long stream cut to half, float32 rows without a shared part
        {"name": "evict_f32_b1_ctx100k", "kind": "evict", "batch": 1, "ctx": 100001, "keep": 50000, "first": 64,
         "recent": 4096, "heads": 1, "rope": 0, "latent": 256, "page": 16, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("store", "step", "step", "step", "weigh", "weigh", "evict"))
    latent, rope = rng.choice(((512, 64), (512, 64), (512, 0), (256, 64), (256, 0)))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    c = {"kind": kind, "latent": latent, "rope": rope, "page": rng.choice((16, 32, 64, 128, 256)), "dtype": dtype,
         "batch": _log(rng, 1, 256), "heads": rng.choice((1, 5, 12, 16, 32, 64, 96, 128))}
    if kind == "store":
        return {**c, "ctx": _log(rng, 1, 1000), "new": rng.choice((1, 1, _log(rng, 2, 128)))}
    if kind == "evict":
        ctx = _log(rng, 100, min(131072, (1 << 19) // c["batch"]))
        return {**c, "ctx": ctx, "keep": _log(rng, 50, ctx), "first": rng.choice((0, 4, 64)),
                "recent": rng.choice((0, _log(rng, 1, ctx)))}
    rows = 1 << 20 if dtype == "bf16" else 1 << 15
    # (the weight of a sequence's only row is the number of heads, whatever the inputs)
    ctx = _log(rng, 1 if kind == "step" else 8, min(131072, rows // c["batch"]))
    if kind == "step":
        return {**c, "ctx": ctx, "new": rng.choice((1, 1, 1, 2, 4))}
    new = rng.choice((1, 1, 1, 3, 16))
    while ctx >= 16 and new * c["batch"] * ctx * c["heads"] > 96 * rows:
        ctx //= 2
    return {**c, "ctx": ctx, "new": new, "form": rng.choice(("q4", "q4", "rows"))}


def _lengths(case):
    """(rows before, new rows) of each sequence, by the case alone; ``step``,
    ``weigh``: rows with the new ones counted."""
    n, ctx = case["batch"], case["ctx"]
    new = case.get("new", 0)
    r = random.Random("%d %d %d" % (n, ctx, new))
    if case["kind"] == "store":
        return [(r.randint(0, ctx), new if new == 1 else r.randint(1, new)) for _ in range(n)]
    ls = [max(new, r.randint(ctx // 2, ctx)) for _ in range(n)]
    ls[at := r.randrange(n)] = max(new, ctx)
    if n > 4:
        ls[at - 1] = 0                      # a padding row of the batch
    return [(a, new) for a in ls]


def _scale(case):
    return 1.0 / math.sqrt(128 + case["rope"])


def _row_bytes(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] in ("store", "step") or case.get("form") == "q4":
        return case["latent"] // 2 + case["latent"] // 32 + es * case["rope"]
    return es * (case["latent"] + case["rope"])


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _encode(x):
    """[R,Dc] to codes [R,Dc/2] and scale bytes [R,Dc/32] (uint8), in float32."""
    x = x.float().view(x.shape[0], -1, 32)
    a = x.abs().amax(-1)
    e = (((a.view(torch.int32) + 0x1FFFFF) >> 23) - 129).clamp(max=125)
    bad, none = ~torch.isfinite(a), a < 2.0 ** -100
    y = x * ((127 - e) << 23).view(torch.float32)[..., None]
    y = torch.where((bad | none)[..., None], 0.0, y)
    m = y.abs()
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    s = torch.where(bad, 255, torch.where(none, 0, e + 127)).to(torch.uint8)
    code = code.flatten(1)
    return code[:, ::2] | code[:, 1::2] << 4, s


def _decode(codes, s):
    """The values of codes [..,Dc/2] and scale bytes [..,Dc/32], in float32."""
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    v = torch.cat((v, -v))
    b = torch.arange(256, device=codes.device)
    pair = torch.stack((v[b & 15], v[b >> 4]), -1)                       # a byte's two values
    f = s.to(torch.int32)
    f = torch.where(f == 0, 0.0, torch.where(f == 255, math.nan, (f << 23).view(torch.float32)))
    x = pair[codes.to(torch.int32)].flatten(-2)
    return (x.unflatten(-1, (-1, 32)) * f[..., None]).flatten(-2)


def _planes(case, cache):
    """A 4-bit cache's codes, scale bytes and shared parts (or None), each [n_pages,page,..], as views."""
    p, Dc = case["page"], case["latent"]
    flat, at, out = cache.view(cache.shape[0], -1), 0, []
    for w in (Dc // 2, Dc // 32):
        out.append(flat[:, at:at + p * w].unflatten(1, (p, w)))
        at += p * w
    out.append(flat[:, at:].view(_TYPES[case["dtype"]]).unflatten(1, (p, case["rope"])) if case["rope"] else None)
    return out


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def rand(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dt)

    kind, B, page, Dc, Dr = case["kind"], case["batch"], case["page"], case["latent"], case["rope"]
    H, T, ls, s = case["heads"], case.get("new", 0), _lengths(case), {"case": case}
    q4 = kind in ("store", "step") or case.get("form") == "q4"
    total = [a + b if kind == "store" else a for a, b in ls]
    pages = [-(-n // page) for n in total]
    s["max_pages"] = max(1, max(pages))
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((B, s["max_pages"]), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = order[at:at + n]
        at += n
    s["table"] = table.to(dev)
    s["lens"] = torch.tensor([a for a, _ in ls], dtype=torch.int32, device=dev)
    # channels of a latent differ in size, as a learned norm leaves them
    width = torch.exp(0.3 * torch.randn(Dc, generator=g, device=dev))

    def latents(*shape):
        return (torch.randn(*shape, Dc, generator=g, device=dev) * width).to(dt)

    if q4:
        s["cache"] = torch.zeros((n_pages, page, _row_bytes(case)), dtype=torch.uint8, device=dev)
        codes, scales, rope = _planes(case, s["cache"])
        for i in range(0, n_pages, max(1, 65536 // page)):
            j = min(n_pages, i + max(1, 65536 // page))
            c, e = _encode(latents((j - i) * page))
            codes[i:j] = c.view(j - i, page, -1)
            scales[i:j] = e.view(j - i, page, -1)
            if Dr:
                rope[i:j] = rand(j - i, page, Dr)
    else:
        s["cache"] = rand(n_pages, page, Dc + Dr)
    if kind == "store":
        cu = _starts([b for _, b in ls])
        packed = T > 1
        shape = (1, cu[-1]) if packed else (B, 1)
        # a slice of the down-projection's output
        s["latent"] = latents(*shape)
        s["k_rope"] = rand(*shape, Dc + Dr)[..., Dc:] if Dr else None
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if packed else None
        # what is read back: the new row of a decode step, or the whole sequences
        back = _starts([1] * B if not packed else total)
        s["cu_back"] = torch.tensor(back, dtype=torch.int32, device=dev)
        s["rows_back"] = back[-1]
        s["from"] = None if packed else s["lens"]
    if kind in ("step", "weigh"):
        # the absorbing product's output, head-major, and the slice of the query projection that it leaves as it is
        s["q_latent"] = rand(H, B * T, Dc, std=0.8).view(H, B, T, Dc).permute(1, 2, 0, 3)
        s["q_rope"] = rand(B, T, H, 128 + Dr)[..., 128:] if Dr else None
    if kind == "weigh":
        s["lse"] = _plain_scores(s)[1]
    if kind in ("weigh", "evict"):
        # weights of a few heavy tokens and many light ones, some of them equal
        w = torch.exp(2 * torch.randn((B, s["max_pages"] * page), generator=g, device=dev))
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device=dev) < 0.1, 0.0, w)
        s["weights_out"] = torch.zeros_like(s["weights"])
    if kind == "evict":
        s["table_out"], s["lens_out"] = torch.zeros_like(s["table"]), torch.zeros_like(s["lens"])
    return s


def _rows(s, b0, b1):
    """The cache rows of sequences b0..b1, [n,rows,Dc+Dr] in float32 (rows of missing pages: some page's)."""
    case, t = s["case"], s["table"][b0:b1].long().clamp(min=0)
    if s["cache"].dtype != torch.uint8:
        return s["cache"][t].flatten(1, 2).float()
    codes, scales, rope = _planes(case, s["cache"])
    x = _decode(codes[t], scales[t]).flatten(1, 2)
    return x if rope is None else torch.cat((x, rope[t].flatten(1, 2).float()), -1)


def _plain_scores(s, second=False):
    """Softmax numerators and what divides them, lse and (with second) the
    output, a few sequences at a time so that rows in float32 fit."""
    case = s["case"]
    Dc, T, B, scale = case["latent"], case["new"], case["batch"], _scale(case)
    q = s["q_latent"].float()
    if s["q_rope"] is not None:
        q = torch.cat((q, s["q_rope"].float()), -1)
    H, L = q.shape[2], s["max_pages"] * case["page"]
    some = max(1, (1 << 30) // (L * max(Dc, T * H)))
    out = []
    for b0 in range(0, B, some):
        b1 = min(B, b0 + some)
        k = _rows(s, b0, b1)
        p = (q[b0:b1].reshape(b1 - b0, T * H, -1) @ k.transpose(1, 2).contiguous()).mul_(scale).view(b1 - b0, T, H, -1)
        t, j = torch.arange(T, device=k.device)[:, None, None], torch.arange(L, device=k.device)
        seen = j < s["lens"][b0:b1, None, None, None] - T + t + 1
        p = p.masked_fill_(~seen, -math.inf)
        if not second and "lse" in s:
            lse = s["lse"][b0:b1, ..., None]
            out.append((p.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_().sum((1, 2)),))
            continue
        m = p.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = p.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        lse = (m + l.log()).squeeze(-1)
        o = None
        if second:
            p = p.div_(torch.where(l == 0, 1.0, l))
            o = (p.view(b1 - b0, T * H, -1) @ k[..., :Dc].contiguous()).view(b1 - b0, T, H, Dc)
            o = o.to(_TYPES[case["dtype"]])
        out.append((o, lse))
    return tuple(None if x[0] is None else torch.cat(x) for x in zip(*out))


def _slots(s, row, pos):
    page = s["case"]["page"]
    return s["table"][row, pos // page].long(), pos % page


def _plain_store(s):
    codes, scales, rope = _planes(s["case"], s["cache"])
    c, e = _encode(s["latent"].flatten(0, 1))
    i = torch.arange(c.shape[0], device=c.device)
    if s["cu"] is None:
        row, pos = i, s["lens"].long()
    else:
        row = torch.searchsorted(s["cu"], i.to(torch.int32), right=True) - 1
        pos = s["lens"][row].long() + i - s["cu"][row]
    p, at = _slots(s, row, pos)
    codes[p, at], scales[p, at] = c, e
    if rope is not None:
        rope[p, at] = s["k_rope"].flatten(0, 1)
    i = torch.arange(s["rows_back"], device=c.device)
    row = torch.searchsorted(s["cu_back"], i.to(torch.int32), right=True) - 1
    pos = i - s["cu_back"][row]
    if s["from"] is not None:
        pos = pos + s["from"][row]
    p, at = _slots(s, row, pos.long())
    x = _decode(codes[p, at], scales[p, at]).to(_TYPES[s["case"]["dtype"]])[None]
    return (x,) if rope is None else (x, rope[p, at][None])


def _plain_weigh(s):
    case = s["case"]
    w, n, T = s["weights"], s["lens"][:, None], case["new"]
    j = torch.arange(w.shape[1], device=w.device)
    old = torch.where(j < n - T, w, 0.0)             # the rows just written have no weight yet
    s["weights_out"].copy_(torch.where(j < n, old + _plain_scores(s)[0], 0.0))
    return s["weights_out"]


def _cut(case):
    """Pages of each sequence: the first that may go, the end of those, how many go, all in use."""
    p, out = case["page"], []
    for n, _ in _lengths(case):
        a, b = -(-case["first"] // p), max(n - case["recent"], 0) // p
        out.append((a, b, min(max((n - case["keep"]) // p, 0), max(b - a, 0)), -(-n // p)))
    return out


def _plain_evict(s):
    case = s["case"]
    p, w, n = case["page"], s["weights"], s["lens"].long()[:, None]
    first, recent, keep = case["first"], case["recent"], case["keep"]
    a, b = -(-first // p), (n - recent).clamp(min=0) // p
    e = torch.minimum(((n - keep) // p).clamp(min=0), (b - a).clamp(min=0))
    used = (n + p - 1) // p
    j = torch.arange(w.shape[1], device=w.device)[None]
    mid = (j >= a * p) & (j < b * p)
    order = torch.sort(torch.where(mid, w, -1.0), dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order))
    stays = rank < (b - a - e) * p
    low = j < (b - e) * p
    hole, mover = mid & low & ~stays & (e > 0), mid & ~low & stays
    row = torch.arange(w.shape[0], device=w.device)[:, None].expand_as(hole)
    jj = j.expand_as(hole)
    rows, dst, src = row[hole], jj[hole], jj[mover]
    cache = s["cache"]
    cache[_slots(s, rows, dst)] = cache[_slots(s, rows, src)]
    w = w.clone()
    w[rows, dst] = w[rows, src]
    up = torch.where(low, j, j + e * p)
    s["weights_out"].copy_(torch.where(j < n - e * p, w.gather(1, up.clamp(max=w.shape[1] - 1)),
                                       torch.where(j < n, 0.0, w)))
    i = torch.arange(s["max_pages"], device=w.device)[None]
    at = torch.where(i < b - e, i, torch.where(i < used - e, i + e, torch.where(i < used, i - (used - b), i)))
    s["table_out"].copy_(s["table"].gather(1, at))
    s["lens_out"].copy_((n - e * p)[:, 0])
    return cache, s["table_out"], s["lens_out"], s["weights_out"]


def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        return _plain_store(s) if kind == "store" else _plain_scores(s, True) if kind == "step" else \
            _plain_weigh(s) if kind == "weigh" else _plain_evict(s)
    import gated_delta_rule_chunk_amd as kda
    if kind == "store":
        kda.mla_cache_append_mx(s["latent"], s["k_rope"], s["cache"], s["table"], s["lens"], cu_seqlens=s["cu"])
        x, r = kda.mla_cache_read_mx(s["cache"], s["table"], s["cu_back"], s["rows_back"], case["latent"],
                                     _TYPES[case["dtype"]], starts=s["from"])
        return (x,) if r is None else (x, r)
    if kind == "step":
        return kda.mla_step_mx(s["q_latent"], s["q_rope"], s["cache"], s["table"], s["lens"], scale=_scale(case))
    if kind == "weigh":
        return kda.mla_weigh(s["q_latent"], s["q_rope"], s["cache"], s["table"], s["lens"], s["lse"], _scale(case),
                             s["weights"], out=s["weights_out"])
    table, lens, w = kda.mla_evict(s["cache"], s["table"], s["lens"], s["weights"], case["keep"], first=case["first"],
                                   recent=case["recent"], out=(s["table_out"], s["lens_out"], s["weights_out"]))
    return s["cache"], table, lens, w


def work(case):
    ls, row, es = _lengths(case), _row_bytes(case), 2 if case["dtype"] == "bf16" else 4
    kind, H, T, D = case["kind"], case["heads"], case.get("new", 0), case["latent"] + case["rope"]
    if kind == "store":
        new = sum(b for _, b in ls)
        back = len(ls) if T == 1 else sum(a + b for a, b in ls)
        # the rows just written need not be read from memory again to be returned, older ones do
        return {"bytes": new * (es * D + row) + (back - new) * row + back * es * D, "flops": 0}
    if kind == "evict":
        cut, p = _cut(case), case["page"]
        # of the pages that go, the share that stays anywhere moves: read and written once
        moved = sum(e * p * (b - a - e) / max(b - a, 1) for a, b, e, _ in cut)
        return {"bytes": int(2 * moved * row) + 8 * sum(a for a, _ in ls), "flops": 0}
    keys = sum(a for a, _ in ls)
    pairs = sum(max(0, a - T + t + 1) for a, _ in ls for t in range(T))
    rows = case["batch"] * T * H
    if kind == "weigh":
        return {"bytes": keys * (row + 8) + rows * (es * D + 4), "flops": 2 * pairs * H * D}
    return {"bytes": keys * row + rows * (es * (D + case["latent"]) + 4),
            "flops": 2 * pairs * H * (D + case["latent"])}


def _exact_rounded(x):
    """4-bit values of [R,Dc] in float64: the nearest multiple of each block's power of two, by distance."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    out = []
    for part in x.to(torch.float64).split(8192):
        y = part.unflatten(1, (-1, 32))
        a = y.abs().amax(-1, keepdim=True)
        m, x2 = torch.frexp(a / 7)                   # a / 7 = m 2^x2, m in [0.5, 1): the least 2^e that is no less
        e = torch.where(m == 0.5, x2 - 1, x2).clamp(max=125)
        two = torch.ldexp(torch.ones_like(a), e)
        d = ((y / two).abs()[..., None] - grid).abs()
        near = d == d.amin(-1, keepdim=True)
        # of two as near, the even code
        pick = torch.where(near, torch.arange(8, device=x.device) % 2, 2).argmin(-1)
        z = torch.copysign(grid[pick], y) * two
        z = torch.where(torch.isfinite(a), torch.where(a < 2.0 ** -100, 0.0, z), math.nan)
        out.append(z.flatten(1))
    return torch.cat(out)


def _exact_rows(s, b, n):
    """Sequence b's first n rows, latents and shared parts, in float64, byte by byte."""
    case, f8 = s["case"], torch.float64
    p, Dc, Dr, dt = case["page"], case["latent"], case["rope"], _TYPES[case["dtype"]]
    pages = s["cache"][s["table"][b, :-(-n // p)].long()]
    if pages.dtype != torch.uint8:
        x = pages.flatten(0, 1)[:n].to(f8)
        return x[:, :Dc], x[:, Dc:]
    flat = pages.flatten(1)
    c = flat[:, :p * Dc // 2].reshape(-1, Dc // 2)[:n]
    e = flat[:, p * Dc // 2:p * (Dc // 2 + Dc // 32)].reshape(-1, Dc // 32)[:n].to(f8)
    c = torch.stack((c % 16, c // 16), -1).flatten(1).to(f8)
    m = torch.where(c >= 8, c - 8, c)
    # codes 0 and 1: 0, 0.5; then (2 + odd) / 2 times a power of two
    v = torch.where(m < 2, m / 2, (2 + m % 2) / 2 * 2 ** (torch.div(m, 2, rounding_mode="floor") - 1))
    x = torch.where(c >= 8, -v, v).unflatten(1, (-1, 32)) * 2 ** (e[..., None] - 127)
    x = torch.where(e[..., None] == 255, math.nan, torch.where(e[..., None] == 0, 0.0, x))
    r = flat[:, p * (Dc // 2 + Dc // 32):].reshape(-1).view(dt).view(-1, Dr)[:n].to(f8) if Dr else None
    return x.flatten(1), r


def exact(case, seed):
    s = prepare(case, seed)
    ls, kind, f8, T = _lengths(case), case["kind"], torch.float64, case.get("new", 0)
    B, H, Dc, Dr = case["batch"], case["heads"], case["latent"], case["rope"]
    if kind == "store":
        new, out, rope, at = _exact_rounded(s["latent"].flatten(0, 1)), [], [], 0
        kr = None if s["k_rope"] is None else s["k_rope"].flatten(0, 1).to(f8)
        for b, (before, n) in enumerate(ls):
            if T > 1 and before:
                x, r = _exact_rows(s, b, before)
                out.append(x)
                rope.append(r)
            out.append(new[at:at + n])
            if kr is not None:
                rope.append(kr[at:at + n])
            at += n
        return (torch.cat(out)[None],) if kr is None else (torch.cat(out)[None], torch.cat(rope)[None])
    if kind == "evict":
        p, flat = case["page"], s["cache"].flatten(0, 1).to(f8)
        w, table = s["weights"].to(f8).cpu(), s["table"].cpu()
        wout, tout, lens = w.clone(), table.clone(), []
        for b, ((n, _), (a, end, e, used)) in enumerate(zip(ls, _cut(case))):
            lens.append(n - e * p)
            if not e:
                continue
            v = w[b].tolist()
            by = sorted(range(a * p, end * p), key=lambda j: (-v[j], j))
            stays = set(by[:(end - a - e) * p])
            src = [j for j in range((end - e) * p, end * p) if j in stays]
            dst = [j for j in range(a * p, (end - e) * p) if j not in stays]
            at = lambda js: torch.tensor([int(table[b, j // p]) * p + j % p for j in js], dtype=torch.long,  # noqa: E731
                                         device=flat.device)
            flat[at(dst)] = flat[at(src)]
            x = w[b].clone()
            x[dst] = x[src]
            wout[b] = torch.cat((x[:(end - e) * p], x[end * p:n], torch.zeros(e * p, dtype=f8), x[n:]))
            t = table[b].tolist()
            tout[b] = torch.tensor(t[:end - e] + t[end:used] + t[end - e:end] + t[used:])
        dev = flat.device
        return (flat.view(s["cache"].shape), tout.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                wout.to(dev))
    scale = _scale(case)
    o = torch.zeros(s["q_latent"].shape, dtype=f8, device="cuda")
    lse = torch.full(o.shape[:3], -math.inf, dtype=f8, device="cuda")
    w = torch.zeros(s["weights"].shape, dtype=f8, device="cuda") if kind == "weigh" else None
    for b, (n, _) in enumerate(ls):
        if n == 0:
            continue
        c, r = _exact_rows(s, b, n)
        for t in range(T):
            m = n - T + t + 1
            x = s["q_latent"][b, t].to(f8) @ c[:m].t()
            if Dr:
                x = x + s["q_rope"][b, t].to(f8) @ r[:m].t()
            x = x * scale
            if kind == "weigh":
                w[b, :m] += torch.exp(x - s["lse"][b, t].to(f8)[:, None]).sum(0)
                continue
            lse[b, t] = torch.logsumexp(x, -1)
            o[b, t] = torch.softmax(x, -1) @ c[:m]
        if kind == "weigh":
            w[b, :max(0, n - T)] += s["weights"][b, :max(0, n - T)].to(f8)
    return w if kind == "weigh" else (o, lse)
