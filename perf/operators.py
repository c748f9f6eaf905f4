"""What is measured of the latent-attention operators, each beside its plain form.

Four operators: the expanded attention's forward (``mla_fwd``), a training step
through it (``autograd.mla``: forward and the gradients of q, kv and k_rope),
the absorbed attention of newly generated tokens over a paged cache of latents
(``mla_step``) and the write of new tokens into that cache
(``mla_cache_append``). The sizes follow the K3 head shape (96 heads of 128
channels, a latent of 512) and smaller generic ones.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    k3 = {"heads": 96, "nope": 128, "rope": 64, "dtype": "bf16"}
    return [
        # one whole prompt of the K3 head shape, as a prefill runs it: bound by the matrix cores
        {"name": "fwd_k3_t4096", "kind": "fwd", "seqs": 1, "tokens": 4096, "prefix": 0, "packed": False, **k3},
        # a packed prefill batch of ragged prompts, some continuing a cached prefix (chunked prefill)
        {"name": "fwd_packed_ragged", "kind": "fwd", "seqs": 9, "tokens": 1531, "prefix": 777, "packed": True, **k3},
        # a short prompt without a shared key part in float32: few tiles, latency and the float32 path
        {"name": "fwd_f32_t333", "kind": "fwd", "seqs": 2, "tokens": 333, "prefix": 0, "packed": False, "heads": 16,
         "nope": 64, "rope": 0, "dtype": "f32"},
        # a training step of the K3 head shape at its benchmark length: the largest case
        {"name": "train_k3_t4096", "kind": "train", "seqs": 1, "tokens": 4096, "prefix": 0, "packed": False, **k3},
        # a packed training batch of ragged documents, fewer heads (one rank's share)
        {"name": "train_packed_ragged", "kind": "train", "seqs": 12, "tokens": 1100, "prefix": 0, "packed": True,
         **k3, "heads": 24},
        # a float32 training step (gradient checks, small models)
        {"name": "train_f32_t500", "kind": "train", "seqs": 1, "tokens": 500, "prefix": 0, "packed": False,
         "heads": 8, "nope": 128, "rope": 64, "dtype": "f32"},
        # one interactive stream: the smallest decode call, where latency counts
        {"name": "step_b1_ctx1000", "kind": "step", "batch": 1, "ctx": 1000, "new": 1, "page": 64, "latent": 512,
         **k3},
        # one stream with a very long context: the split over the long axis
        {"name": "step_b1_ctx100k", "kind": "step", "batch": 1, "ctx": 100001, "new": 1, "page": 64, "latent": 512,
         **k3},
        # a serving batch of ragged contexts with padding rows: bound by the cache's bytes
        {"name": "step_b128_ctx8k", "kind": "step", "batch": 128, "ctx": 8192, "new": 1, "page": 64, "latent": 512,
         **k3},
        # three speculated tokens a row, few heads, small pages, float32 cache
        {"name": "step_f32_b8_new3", "kind": "step", "batch": 8, "ctx": 2047, "new": 3, "page": 16, "latent": 256,
         "heads": 16, "nope": 64, "rope": 64, "dtype": "f32"},
        # the cache write that goes with one decode step of a serving batch
        {"name": "append_b128_new1", "kind": "append", "batch": 128, "ctx": 600, "new": 1, "page": 64, "latent": 512,
         "rope": 64, "dtype": "bf16"},
        # the cache write after a packed prefill
        {"name": "append_prefill_16k", "kind": "append", "batch": 7, "ctx": 2000, "new": 8192, "page": 64,
         "latent": 512, "rope": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("fwd", "fwd", "train", "train", "step", "step", "step", "append"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if kind in ("fwd", "train"):
        heads = rng.choice((1, 3, 8, 16, 24, 96))
        # a training document has a few tokens at least: one key's gradients of q and k are zero
        tokens = _log(rng, 1 if kind == "fwd" else 8, 4096 if dtype == "bf16" else 1024)
        packed = rng.random() < 0.5
        seqs = _log(rng, 1, 16)
        prefix = rng.choice((0, 0, _log(rng, 1, 1000))) if kind == "fwd" else 0
        # no more pairs than the largest listed case (float32: a sixteenth of them)
        most = 4096 * 4096 * 96 // (1 if dtype == "bf16" else 16)
        while seqs > 1 and seqs * tokens * (tokens + prefix) * heads > most:
            seqs -= 1
        while heads > 1 and seqs * tokens * (tokens + prefix) * heads > most:
            heads //= 2
        nope, rope = rng.choice(((128, 64), (128, 64), (128, 0), (64, 64), (64, 0)))
        return {"kind": kind, "seqs": seqs, "tokens": tokens, "prefix": prefix, "packed": packed, "heads": heads,
                "nope": nope, "rope": rope, "dtype": dtype}
    latent, rope = rng.choice(((512, 64), (512, 64), (512, 0), (256, 64), (256, 0)))
    page = rng.choice((16, 32, 64, 128, 256))
    if kind == "append":
        return {"kind": kind, "batch": _log(rng, 1, 256), "ctx": _log(rng, 1, 1000),
                "new": rng.choice((1, 1, _log(rng, 2, 128))), "page": page, "latent": latent, "rope": rope,
                "dtype": dtype}
    batch = _log(rng, 1, 256)
    ctx = _log(rng, 1, min(131072, (1 << 20 if dtype == "bf16" else 1 << 15) // batch))
    return {"kind": kind, "batch": batch, "ctx": ctx, "new": rng.choice((1, 1, 1, 2, 4)), "page": page,
            "latent": latent, "rope": rope, "heads": rng.choice((1, 5, 16, 32, 64, 96, 128)), "nope": 128,
            "dtype": dtype}


def _lengths(case):
    """(queries, keys) of each sequence of an expanded case; (before, new) of
    each row of a cached one. They go by the case alone."""
    if case["kind"] in ("fwd", "train"):
        n, t, p = case["seqs"], case["tokens"], case["prefix"]
        if not case["packed"]:
            return [(t, t + p)] * n
        r = random.Random("%d %d %d" % (n, t, p))
        ls = [(r.randint(1, t) if r.random() < 0.6 else _log(r, 1, t), r.randint(0, p)) for _ in range(n)]
        ls[at := r.randrange(n)] = (t, p)
        if n > 3:
            ls[at - 1] = (0, 0)             # an empty sequence
        return [(a, a + b) for a, b in ls]
    n, ctx, new = case["batch"], case["ctx"], case["new"]
    r = random.Random("%d %d %d" % (n, ctx, new))
    if case["kind"] == "append":
        return [(r.randint(0, ctx), new if new == 1 else r.randint(1, new)) for _ in range(n)]
    ls = [max(new, r.randint(ctx // 2, ctx)) for _ in range(n)]
    ls[at := r.randrange(n)] = max(new, ctx)
    if n > 4:
        ls[at - 1] = 0                      # a padding row of the batch
    return [(a, new) for a in ls]


def _scale(case):
    return 1.0 / math.sqrt(case["nope"] + case["rope"])


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def rand(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dt)

    ls, s = _lengths(case), {"case": case}
    if case["kind"] in ("fwd", "train"):
        H, Dn, Dr = case["heads"], case["nope"], case["rope"]
        cq, ck = _starts([a for a, _ in ls]), _starts([b for _, b in ls])
        B, Tq, Tk = (1, cq[-1], ck[-1]) if case["packed"] else (len(ls), ls[0][0], ls[0][1])
        s["q"] = rand(B, Tq, H, Dn + Dr)
        s["kv"] = rand(B, Tk, H, 2 * Dn)
        # the shared key part is a slice of the down-projection's output
        s["k_rope"] = rand(B, Tk, 4 * Dr)[..., 3 * Dr:] if Dr else None
        if case["kind"] == "train":
            s["d_o"] = rand(B, Tq, H, Dn)
        s["cu_q"] = torch.tensor(cq, dtype=torch.int32, device=dev) if case["packed"] else None
        s["cu_k"] = torch.tensor(ck, dtype=torch.int32, device=dev) if case["packed"] else None
        s["max_q"], s["max_k"] = max(a for a, _ in ls), max(b for _, b in ls)
        return s
    B, Dc, Dr, page = case["batch"], case["latent"], case["rope"], case["page"]
    step = case["kind"] == "step"
    total = [a if step else a + b for a, b in ls]
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
    s["cache"] = rand(n_pages, page, Dc + Dr)
    s["lens"] = torch.tensor([a for a, _ in ls], dtype=torch.int32, device=dev)
    if step:
        H, T = case["heads"], case["new"]
        # the absorbing product's output, head-major, and the slice of the query projection that it leaves as it is
        s["q_latent"] = rand(H, B * T, Dc, std=0.8).view(H, B, T, Dc).permute(1, 2, 0, 3)
        s["q_rope"] = rand(B, T, H, case["nope"] + Dr)[..., case["nope"]:] if Dr else None
    else:
        new = [b for _, b in ls]
        cu = _starts(new)
        packed = case["new"] > 1
        shape = (1, cu[-1]) if packed else (B, 1)
        s["latent"] = rand(*shape, Dc)
        s["k_rope"] = rand(*shape, Dc + Dr)[..., Dc:] if Dr else None
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if packed else None
    return s


def _gather(x, cu, most):
    """Rows of a packed [1,T,...] tensor as [N,most,...], and which of them are rows of their sequence."""
    at = cu[:-1, None].long() + torch.arange(most, device=x.device)
    valid = at < cu[1:, None].long()
    return x[0, torch.where(valid, at, 0)], valid


def _plain_attend(s, train):
    case = s["case"]
    Dn, Dr, scale, dt = case["nope"], case["rope"], _scale(case), _TYPES[case["dtype"]]
    q, kv, r, do = s["q"], s["kv"], s["k_rope"], s.get("d_o")
    packed = s["cu_q"] is not None
    if packed:
        q, vq = _gather(q, s["cu_q"], s["max_q"])
        kv, vk = _gather(kv, s["cu_k"], s["max_k"])
        r = None if r is None else _gather(r, s["cu_k"], s["max_k"])[0]
        do = None if do is None else _gather(do, s["cu_q"], s["max_q"])[0]
        lq, lk = s["cu_q"].diff()[:, None, None], s["cu_k"].diff()[:, None, None]
    else:
        lq, lk = s["max_q"], s["max_k"]
    H, dev = q.shape[2], q.device
    q = q.float().transpose(1, 2)
    k, v = kv[..., :Dn].float().transpose(1, 2), kv[..., Dn:].float().transpose(1, 2).contiguous()
    if r is not None:
        k = torch.cat((k, r.float()[:, None].expand(-1, H, -1, -1)), -1)
    k = k.contiguous()
    i, j = torch.arange(s["max_q"], device=dev)[:, None], torch.arange(s["max_k"], device=dev)[None]
    seen = (j <= i + lk - lq) & (j < lk) & (i < lq)
    seen = seen[:, None] if packed else seen
    p = (q @ k.transpose(2, 3)).mul_(scale).masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)
    p = p.div_(torch.where(l == 0, 1.0, l))
    o = p @ v

    def back(x, valid):      # [N,H,L,D] to the caller's layout
        x = x.transpose(1, 2)
        return x[valid][None].to(dt) if packed else x.to(dt).contiguous()

    vq, vk = (vq, vk) if packed else (None, None)
    out = back(o, vq)
    if not train:
        return out, (lse.transpose(1, 2)[vq].t()[None].contiguous() if packed else lse)
    do = do.float().transpose(1, 2)
    dv = p.transpose(2, 3) @ do
    ds = (do @ v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = ds @ k
    dk = ds.transpose(2, 3) @ q
    dkv = back(torch.cat((dk[..., :Dn], dv), -1), vk)
    if r is None:
        return out, back(dq, vq), dkv
    dr = dk[..., Dn:].sum(1, keepdim=True)
    return out, back(dq, vq), dkv, back(dr, vk).squeeze(2)


def _plain_step(s):
    case = s["case"]
    Dc, T, scale = case["latent"], case["new"], _scale(case)
    B = case["batch"]
    q = s["q_latent"].float()
    if s["q_rope"] is not None:
        q = torch.cat((q, s["q_rope"].float()), -1)
    H = q.shape[2]
    k = s["cache"][s["table"].long().clamp(min=0)].flatten(1, 2).float()
    p = (q.reshape(B, T * H, -1) @ k.transpose(1, 2)).mul_(scale).view(B, T, H, -1)
    t, j = torch.arange(T, device=k.device)[:, None, None], torch.arange(k.shape[1], device=k.device)
    seen = j < s["lens"][:, None, None, None] - T + t + 1
    p = p.masked_fill_(~seen, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)
    p = p.div_(torch.where(l == 0, 1.0, l))
    o = p.view(B, T * H, -1) @ k[..., :Dc].contiguous()
    return o.view(B, T, H, Dc).to(_TYPES[case["dtype"]]), lse


def _plain_append(s):
    case = s["case"]
    page, x = case["page"], s["latent"]
    if s["k_rope"] is not None:
        x = torch.cat((x, s["k_rope"]), -1)
    x = x.flatten(0, 1)
    i = torch.arange(x.shape[0], device=x.device)
    if s["cu"] is None:
        row, pos = i, s["lens"].long()
    else:
        row = torch.searchsorted(s["cu"], i.to(torch.int32), right=True) - 1
        pos = s["lens"][row].long() + i - s["cu"][row]
    slot = s["table"][row, pos // page].long() * page + pos % page
    s["cache"].flatten(0, 1)[slot] = x
    return s["cache"]


def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        return _plain_step(s) if kind == "step" else _plain_append(s) if kind == "append" else \
            _plain_attend(s, kind == "train")
    import gated_delta_rule_chunk_amd as kda
    from gated_delta_rule_chunk_amd import autograd
    if kind == "fwd":
        return kda.mla_fwd(s["q"], s["kv"], s["k_rope"], cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"],
                           scale=_scale(case))
    if kind == "train":
        leaves = [x.detach().requires_grad_() for x in (s["q"], s["kv"], s["k_rope"]) if x is not None]
        o = autograd.mla(*leaves, cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"], scale=_scale(case))
        return (o.detach(),) + torch.autograd.grad(o, leaves, s["d_o"])
    if kind == "step":
        return kda.mla_step(s["q_latent"], s["q_rope"], s["cache"], s["table"], s["lens"], scale=_scale(case))
    kda.mla_cache_append(s["latent"], s["k_rope"], s["cache"], s["table"], s["lens"], cu_seqlens=s["cu"])
    return s["cache"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    ls, Dr = _lengths(case), case["rope"]
    if case["kind"] in ("fwd", "train"):
        H, Dn = case["heads"], case["nope"]
        nq, nk = sum(a for a, _ in ls), sum(b for _, b in ls)
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in ls)
        q, kv, r, o = nq * H * (Dn + Dr), nk * H * 2 * Dn, nk * Dr, nq * H * Dn
        if case["kind"] == "fwd":
            return {"bytes": es * (q + kv + r + o) + 4 * nq * H, "flops": 2 * pairs * H * (2 * Dn + Dr)}
        # the forward's two products and the gradients' four; d_o is read, o and the gradients are written
        return {"bytes": es * 2 * (q + kv + r + o), "flops": 6 * pairs * H * (2 * Dn + Dr)}
    D = case["latent"] + Dr
    if case["kind"] == "append":
        return {"bytes": 2 * es * D * sum(b for _, b in ls), "flops": 0}
    H, T = case["heads"], case["new"]
    keys = sum(a for a, _ in ls)
    pairs = sum(max(0, a - T + t + 1) for a, _ in ls for t in range(T))
    rows = case["batch"] * T * H
    return {"bytes": es * (keys * D + rows * (D + case["latent"])) + 4 * rows,
            "flops": 2 * pairs * H * (D + case["latent"])}


def exact(case, seed):
    s = prepare(case, seed)
    ls, scale, Dr = _lengths(case), _scale(case) if "nope" in case else 1.0, case["rope"]
    f8 = torch.float64
    if case["kind"] == "append":
        flat = s["cache"].to(f8).view(-1, s["cache"].shape[-1])
        table, page, at = s["table"].cpu().tolist(), case["page"], 0
        new = s["latent"].flatten(0, 1).to(f8)
        rope = None if s["k_rope"] is None else s["k_rope"].flatten(0, 1).to(f8)
        for row, (before, n) in zip(table, ls):
            slots = torch.tensor([row[p // page] * page + p % page for p in range(before, before + n)],
                                 device=flat.device)
            flat[slots, :case["latent"]] = new[at:at + n]
            if rope is not None:
                flat[slots, case["latent"]:] = rope[at:at + n]
            at += n
        return flat.view(s["cache"].shape)
    if case["kind"] == "step":
        Dc, T = case["latent"], case["new"]
        o = torch.zeros(s["q_latent"].shape, dtype=f8, device="cuda")
        lse = torch.full(o.shape[:3], -math.inf, dtype=f8, device="cuda")
        for b, (n, _) in enumerate(ls):
            if n == 0:
                continue
            pages = s["table"][b, :-(-n // case["page"])].long()
            rows = s["cache"][pages].reshape(-1, Dc + Dr)[:n].to(f8)
            for t in range(T):
                m = n - T + t + 1
                x = s["q_latent"][b, t].to(f8) @ rows[:m, :Dc].t()
                if Dr:
                    x = x + s["q_rope"][b, t].to(f8) @ rows[:m, Dc:].t()
                x = x * scale
                lse[b, t] = torch.logsumexp(x, -1)
                o[b, t] = torch.softmax(x, -1) @ rows[:m, :Dc]
        return o, lse
    train, H, Dn = case["kind"] == "train", case["heads"], case["nope"]
    q, kv, r = s["q"], s["kv"], s["k_rope"]
    o = torch.zeros(q.shape[:3] + (Dn,), dtype=f8, device="cuda")
    lse = torch.zeros((q.shape[0], H, q.shape[1]), dtype=f8, device="cuda")
    if train:
        dq, dkv = torch.zeros(q.shape, dtype=f8, device="cuda"), torch.zeros(kv.shape, dtype=f8, device="cuda")
        dr = None if r is None else torch.zeros(r.shape, dtype=f8, device="cuda")
    q0 = k0 = 0
    for n, (a, b) in enumerate(ls):
        if not a:
            k0 += b
            continue
        bi = 0 if case["packed"] else n
        rq, rk = (slice(q0, q0 + a), slice(k0, k0 + b)) if case["packed"] else (slice(0, a), slice(0, b))
        hide = torch.ones(a, b, dtype=torch.bool, device="cuda").triu(b - a + 1)
        for h in range(H):
            x = q[bi, rq, h].to(f8)
            y, v = kv[bi, rk, h, :Dn].to(f8), kv[bi, rk, h, Dn:].to(f8)
            if r is not None:
                y = torch.cat((y, r[bi, rk].to(f8)), 1)
            z = (scale * (x @ y.t())).masked_fill(hide, -math.inf)
            lse[bi, h, rq] = torch.logsumexp(z, 1)
            w = torch.softmax(z, 1)
            oh = w @ v
            o[bi, rq, h] = oh
            if train:
                d = s["d_o"][bi, rq, h].to(f8)
                dz = w * (d @ v.t() - (d * oh).sum(1, keepdim=True))
                dq[bi, rq, h] = scale * (dz @ y)
                dy = scale * (dz.t() @ x)
                dkv[bi, rk, h, :Dn] = dy[:, :Dn]
                dkv[bi, rk, h, Dn:] = w.t() @ d
                if r is not None:
                    dr[bi, rk] += dy[:, Dn:]
        q0, k0 = q0 + a, k0 + b
    if not train:
        return o, lse
    return (o, dq, dkv) if r is None else (o, dq, dkv, dr)
