"""Cases that measure the serving and cross-attention operators: the paged append with the
position rotation, attention over a paged cache whose batch shares a prefix, and cross
attention (single tokens, and a training step's forward and backward).

Every case is made from its sizes and a seed; ``run`` computes it either in elementary torch
operations in 32 bits (64 for the angles) or, where ``own`` is true, through the library's
entry points.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one sequence writes one token: the latency of a single user's decode step
        dict(name="append_one_token", op="append", B=1, new_lo=1, new_hi=1, own_lo=1000,
             own_hi=1000, page=16, hq=32, hkv=8, d=128, rot=128, inter=False, offset=0),
        # one decode step of a full serving batch behind a shared prefix
        dict(name="append_decode_batch", op="append", B=256, new_lo=1, new_hi=1, own_lo=7,
             own_hi=250, page=16, hq=32, hkv=8, d=128, rot=128, inter=False, offset=32768),
        # ragged prompts enter the cache; half of each head is rotated, pairs interleaved
        dict(name="append_prompts", op="append", B=7, new_lo=501, new_hi=4093, own_lo=501,
             own_hi=4095, page=64, hq=32, hkv=8, d=128, rot=64, inter=True, offset=0),
        # a few users, a short system prompt: latency counts
        dict(name="prefix_decode_few", op="prefix", B=4, new_lo=1, new_hi=1, own_lo=33,
             own_hi=300, page=16, hq=8, hkv=2, d=64, prefix=1000),
        # a serving batch behind one long document
        dict(name="prefix_decode_batch", op="prefix", B=64, new_lo=1, new_hi=1, own_lo=17,
             own_hi=1024, page=64, hq=32, hkv=8, d=128, prefix=32768),
        # no shared part: plain decode over long caches of very different lengths
        dict(name="paged_decode_long", op="prefix", B=12, new_lo=1, new_hi=1, own_lo=1001,
             own_hi=16384, page=32, hq=32, hkv=8, d=128, prefix=0),
        # several drafted tokens per sequence are checked at once, every head with its own K/V
        dict(name="prefix_verify_drafts", op="prefix", B=24, new_lo=3, new_hi=8, own_lo=100,
             own_hi=777, page=16, hq=16, hkv=16, d=64, prefix=8191),
        # questions of some hundred tokens about one long document (prefill behind the prefix)
        dict(name="prefix_questions", op="prefix", B=4, new_lo=199, new_hi=301, own_lo=199,
             own_hi=301, page=64, hq=32, hkv=8, d=128, prefix=16384),
        # a decoder's token step over the encoder's states
        dict(name="cross_decode", op="cross", B=32, lq=1, lk_lo=333, lk_hi=1500, hq=16, hkv=16,
             d=64, train=False),
        # a short sample: training step, odd sizes
        dict(name="cross_train_small", op="cross", B=2, lq=129, lk_lo=190, lk_hi=257, hq=8,
             hkv=8, d=64, train=True),
        # ordinary training step over padded encoder states
        dict(name="cross_train_ragged", op="cross", B=8, lq=447, lk_lo=700, lk_hi=1500, hq=16,
             hkv=16, d=64, train=True),
        # long states, grouped heads
        dict(name="cross_train_long", op="cross", B=2, lq=2048, lk_lo=4001, lk_hi=4096, hq=32,
             hkv=8, d=128, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    hkv = rng.choice([2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8] if hkv < 8 else [1, 2, 4])
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["append", "decode", "paged", "chunk", "cross_decode", "cross_train"])
    if kind == "append":
        if rng.random() < 0.5:
            B, new_lo, new_hi = _log(rng, 1, 256), 1, 1
            own_lo, own_hi = 1, _log(rng, 2, 250)
        else:
            B = _log(rng, 1, 7)
            new_hi = _log(rng, 16, 4000)
            new_lo = rng.randint(1, new_hi)
            own_lo, own_hi = new_lo, new_hi + rng.randint(0, 90)
        return dict(op="append", B=B, new_lo=new_lo, new_hi=new_hi, own_lo=own_lo, own_hi=own_hi,
                    page=page, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d // 2]),
                    inter=rng.random() < 0.5, offset=_log(rng, 1, 900000))
    if kind == "decode":
        new = rng.choice([1, 1, 1, 2, 5, 8])
        own_hi = _log(rng, 40, 1024)
        return dict(op="prefix", B=_log(rng, 2, 64), new_lo=rng.randint(1, new), new_hi=new,
                    own_lo=rng.randint(new, own_hi), own_hi=own_hi, page=page, hq=hq, hkv=hkv,
                    d=d, prefix=_log(rng, 200, 16384))
    if kind == "paged":
        own_hi = _log(rng, 200, 16384)
        return dict(op="prefix", B=_log(rng, 1, 12), new_lo=1, new_hi=1,
                    own_lo=rng.randint(1, own_hi), own_hi=own_hi, page=page, hq=hq, hkv=hkv, d=d,
                    prefix=0)
    if kind == "chunk":
        new_hi = _log(rng, 16, 300)
        new_lo = rng.randint(max(1, new_hi // 2), new_hi)
        return dict(op="prefix", B=rng.randint(1, 4), new_lo=new_lo, new_hi=new_hi,
                    own_lo=new_lo, own_hi=new_hi + rng.randint(0, 200), page=page, hq=hq,
                    hkv=hkv, d=d, prefix=_log(rng, 500, 16384))
    if kind == "cross_decode":
        hi = _log(rng, 64, 4096)
        return dict(op="cross", B=_log(rng, 1, 64), lq=rng.choice([1, 1, 2, 4]),
                    lk_lo=rng.randint(max(1, hi // 4), hi), lk_hi=hi, hq=hq, hkv=hkv, d=d,
                    train=False)
    hi = _log(rng, 100, 4096)
    return dict(op="cross", B=rng.randint(1, 4 if hi < 1600 else 2), lq=_log(rng, 40, 2048),
                lk_lo=rng.randint(max(64, hi // 2), hi), lk_hi=hi, hq=min(hq, 16), hkv=hkv, d=d,
                train=True)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """Per sequence: its new tokens, and its own length (the new ones included)."""
    n = case["B"]
    new = _spread(case["new_lo"], case["new_hi"], n)
    length = _spread(case["own_lo"], case["own_hi"], n)
    if case["own_hi"] > 2 * case["new_hi"]:  # long caches need not be the ones with many new tokens
        new = [new[(5 * i + 1) % n] for i in range(n)] if n % 5 else new[::-1]
    return [(t, max(t, m)) for t, m in zip(new, length)]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        n = sum(t for t, _ in _lengths(case))
        return {"bytes": n * (hq + 2 * hkv) * d * 4, "flops": n * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "prefix":
        pairs = byte = n = 0
        for t, m in _lengths(case):
            pairs += t * (case["prefix"] + m) - t * (t - 1) // 2
            byte += m * hkv * d * 4
            n += t
        byte += case["prefix"] * hkv * d * 4 + n * hq * (d * 4 + 4)
        return {"bytes": byte, "flops": 4 * d * hq * pairs}
    keys = sum(_spread(case["lk_lo"], case["lk_hi"], case["B"]))
    rows = case["B"] * case["lq"] * hq
    byte = keys * hkv * d * 4 + rows * (d * 4 + 4)
    flops = 4 * d * hq * case["lq"] * keys
    if case["train"]:  # o and the gradient of o in, three gradients out, and q, k, v again
        byte = keys * hkv * d * 8 + case["B"] * (case["lk_hi"] * hkv * d * 4) + rows * d * 12
        flops = 14 * d * hq * case["lq"] * keys
    return {"bytes": byte, "flops": flops}


class State:
    pass


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    s = State()
    s.case, s.scale = case, case["d"] ** -0.5
    B, hq, hkv, d = case["B"], case["hq"], case["hkv"], case["d"]
    order = torch.randperm(B, generator=host).tolist()
    if case["op"] == "cross":
        lens = _spread(case["lk_lo"], case["lk_hi"], B)
        s.kv_lens = torch.tensor([lens[i] for i in order], dtype=torch.int32, device=DEV)
        s.q = _normal(gen, B, case["lq"], hq, d)
        kv = _normal(gen, B, case["lk_hi"], 2, hkv, d)  # one projection gives both
        s.k, s.v = kv[:, :, 0], kv[:, :, 1]
        if case["train"]:
            for t in (s.q, s.k, s.v):
                t.requires_grad_()
            s.do = _normal(gen, B, case["lq"], hq, d)
        return s
    pairs = _lengths(case)
    new, length = [pairs[i][0] for i in order], [pairs[i][1] for i in order]
    s.n = sum(new)
    s.max_new, s.max_len = max(new), max(length)
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    s.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s.lens = torch.tensor(length, dtype=torch.int32, device=DEV)
    # pages of the prefix and of every sequence lie anywhere in the cache
    page = case["page"]
    prefix = case.get("prefix", 0)
    n_prefix, n_own = -(-prefix // page), -(-s.max_len // page)
    total = n_prefix + B * n_own
    pages = torch.randperm(total, generator=host).to(torch.int32).to(DEV)
    s.prefix_table = pages[:n_prefix].contiguous()
    s.tables = pages[n_prefix:].view(B, n_own).contiguous()
    s.k_pages = _normal(gen, total, page, hkv, d)
    s.v_pages = _normal(gen, total, page, hkv, d)
    if case["op"] == "append":
        qkv = _normal(gen, s.n, hq + 2 * hkv, d)  # one projection gives all three
        s.q, s.k, s.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        j = torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64)
        s.inv_freq = (500000.0 ** (-j / case["rot"])).float()
    else:
        s.q = _normal(gen, s.n, hq, d)
    return s


# ------------------------------------------------------------------ plain forms
def _token_index(s):
    """Per token: its sequence, and its place among the sequence's own keys."""
    at = torch.arange(s.n, device=DEV)
    seq = (at[:, None] >= s.cu[None, 1:]).sum(1)
    return seq, s.lens[seq] - s.cu[seq + 1] + at


def _rotate(x, cos, sin, rot, inter):
    x = x.float()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1).bfloat16()


def _plain_append(s):
    c = s.case
    seq, place = _token_index(s)
    angle = (place + c["offset"]).double()[:, None] * s.inv_freq.double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    page = s.tables[seq, place // c["page"]].long()
    slot = place % c["page"]
    s.k_pages[page, slot] = _rotate(s.k, cos, sin, c["rot"], c["inter"])
    s.v_pages[page, slot] = s.v
    return _rotate(s.q, cos, sin, c["rot"], c["inter"]), s.k_pages, s.v_pages


def _plain_prefix(s):
    c = s.case
    g, d, page = c["hkv"], c["d"], c["page"]
    r = c["hq"] // g
    seq, place = _token_index(s)
    t = torch.arange(s.max_new, device=DEV)
    tok = (s.cu[:-1, None] + t).clamp(max=s.n - 1)  # [B, T]; rows past a sequence's last are unused
    q = s.q.float()[tok].view(c["B"], s.max_new, g, r, d)
    j = torch.arange(s.max_len, device=DEV)
    rows = s.tables[:, j // page].long()
    k = s.k_pages[rows, j % page].float()
    v = s.v_pages[rows, j % page].float()
    score = torch.einsum("btgrd,bkgd->bgrtk", q, k) * s.scale
    last = s.lens[:, None] - (s.cu[1:] - s.cu[:-1])[:, None] + t
    seen = j <= last[:, :, None]
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1)
    if c["prefix"]:
        i = torch.arange(c["prefix"], device=DEV)
        kp = s.k_pages[s.prefix_table[i // page].long(), i % page].float()
        vp = s.v_pages[s.prefix_table[i // page].long(), i % page].float()
        shared = torch.einsum("btgrd,kgd->bgrtk", q, kp) * s.scale
        top = torch.maximum(top, shared.amax(-1))
        shared = torch.exp(shared - top[..., None])
    weight = torch.exp(score - top[..., None])
    total = weight.sum(-1)
    out = torch.einsum("bgrtk,bkgd->bgrtd", weight, v)
    if c["prefix"]:
        total = total + shared.sum(-1)
        out = out + torch.einsum("bgrtk,kgd->bgrtd", shared, vp)
    out = (out / total[..., None]).flatten(1, 2)  # [B, hq, T, d]
    lse = (top + torch.log(total)).flatten(1, 2)
    at = torch.arange(s.n, device=DEV) - s.cu[seq]
    return out[seq, :, at].bfloat16(), lse[seq, :, at].t().contiguous()


def _plain_cross(s):
    c = s.case
    B, g, d = c["B"], c["hkv"], c["d"]
    r = c["hq"] // g
    q = s.q.detach().float().view(B, c["lq"], g, r, d)
    k, v = s.k.detach().float(), s.v.detach().float()
    score = torch.einsum("btgrd,bkgd->bgrtk", q, k) * s.scale
    seen = torch.arange(k.shape[1], device=DEV) < s.kv_lens[:, None]
    score = torch.where(seen[:, None, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    weight = weight / total
    out = torch.einsum("bgrtk,bkgd->btgrd", weight, v)
    o = out.flatten(2, 3).bfloat16()
    if not c["train"]:
        return o, (top + torch.log(total))[..., 0].flatten(1, 2)
    do = s.do.float().view(B, c["lq"], g, r, d)
    delta = (do * out).sum(-1).permute(0, 2, 3, 1)[..., None]
    ds = weight * (torch.einsum("btgrd,bkgd->bgrtk", do, v) - delta) * s.scale
    dq = torch.einsum("bgrtk,bkgd->btgrd", ds, k).flatten(2, 3)
    dk = torch.einsum("bgrtk,btgrd->bkgd", ds, q)
    dv = torch.einsum("bgrtk,btgrd->bkgd", weight, do)
    return o, dq.bfloat16(), dk.bfloat16(), dv.bfloat16()


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from sequence_parallelism_attn_b200 import autograd, ra
    c = s.case
    if c["op"] == "append":
        q = ra.paged_kv_append(s.q, s.k, s.v, s.k_pages, s.v_pages, s.cu, s.lens, s.tables,
                               s.inv_freq, s.max_new, pos_offset=c["offset"],
                               interleaved=c["inter"])
        return q, s.k_pages, s.v_pages
    if c["op"] == "prefix":
        return ra.prefix_attn_fwd(s.q, s.k_pages, s.v_pages, s.cu, s.lens, s.tables, s.max_new,
                                  max_len=s.max_len, prefix_table=s.prefix_table,
                                  prefix_len=c["prefix"], scale=s.scale,
                                  out_dtype=torch.bfloat16)
    if not c["train"]:
        return ra.cross_attn_fwd(s.q, s.k, s.v, kv_lens=s.kv_lens, scale=s.scale,
                                 out_dtype=torch.bfloat16)
    o = autograd.cross_attention(s.q, s.k, s.v, kv_lens=s.kv_lens, scale=s.scale)
    dq, dk, dv = torch.autograd.grad(o, (s.q, s.k, s.v), s.do)
    return o, dq, dk, dv


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "prefix": _plain_prefix,
            "cross": _plain_cross}[state.case["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    if case["op"] == "cross":
        out, lse = [], []
        grads = [torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in (s.q, s.k, s.v)]
        for b in range(case["B"]):
            n = int(s.kv_lens[b])
            q = s.q.detach()[b].double().transpose(0, 1)  # [hq, lq, d]
            k = s.k.detach()[b, :n].double().transpose(0, 1).repeat_interleave(group, 0)
            v = s.v.detach()[b, :n].double().transpose(0, 1).repeat_interleave(group, 0)
            x = q @ k.mT * s.scale
            l = torch.logsumexp(x, -1, keepdim=True)
            p = torch.exp(x - l)
            o = p @ v
            out.append(o.transpose(0, 1))
            lse.append(l[..., 0])
            if case["train"]:
                do = s.do[b].double().transpose(0, 1)
                dp = do @ v.mT
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s.scale
                grads[0][b] = (ds @ k).transpose(0, 1)
                grads[1][b, :n] = (ds.mT @ q).view(hkv, group, n, d).sum(1).transpose(0, 1)
                grads[2][b, :n] = (p.mT @ do).view(hkv, group, n, d).sum(1).transpose(0, 1)
        return (torch.stack(out), *grads) if case["train"] else (torch.stack(out),
                                                                  torch.stack(lse))
    cu, lens = s.cu.tolist(), s.lens.tolist()
    page = case["page"]
    if case["op"] == "append":
        half = case["rot"] // 2
        q, kp, vp = s.q.double(), s.k_pages.double(), s.v_pages.double()
        i = torch.arange(half, device=DEV)
        a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)

        def turn(x, pos):
            z = torch.complex(x[..., a], x[..., b])
            w = pos.double()[:, None] * s.inv_freq.double()
            z = z * torch.polar(torch.ones_like(w), w)[:, None]
            x = x.clone()
            x[..., a], x[..., b] = z.real, z.imag
            return x

        for n in range(case["B"]):
            own_at = torch.arange(lens[n] - (cu[n + 1] - cu[n]), lens[n], device=DEV)
            pos = own_at + case["offset"]
            q[cu[n]:cu[n + 1]] = turn(q[cu[n]:cu[n + 1]], pos)
            where = (s.tables[n].long()[own_at // page], own_at % page)
            kp[where] = turn(s.k[cu[n]:cu[n + 1]].double(), pos)
            vp[where] = s.v[cu[n]:cu[n + 1]].double()
        return q, kp, vp
    out = torch.empty(s.n, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(hq, s.n, dtype=torch.float64, device=DEV)
    for n in range(case["B"]):
        pages = torch.cat([s.prefix_table, s.tables[n]]).long()
        npre = len(s.prefix_table) * page
        keep = torch.cat([torch.arange(case["prefix"], device=DEV),
                          npre + torch.arange(lens[n], device=DEV)])
        k = s.k_pages[pages].flatten(0, 1)[keep].double().transpose(0, 1)
        v = s.v_pages[pages].flatten(0, 1)[keep].double().transpose(0, 1)
        q = s.q[cu[n]:cu[n + 1]].double().transpose(0, 1)  # [hq, t, d]
        t = q.shape[1]
        x = q @ k.repeat_interleave(group, 0).mT * s.scale
        hidden = torch.ones(t, t, dtype=torch.bool, device=DEV).triu(1)  # later new tokens
        x[:, :, x.shape[-1] - t:].masked_fill_(hidden, -math.inf)
        l = torch.logsumexp(x, -1)
        out[cu[n]:cu[n + 1]] = (torch.exp(x - l[..., None]) @ v.repeat_interleave(group, 0)
                                ).transpose(0, 1)
        lse[:, cu[n]:cu[n + 1]] = l
    return out, lse
