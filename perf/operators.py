"""Cases for the attention operators over the 8-bit paged key/value cache.

Two operators: ``append`` (per-head RMS norms of queries and keys, the rotary embedding and the
write of keys and values into the E4M3 cache, in one pass) and ``attend`` (attention of the
new tokens over the cache, from one decoded token a sequence to whole prompts).

``run`` computes either in plain fp32 torch operations or, with ``own`` set, through the
package's entry points ``kv_append`` and ``attention``.
"""
import math
import random

import torch

own = False

# Head layouts.  "h5120" is a hidden size of 5120 as 40 heads of 128 with 8 key/value heads;
# "h6144" 24 heads of 256 with 4 key/value heads, whose 6144 attention outputs feed a 5120 x 6144
# output projection, with a quarter of each head rotated; "h2048" a hidden size of 2048 as 32
# heads of 64 with 4 key/value heads.
HEADS = {
    "h5120": {"hq": 40, "hkv": 8, "d": 128, "rot": 128, "offset": 0.0, "interleaved": False},
    "h6144": {"hq": 24, "hkv": 4, "d": 256, "rot": 64, "offset": 1.0, "interleaved": False},
    "h2048": {"hq": 32, "hkv": 4, "d": 64, "rot": 64, "offset": 0.0, "interleaved": True},
}
EPS = 1e-6


def listed():
    return [
        # one decoded token of one sequence: the latency of a single user's step
        dict(name="append_one", op="append", heads="h5120", seqs=1, new=1, ctx=900, page=64, ragged=0),
        # one decoded token of each of 64 users, most of them inside a page that holds tokens
        dict(name="append_batch", op="append", heads="h5120", seqs=64, new=1, ctx=512, page=64, ragged=1),
        # a whole prompt into an empty cache
        dict(name="append_prompt", op="append", heads="h5120", seqs=1, new=4096, ctx=0, page=64, ragged=0),
        # prompts and chunks of several users in one call, odd lengths, small pages, wide heads
        dict(name="append_ragged", op="append", heads="h6144", seqs=7, new=1201, ctx=300, page=16, ragged=2),
        # one decoded token, short context: latency
        dict(name="decode_one", op="attend", heads="h5120", seqs=1, new=1, ctx=776, page=64, window=0, ragged=0),
        # one decoded token, one long document: the length has to be split over the GPU
        dict(name="decode_long", op="attend", heads="h6144", seqs=1, new=1, ctx=131000, page=64, window=0, ragged=0),
        # one decoded token of each of 64 users with very different lengths
        dict(name="decode_batch", op="attend", heads="h5120", seqs=64, new=1, ctx=8192, page=32, window=0, ragged=3),
        # speculative verification: four tokens of each of 16 users
        dict(name="verify", op="attend", heads="h6144", seqs=16, new=4, ctx=8000, page=64, window=0, ragged=4),
        # a prompt of ordinary length
        dict(name="prefill", op="attend", heads="h5120", seqs=1, new=2048, ctx=0, page=64, window=0, ragged=0),
        # a chunk of a long prompt, most of it in the cache already
        dict(name="prefill_chunk", op="attend", heads="h6144", seqs=1, new=512, ctx=32768, page=64, window=0, ragged=0),
        # several prompts of odd lengths under a sliding window, small heads and pages
        dict(name="prefill_window", op="attend", heads="h2048", seqs=6, new=2777, ctx=333, page=16, window=1024, ragged=5),
        # the longest prompt
        dict(name="prefill_long", op="attend", heads="h5120", seqs=1, new=8192, ctx=0, page=64, window=0, ragged=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, page, ragged = rng.choice(sorted(HEADS)), rng.choice([16, 32, 64, 128]), rng.randrange(1, 1 << 20)
    kind = rng.choice(["append_few", "append_many", "decode", "verify", "prefill"])
    if kind == "append_few":
        return dict(op="append", heads=heads, seqs=_log(rng, 1, 96), new=rng.randint(1, 4), ctx=_log(rng, 1, 700), page=page, ragged=ragged)
    if kind == "append_many":
        seqs = _log(rng, 1, 12)
        return dict(op="append", heads=heads, seqs=seqs, new=_log(rng, 5, 6000 // seqs), ctx=_log(rng, 1, 600), page=page, ragged=ragged)
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    if kind in ("decode", "verify"):
        seqs = _log(rng, 1, 64)
        return dict(op="attend", heads=heads, seqs=seqs, new=1 if kind == "decode" else rng.randint(2, 4),
                    ctx=_log(rng, 50, min(100000, 400000 // seqs)), page=page, window=window, ragged=ragged)
    seqs = _log(rng, 1, 6)
    new = _log(rng, 5, 4000 // seqs)
    return dict(op="attend", heads=heads, seqs=seqs, new=new, ctx=_log(rng, 1, 16000 // seqs), page=page, window=window, ragged=ragged)


def _lengths(case):
    """(new tokens, length with them) of every sequence.  ragged 0: all alike; else drawn from
    1..new and 0..ctx (one sequence at both maxima), new left alone where it is 4 or less."""
    n, new, ctx = case["seqs"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * n, [ctx + new] * n
    r = random.Random(case["ragged"])
    news = [new if new <= 4 or i == 0 else r.randint(max(1, new // 8), new) for i in range(n)]
    ctxs = [ctx if i == 0 else r.randint(0, ctx) for i in range(n)]
    return news, [c + t for c, t in zip(ctxs, news)]


def work(case):
    h = HEADS[case["heads"]]
    hq, hkv, d = h["hq"], h["hkv"], h["d"]
    news, lens = _lengths(case)
    n = sum(news)
    if case["op"] == "append":
        pages = sum(-(-l // case["page"]) - (l - t) // case["page"] for t, l in zip(news, lens))
        return {"bytes": 2 * n * (hq + 2 * hkv) * d + 2 * n * hq * d + 2 * n * hkv * d + 8 * pages * hkv + 4 * n * h["rot"],
                "flops": n * (hq + hkv) * d * 8 + n * hkv * d * 4}
    w = case["window"] or (1 << 40)
    seen = sum(min(p + 1, w) for t, l in zip(news, lens) for p in range(l - t, l))
    read = sum(min(l, t - 1 + w) for t, l in zip(news, lens))
    return {"bytes": 2 * read * hkv * d + 8 * hkv * (read // case["page"]) + 4 * n * hq * d, "flops": 4 * d * hq * seen}


def _power_of_two(x):
    return ((x + 127) << 23).to(torch.int32).view(torch.float32)


def _scale(amax):
    """The smallest power of two s (2^-100 to 2^120) with amax <= 448 s."""
    m, e = torch.frexp(amax)
    return _power_of_two((e.to(torch.int32) - 9 + (m > 0.875)).clamp(-100, 120))


def _quantised(g, dev, pages, hkv, page, d, spread):
    """Codes and scales of pages of normal values whose size differs from page to page and channel to channel."""
    x = torch.randn(pages, hkv, page, d, device=dev, generator=g, dtype=torch.float32)
    x *= torch.exp(spread * torch.randn(pages, hkv, 1, 1, device=dev, generator=g))
    x *= torch.exp(0.3 * torch.randn(1, hkv, 1, d, device=dev, generator=g))
    s = _scale(x.abs().amax(dim=(2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    h, dev = HEADS[case["heads"]], "cuda"
    hq, hkv, d, page = h["hq"], h["hkv"], h["d"], case["page"]
    g = torch.Generator(device=dev).manual_seed(int(seed))
    news, lens = _lengths(case)
    n, top = sum(news), max(lens)
    per = [-(-l // page) for l in lens]
    # the sequences' pages lie scattered over the pool, as they do after some hours of serving
    order = torch.randperm(sum(per), device=dev, generator=g).to(torch.int32)
    table = torch.zeros(len(lens), max(per), dtype=torch.int32, device=dev)
    at = 0
    for b, c in enumerate(per):
        table[b, :c] = order[at:at + c]
        at += c
    starts = [0]
    for t in news:
        starts.append(starts[-1] + t)
    kc, ks = _quantised(g, dev, sum(per), hkv, page, d, 0.2)
    vc, vs = _quantised(g, dev, sum(per), hkv, page, d, 0.5)
    s = dict(case=case, h=h, kc=kc, ks=ks, vc=vc, vs=vs, table=table, top=top, max_new=max(news),
             start=torch.tensor(starts, dtype=torch.int32, device=dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if case["op"] == "append":
        # the rows of a fused QKV projection
        qkv = torch.randn(n, (hq + 2 * hkv) * d, device=dev, generator=g) * 1.5
        qkv = qkv.to(torch.bfloat16).view(n, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        one = 1.0 - h["offset"]
        s["qw"], s["kw"] = ((one + 0.2 * torch.randn(d, device=dev, generator=g)).to(torch.bfloat16) for _ in range(2))
        f = 10000.0 ** (-torch.arange(0, h["rot"], 2, device=dev, dtype=torch.float64) / h["rot"])
        a = torch.arange(top + 8, device=dev, dtype=torch.float64)[:, None] * f
        s["cs"] = torch.cat([a.cos(), a.sin()], 1).float()
        s["out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=dev)
    else:
        s["q"] = (1.5 * torch.randn(n, hq, d, device=dev, generator=g)).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
    if own:
        import prefill_dequant_gemv_gb300 as lib
        s["lib"] = lib
        s["cache"] = lib.KVCache(kc, vc, ks, vs)
        s["batch"] = lib.KVBatch(s["start"], s["lens"], table, max_new=s["max_new"], max_len=top)
        if case["op"] == "append":
            s["nr"] = lib.NormRope(q_weight=s["qw"], k_weight=s["kw"], eps=EPS, weight_offset=h["offset"], cos_sin=s["cs"],
                                   interleaved=h["interleaved"])
            s["ws"] = lib.Workspace(lib.qkv_append_workspace_size(), dev)
        else:
            s["ws"] = lib.Workspace(lib.attention_workspace_size(s["cache"], s["batch"], n, hq), dev)
    return s


def run(s):
    if own:
        lib = s["lib"]
        if s["case"]["op"] == "append":
            q = lib.kv_append(s["cache"], s["batch"], s["q"], s["k"], s["v"], s["nr"], out=s["out"], workspace=s["ws"])
            return {"q": q, "k_codes": s["kc"], "k_scales": s["ks"], "v_codes": s["vc"], "v_scales": s["vs"]}
        return lib.attention(s["cache"], s["batch"], s["q"], s["h"]["d"] ** -0.5, window=s["case"]["window"], out=s["out"],
                             workspace=s["ws"])
    return _append(s) if s["case"]["op"] == "append" else _attend(s)


# ---------------------------------------------------------------------------- plain forms
def _rows(s, n):
    """Sequence and position of every row."""
    i = torch.arange(n, device="cuda")
    b = (i[:, None] >= s["start"][1:]).sum(1)
    return b, s["lens"].long()[b] - s["start"].long()[b + 1] + i


def _norm_rope(x, w, pos, s):
    h = s["h"]
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * (w.float() + h["offset"])
    half = h["rot"] // 2
    cos, sin = s["cs"][pos, None, :half], s["cs"][pos, None, half:]
    if h["interleaved"]:
        a, b = y[..., 0:h["rot"]:2], y[..., 1:h["rot"]:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:h["rot"]]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., h["rot"]:]], -1)


def _store(s, x, codes, scales, page, off, page0, off0):
    """x [n][heads][d] into the cache: scales of the touched pages, the tokens that they hold already, the new ones."""
    amax = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax")
    touched = torch.zeros(scales.shape[0], 1, dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    old = scales[page0]
    need = _scale(amax)
    need[page0] = torch.where(off0[:, None] > 0, torch.maximum(need[page0], old), need[page0])
    scales.copy_(torch.where(touched, need, scales))
    raw = codes.view(torch.uint8)
    held = codes[page0].float() * (old / need[page0])[:, :, None, None]
    keep = torch.arange(codes.shape[2], device="cuda")[:, None] < off0[:, None, None, None]
    raw[page0] = torch.where(keep, held.to(torch.float8_e4m3fn).view(torch.uint8), raw[page0])
    raw[page, :, off] = (x / scales[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _append(s):
    size = s["case"]["page"]
    b, pos = _rows(s, s["q"].shape[0])
    first = s["lens"].long() - (s["start"][1:] - s["start"][:-1]).long()
    q = _norm_rope(s["q"], s["qw"], pos, s).to(torch.bfloat16)
    k = _norm_rope(s["k"], s["kw"], pos, s)
    page, off = s["table"][b, pos // size].long(), pos % size
    page0 = s["table"].gather(1, (first // size)[:, None])[:, 0].long()
    _store(s, k, s["kc"], s["ks"], page, off, page0, first % size)
    _store(s, s["v"].float(), s["vc"], s["vs"], page, off, page0, first % size)
    return {"q": q, "k_codes": s["kc"], "k_scales": s["ks"], "v_codes": s["vc"], "v_scales": s["vs"]}


def _attend(s):
    h, size = s["h"], s["case"]["page"]
    hq, hkv, d = h["hq"], h["hkv"], h["d"]
    table = s["table"].long()
    k, v = ((c[table].float() * sc[table][..., None, None]).transpose(1, 2).flatten(2, 3)
            for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))  # [b][hkv][length][d]
    n, nb, t, length = s["q"].shape[0], len(s["lens"]), s["max_new"], k.shape[2]
    b, pos = _rows(s, n)
    slot = b * t + torch.arange(n, device="cuda") - s["start"].long()[b]
    q = torch.zeros(nb * t, hq, d, device="cuda")
    q[slot] = s["q"].float()
    at = torch.full((nb * t,), -1, device="cuda", dtype=torch.long)
    at[slot] = pos
    q = q.view(nb, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(nb, hkv, -1, d)
    score = torch.matmul(q, k.transpose(2, 3)).view(nb, hq, t, length).mul_(d ** -0.5)
    j = torch.arange(length, device="cuda")
    at = at.view(nb, 1, t, 1)
    seen = j <= at
    if s["case"]["window"]:
        seen = seen & (j > at - s["case"]["window"])
    score.masked_fill_(~seen, -torch.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -torch.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(nb, hkv, -1, length), v).view(nb, hq, t, d) / torch.where(total == 0, 1.0, total)
    return o.transpose(1, 2).reshape(nb * t, hq, d)[slot].to(torch.bfloat16)


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    h, news, lens = s["h"], *_lengths(case)
    hq, hkv, d, size = h["hq"], h["hkv"], h["d"], case["page"]
    starts = s["start"].tolist()
    if case["op"] == "attend":
        out = torch.zeros(starts[-1], hq, d, dtype=torch.float64, device="cuda")
        grp = hq // hkv
        for b, (t, length) in enumerate(zip(news, lens)):
            ids = s["table"][b, :-(-length // size)].long()
            pos = torch.arange(length - t, length, device="cuda").repeat(grp)[:, None]
            j = torch.arange(length, device="cuda")
            hidden = j > pos
            if case["window"]:
                hidden |= j <= pos - case["window"]
            for i in range(hkv):
                k, v = ((c[ids, i].double() * sc[ids, i].double()[:, None, None]).reshape(-1, d)[:length]
                        for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
                q = s["q"][starts[b]:starts[b + 1], i * grp:(i + 1) * grp].double().transpose(0, 1).reshape(-1, d)
                p = torch.softmax((q @ k.T / math.sqrt(d)).masked_fill_(hidden, -math.inf), -1)
                out[starts[b]:starts[b + 1], i * grp:(i + 1) * grp] = (p @ v).view(grp, t, d).transpose(0, 1)
        return out

    half, rot = h["rot"] // 2, h["rot"]
    pos = torch.cat([torch.arange(l - t, l) for t, l in zip(news, lens)]).cuda()
    angle = s["cs"][pos].double()

    def turn(x, w):
        x = x.double()
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * (w.double() + h["offset"])
        pairs = [(2 * i, 2 * i + 1) if h["interleaved"] else (i, i + half) for i in range(half)]
        a, b = (torch.tensor([p[i] for p in pairs], device="cuda") for i in (0, 1))
        y = x.clone()
        y[..., a] = x[..., a] * angle[:, None, :half] - x[..., b] * angle[:, None, half:]
        y[..., b] = x[..., b] * angle[:, None, :half] + x[..., a] * angle[:, None, half:]
        return y

    done = {}
    for name, x, codes, scales in (("k", turn(s["k"], s["kw"]), s["kc"], s["ks"]), ("v", s["v"].double(), s["vc"], s["vs"])):
        codes, scales = codes.double(), scales.double()
        table = s["table"].tolist()
        for b, (t, length) in enumerate(zip(news, lens)):
            for at in range((length - t) // size, -(-length // size)):
                lo, hi, pg = max(length - t, at * size), min(length, (at + 1) * size), table[b][at]
                new = x[starts[b] + lo - length + t:starts[b] + hi - length + t].transpose(0, 1)  # [hkv][tokens][d]
                m, e = torch.frexp(new.abs().amax((1, 2)) / 448)
                need = torch.exp2((e - (m == 0.5).int()).clamp(-100, 120).double())
                held = lo - at * size
                if held:
                    need = torch.maximum(need, scales[pg])
                    codes[pg, :, :held] = (codes[pg, :, :held] * (scales[pg] / need)[:, None, None]).to(torch.float8_e4m3fn).double()
                scales[pg] = need
                codes[pg, :, held:held + hi - lo] = (new / need[:, None, None]).to(torch.float8_e4m3fn).double()
        done[name + "_codes"], done[name + "_scales"] = codes, scales
    return {"q": turn(s["q"], s["qw"]), **done}
