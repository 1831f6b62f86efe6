"""Cases for the operators around the quantised products of a layer.

Three operators: ``norm`` (the residual's addition and the RMS norm before the projections, its output in
bf16 or in E4M3 with scales), ``lora`` (low-rank adapters of many requests beside a shared projection) and
``route`` (routing to experts: sigmoid or softmax scores, a bias for balance, groups, top-k, weights).

``run`` computes each in plain torch operations or, with ``own`` set, through the package's entry points
``rms_norm``, ``rms_norm_fp8``, ``lora`` and ``route`` with a ``RouteRule``.
"""
import math
import random

import torch

own = False

EPS = 1e-6
# Hidden sizes and widths of the quantised products that this repository measures: inputs and outputs of a projection.
PROJECTIONS = {
    "qkv": (5120, 7168),    # 40 + 2 x 8 heads of 128
    "out": (6144, 5120),    # 24 heads of 256 back to the hidden size
    "up": (5120, 17408),    # one of gate and up
    "down": (17408, 5120),
    "small": (2048, 2560),  # 32 + 2 x 4 heads of 64
}


def listed():
    return [
        # one token of one user between two projections: latency
        dict(name="norm_one", op="norm", rows=1, k=5120, residual=True, fp8=-1, offset=0.0),
        # one token of each of 64 users, for products of 8-bit activations in groups of 128
        dict(name="norm_batch", op="norm", rows=64, k=5120, residual=True, fp8=128, offset=0.0),
        # a prompt of ordinary length
        dict(name="norm_prompt", op="norm", rows=4096, k=5120, residual=True, fp8=-1, offset=1.0),
        # prompts of several users, an odd number of rows, one scale a row
        dict(name="norm_ragged", op="norm", rows=18001, k=2048, residual=True, fp8=0, offset=0.0),
        # one token of one user with an adapter: latency
        dict(name="lora_one", op="lora", proj="qkv", seqs=1, rows=1, adapters=8, rank=16, mixed=False, seed=1),
        # one token of each of 64 users, most of them with an adapter, some adapters shared, ranks of 8 to 64
        dict(name="lora_batch", op="lora", proj="qkv", seqs=64, rows=64, adapters=48, rank=64, mixed=True, seed=2),
        # prompts of seven users, odd lengths, in one call
        dict(name="lora_prompts", op="lora", proj="out", seqs=7, rows=3999, adapters=5, rank=16, mixed=False, seed=3),
        # long prompts of three users through the widest projection
        dict(name="lora_long", op="lora", proj="up", seqs=3, rows=8192, adapters=3, rank=64, mixed=False, seed=4),
        # one token: latency; scores by sigmoid, a bias, four of eight groups
        dict(name="route_one", op="route", rows=1, experts=256, topk=8, score="sigmoid", bias=True, groups=8, kept=4, best=2,
             norm=True, scale=2.5),
        # one token of each of 64 users
        dict(name="route_batch", op="route", rows=64, experts=512, topk=10, score="softmax", bias=True, groups=1, kept=1, best=1,
             norm=True, scale=1.0),
        # a long prompt
        dict(name="route_prompt", op="route", rows=8192, experts=512, topk=10, score="sigmoid", bias=True, groups=1, kept=1,
             best=1, norm=True, scale=1.0),
        # prompts of odd lengths, groups whose size is no power of two, the best expert of a group for the group, weights as they are
        dict(name="route_ragged", op="route", rows=5001, experts=160, topk=6, score="softmax", bias=False, groups=8, kept=3, best=1,
             norm=False, scale=16.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "lora", "route"])
    if op == "norm":
        k = rng.choice([2048, 5120, 6144, _log(rng, 256, 17408)])
        return dict(op=op, rows=_log(rng, 1, 36000000 // k), k=k, residual=rng.random() < 0.7, fp8=rng.choice([-1, -1, 0, 32, 64, 128]),
                    offset=rng.choice([0.0, 1.0]))
    if op == "lora":
        proj = rng.choice(sorted(PROJECTIONS))
        seqs = _log(rng, 1, 96)
        rows = seqs * rng.randint(1, 3) if rng.random() < 0.5 else seqs + _log(rng, 1, 6000)
        return dict(op=op, proj=proj, seqs=seqs, rows=rows, adapters=_log(rng, 1, 64), rank=rng.choice([8, 16, 32, 64]),
                    mixed=rng.random() < 0.5, seed=rng.randrange(1 << 20))
    groups = rng.choice([1, 1, 2, 4, 8, 16])
    experts = groups * rng.randint(max(2, 24 // groups), 512 // groups)
    kept = rng.randint(max(1, groups // 4), groups)
    return dict(op=op, rows=_log(rng, 1, 8000), experts=experts, topk=rng.randint(1, min(16, kept * (experts // groups))),
                score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6, groups=groups, kept=kept,
                best=rng.choice([1, 2]), norm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]))


def _requests(case):
    """(adapter of every row, -1 for none; rank of every adapter)."""
    r = random.Random(case["seed"])
    n, seqs = case["rows"], case["seqs"]
    cuts = [0, *sorted(r.sample(range(1, n), seqs - 1)), n]
    ids = []
    for a, b in zip(cuts, cuts[1:]):
        who = -1 if seqs > 1 and r.random() < 0.1 else r.randrange(case["adapters"])
        ids += [who] * (b - a)
    ranks = [r.choice([x for x in (8, 12, 16, 32, 64) if x <= case["rank"]]) if case["mixed"] else case["rank"]
             for _ in range(case["adapters"])]
    return ids, ranks


def _pad8(n):
    return -(-n // 8) * 8


def work(case):
    n = case["rows"]
    if case["op"] == "norm":
        k, g = case["k"], case["fp8"]
        out = 2 * n * k if g < 0 else n * k + 4 * n * (1 if g == 0 else -(-k // g))
        return {"bytes": 2 * n * k + (4 * n * k if case["residual"] else 0) + 2 * k + out, "flops": 5 * n * k}
    if case["op"] == "lora":
        k, m = PROJECTIONS[case["proj"]]
        ids, ranks = _requests(case)
        used = sum(ranks[a] for a in set(ids) if a >= 0)
        return {"bytes": 2 * (n * k + 2 * n * m + used * (k + m)) + 4 * n, "flops": 2 * (k + m) * sum(ranks[a] for a in ids if a >= 0)}
    return {"bytes": 4 * n * case["experts"] + 8 * n * case["topk"], "flops": 8 * n * case["experts"]}


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, device=dev, generator=g)

    n, s = case["rows"], dict(case=case)
    if case["op"] == "norm":
        k, ld = case["k"], _pad8(case["k"])
        # a residual stream: a few channels much larger than the others
        channel = torch.exp(0.5 * randn(k)) * torch.where(torch.rand(k, device=dev, generator=g) < 0.002, 20.0, 1.0)
        rows = lambda dtype: torch.empty(n, ld, dtype=dtype, device=dev)[:, :k]  # noqa: E731
        s["x"] = rows(torch.bfloat16).copy_(randn(n, k))
        s["residual"] = rows(torch.bfloat16).copy_(randn(n, k) * channel) if case["residual"] else None
        s["weight"] = (1.0 - case["offset"] + 0.2 * randn(k)).to(torch.bfloat16)
        s["sum"] = rows(torch.bfloat16) if case["residual"] else None
        s["out"] = rows(torch.bfloat16 if case["fp8"] < 0 else torch.float8_e4m3fn)
        s["scales"] = torch.empty(n, 1 if case["fp8"] == 0 else -(-k // case["fp8"]), device=dev) if case["fp8"] >= 0 else None
    elif case["op"] == "lora":
        k, m = PROJECTIONS[case["proj"]]
        ids, ranks = _requests(case)
        top, count = case["rank"], case["adapters"]
        s["x"] = randn(n, k).to(torch.bfloat16)
        s["y"] = randn(n, m).to(torch.bfloat16)
        s["a"] = (randn(count, top, k) * k ** -0.5).to(torch.bfloat16)
        s["b"] = (randn(count, m, top) * 0.05).to(torch.bfloat16)
        s["scale"] = 0.5 + 1.5 * torch.rand(count, device=dev, generator=g)
        s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device=dev)
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device=dev)
        s["out"] = torch.empty_like(s["y"])
    else:
        s["logits"] = 1.5 * randn(n, case["experts"])
        s["bias"] = 0.1 * randn(case["experts"]) if case["bias"] else None
    if own:
        import prefill_dequant_gemv_gb300 as lib
        s["lib"] = lib
        if case["op"] == "lora":
            s["adapters"] = lib.LoraAdapters(s["a"], s["b"], s["scale"], s["ranks"])
            s["ws"] = lib.Workspace(lib.lora_workspace_size(s["adapters"], n), dev)
        elif case["op"] == "route":
            s["rule"] = lib.RouteRule(score=case["score"], bias=s["bias"], groups=case["groups"], topk_groups=case["kept"],
                                      group_best=case["best"], renormalise=case["norm"], scale=case["scale"])
            s["ws"] = lib.Workspace(lib.qmoe_route_workspace_size(n, case["experts"], case["topk"]), dev)
    return s


def run(s):
    case = s["case"]
    if own:
        lib = s["lib"]
        if case["op"] == "lora":
            return lib.lora(s["adapters"], s["ids"], s["x"], s["y"], out=s["out"], workspace=s["ws"])
        if case["op"] == "route":
            ids, weights, _ = lib.route(s["logits"], case["topk"], workspace=s["ws"], rule=s["rule"])
            return {"ids": ids, "weights": weights}
        if case["fp8"] < 0:
            y, h = lib.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, weight_offset=case["offset"], out=s["out"],
                                sum_out=s["sum"])
            return {"y": y, "sum": h}
        codes, scales, h = lib.rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=EPS, weight_offset=case["offset"],
                                            group=case["fp8"], out=s["out"], scales=s["scales"], sum_out=s["sum"])
        return {"codes": codes, "scales": scales, "sum": h}
    return _norm(s) if case["op"] == "norm" else _lora(s) if case["op"] == "lora" else _route(s)


# ---------------------------------------------------------------------------- plain forms
def _norm(s):
    case = s["case"]
    h = None
    x = s["x"].float()
    if case["residual"]:
        h = (x + s["residual"].float()).to(torch.bfloat16)
        x = h.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (s["weight"].float() + case["offset"])
    if case["fp8"] < 0:
        return {"y": y.to(torch.bfloat16), "sum": h}
    k, g = case["k"], case["fp8"] or case["k"]
    groups = torch.nn.functional.pad(y, (0, -k % g)).view(len(y), -1, g)
    scales = (groups.abs().amax(-1) / 448.0).clamp_min(2.0 ** -100)
    codes = (groups / scales[..., None]).clamp(-448.0, 448.0).flatten(1)[:, :k].to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": scales, "sum": h}


def _lora(s):
    # every row through every adapter, then its own one's share; one product each way
    case = s["case"]
    count, top = case["adapters"], case["rank"]
    h = torch.matmul(s["x"].float(), s["a"].float().flatten(0, 1).T).view(-1, count, top)
    mine = s["ids"][:, None] == torch.arange(count, device="cuda")
    live = torch.arange(top, device="cuda") < s["ranks"][:, None]
    h = torch.where(mine[..., None] & live, h * s["scale"][:, None], 0.0).flatten(1)
    return torch.matmul(h, s["b"].float().transpose(1, 2).flatten(0, 1)).add_(s["y"].float()).to(torch.bfloat16)


def _route(s):
    # in 64 bits: which of two experts comes first can hang on the last bits
    case = s["case"]
    logits = s["logits"].double()
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        per = choice.view(len(choice), case["groups"], -1)
        value = per.sort(dim=-1, descending=True).values[..., :case["best"]].sum(-1)
        kept = value.sort(dim=-1, descending=True, stable=True).indices[:, :case["kept"]]
        out = torch.ones_like(value, dtype=torch.bool).scatter_(1, kept, False)
        choice = per.masked_fill(out[..., None], -torch.inf).flatten(1)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk"]]
    weights = score.gather(1, ids)
    if case["norm"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (weights * case["scale"]).float()}


# ---------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        k = case["k"]
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(torch.bfloat16).double()
        root = torch.sqrt(torch.linalg.vector_norm(h, dim=1).square() / k + EPS)
        y = h / root[:, None] * (s["weight"].double() + case["offset"])
        done = {"sum": h if case["residual"] else None}
        if case["fp8"] < 0:
            return {"y": y, **done}
        size = case["fp8"] or k
        scales, codes = torch.empty_like(s["scales"], dtype=torch.float64), torch.empty_like(y)
        for i, lo in enumerate(range(0, k, size)):
            part = y[:, lo:lo + size]
            scales[:, i] = torch.maximum(part.amax(1), -part.amin(1)) / 448
            scales[:, i].clamp_(min=2.0 ** -100)
            codes[:, lo:lo + size] = (part / scales[:, i:i + 1]).to(torch.float8_e4m3fn).double()
        return {"codes": codes, "scales": scales, **done}
    if case["op"] == "lora":
        out = s["y"].double()
        for i, rank in enumerate(s["ranks"].tolist()):
            rows = (s["ids"] == i).nonzero()[:, 0]
            h = s["x"][rows].double() @ s["a"][i, :rank].double().T
            out[rows] += s["scale"][i].double() * (h @ s["b"][i, :, :rank].double().T)
        return out
    logits = s["logits"].cpu().double()
    score = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)
    choice = score + (0 if s["bias"] is None else s["bias"].cpu().double())
    size = case["experts"] // case["groups"]
    value = torch.stack([choice[:, i * size:(i + 1) * size].topk(case["best"], 1).values.sum(1) for i in range(case["groups"])], 1)
    order = torch.argsort(value, dim=1, descending=True, stable=True)
    for i in range(case["kept"], case["groups"]):
        gone = order[:, i:i + 1] * size + torch.arange(size)
        choice.scatter_(1, gone, -math.inf)
    ids = torch.argsort(choice, dim=1, descending=True, stable=True)[:, :case["topk"]]
    weights = torch.gather(score, 1, ids)
    if case["norm"]:
        weights /= weights.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": weights * case["scale"]}
