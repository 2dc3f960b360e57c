"""Row operators inside a language model's blocks and at its end: the norm of
each head's queries and keys with the position rotation in the same pass, the
log-probability of a token with the entropy and the top alternatives, the
routing of tokens to experts; each with its gradient.

listed() and draw() give cases, prepare() their inputs, run() one call of an
operator: in plain torch operations, or (own) through the library's entry
points; exact() is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NEG = float("-inf")


def listed():
    return [
        # one token of each of 16 running requests: latency counts
        {"name": "qk_fwd_bf16_16x32+8x128", "op": "qk_fwd", "dtype": "bf16", "tokens": 16, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "pairs": "halves", "seqs": 16, "pad": 0.0},
        # prompts of a serving batch, or a training batch, with grouped key heads
        {"name": "qk_fwd_bf16_16384x32+8x128", "op": "qk_fwd", "dtype": "bf16", "tokens": 16384, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "pairs": "halves", "seqs": 4, "pad": 0.0},
        # the gradient on a training batch
        {"name": "qk_bwd_bf16_8192x32+8x128", "op": "qk_bwd", "dtype": "bf16", "tokens": 8192, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "pairs": "halves", "seqs": 4, "pad": 0.0},
        # a ragged, padded batch: half of each head rotated, neighbours paired
        {"name": "qk_bwd_f16_2777x12+12x80", "op": "qk_bwd", "dtype": "f16", "tokens": 2777, "hq": 12, "hk": 12, "d": 80,
         "rot": 40, "pairs": "neighbours", "seqs": 7, "pad": 0.1},
        # the sampled tokens of a decoding step with a few alternatives
        {"name": "top_fwd_bf16_16x32768_5", "op": "top_fwd", "dtype": "bf16", "rows": 16, "n": 32768, "k": 5, "out": 0.0, "masked": 0.0},
        # scoring a batch: prompts and padding take no part
        {"name": "top_fwd_bf16_4096x131072_20", "op": "top_fwd", "dtype": "bf16", "rows": 4096, "n": 131072, "k": 20, "out": 0.25, "masked": 0.0},
        # an odd vocabulary in binary32, half of it ruled out by a grammar
        {"name": "top_fwd_f32_513x50001_8", "op": "top_fwd", "dtype": "f32", "rows": 513, "n": 50001, "k": 8, "out": 0.1, "masked": 0.5},
        # a training step with an entropy bonus and a distillation term on the teacher's top tokens
        {"name": "top_bwd_bf16_2048x131072_8", "op": "top_bwd", "dtype": "bf16", "rows": 2048, "n": 131072, "k": 8, "out": 0.25, "masked": 0.0},
        # a small model's router
        {"name": "route_fwd_f32_64x64_6", "op": "route_fwd", "dtype": "f32", "tokens": 64, "experts": 64, "k": 6, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": False},
        # a large batch through a router with a bias for balance and limited groups
        {"name": "route_fwd_bf16_65536x256_8", "op": "route_fwd", "dtype": "bf16", "tokens": 65536, "experts": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True},
        # the gradient of renormalised softmax weights on a training batch
        {"name": "route_bwd_bf16_16384x128_8", "op": "route_bwd", "dtype": "bf16", "tokens": 16384, "experts": 128, "k": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": True, "balance": False},
        # the same with the gradient of a balance term on every score
        {"name": "route_bwd_f32_8191x160_6", "op": "route_bwd", "dtype": "f32", "tokens": 8191, "experts": 160, "k": 6, "score": "softmax",
         "bias": False, "groups": 8, "top_groups": 3, "group_top": 1, "renorm": False, "balance": True},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; half of them multiples of 64 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "top_fwd", "top_bwd", "route_fwd", "route_bwd"])
    c = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if op.startswith("qk"):
        c["hk"] = rng.choice([1, 2, 4, 5, 8, 12, 16])
        c["hq"] = c["hk"] * rng.choice([1, 2, 3, 4, 7, 8])
        c["d"] = rng.choice([32, 64, 64, 72, 80, 96, 112, 128, 128, 128, 192, 256, 50])
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 4 * 2, 16])
        c["pairs"] = rng.choice(["halves", "halves", "neighbours"])
        c["tokens"] = _size(rng, 1, min(16384, 2 ** 25 // ((c["hq"] + c["hk"]) * c["d"])))
        c["seqs"] = c["tokens"] if rng.random() < 0.3 else rng.randint(1, min(16, c["tokens"]))
        c["pad"] = rng.choice([0.0, 0.0, 0.05, 0.3])
    elif op.startswith("top"):
        c["n"] = _size(rng, 1000, 160000)
        c["rows"] = _size(rng, 1, min(8192, 2 ** 27 // c["n"]))
        c["k"] = rng.choice([0, 1, 2, 5, 8, 20, 20, 32])
        c["out"] = round(rng.uniform(0.0, 0.5), 2)
        c["masked"] = rng.choice([0.0, 0.0, 0.3, 0.9])
    else:
        c["groups"] = rng.choice([1, 1, 1, 4, 8])
        c["experts"] = c["groups"] * rng.randint(4, 512 // c["groups"] if c["groups"] > 1 else 256)
        c["tokens"] = _size(rng, 1, min(32768, 2 ** 23 // c["experts"]))
        c["top_groups"] = rng.randint(1, c["groups"])
        c["group_top"] = rng.choice([1, 2])
        c["k"] = min(rng.choice([1, 2, 4, 6, 8, 8, 10]), c["experts"] // c["groups"] * c["top_groups"])
        c["score"] = rng.choice(["softmax", "sigmoid"])
        c["bias"] = rng.random() < 0.5
        c["renorm"] = rng.random() < 0.6
        if op == "route_bwd":
            c["balance"] = rng.random() < 0.3
    return c


def work(case):
    op, es = case["op"], SIZE[case["dtype"]]
    if op.startswith("qk"):
        t, d = case["tokens"], case["d"]
        live = t - int(t * case["pad"])
        x = (case["hq"] + case["hk"]) * d
        rows = min(live, 32768) if case["seqs"] == t else -(-live // case["seqs"])  # of the table
        small = 8 * t + 4 * rows * case["rot"] + 2 * d * es
        if op == "qk_fwd":
            return {"bytes": (live + t) * x * es + small, "flops": 7 * live * x}
        return {"bytes": (2 * live + t) * x * es + small + 8 * d, "flops": 15 * live * x}
    if op.startswith("top"):
        r, n, k = case["rows"], case["n"], case["k"]
        live = r - int(r * case["out"])
        if op == "top_fwd":
            return {"bytes": live * n * es + r * (8 + 16 + 12 * k), "flops": 7 * live * n}
        return {"bytes": (live + r) * n * es + r * (8 + 20 + 12 * k), "flops": 8 * live * n}
    t, e, k = case["tokens"], case["experts"], case["k"]
    extra = 4 * e * case["bias"]
    if op == "route_fwd":
        return {"bytes": t * (e * es + 12 * k) + extra, "flops": 6 * t * e}
    return {"bytes": t * (2 * e * es + 12 * k + 4 * e * case["balance"]), "flops": 8 * t * e}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"op": op}
    if op.startswith("qk"):
        t, hq, hk, d, rot = case["tokens"], case["hq"], case["hk"], case["d"], case["rot"]
        # the fused projection's output, of which q and k are slices
        qkv = (randn(t, hq + 2 * hk, d) * (0.5 + rand(hq + 2 * hk, 1))).to(dt)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["wq"], s["wk"] = (1.0 + 0.1 * randn(d)).to(dt), (1.0 + 0.1 * randn(d)).to(dt)
        most = 32768
        if case["seqs"] == t:  # one token each, anywhere
            pos = torch.randint(0, most, (t,), generator=g, device="cuda")
        else:  # sequences of equal share, one behind the other
            share = -(-t // case["seqs"])
            pos = torch.arange(t, device="cuda") % share
        pos[torch.randperm(t, generator=g, device="cuda")[: int(t * case["pad"])]] = -1
        s["pos"] = pos
        # angles of far positions in 64 bits; the table holds cosines, then sines
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ang = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * freq
        s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["eps"], s["near"] = 1e-6, case["pairs"] == "neighbours"
        if op == "qk_bwd":
            s["dq"], s["dk"] = randn(t, hq, d).to(dt), randn(t, hk, d).to(dt)
        return s
    if op.startswith("top"):
        r, n, k = case["rows"], case["n"], case["k"]
        t = torch.randint(0, n, (r,), generator=g, device="cuda")
        z = 2.5 * randn(r, n)
        z[torch.arange(r, device="cuda"), t] += 14.0 * rand(r)
        if case["masked"]:
            ruled = rand(n) < case["masked"]
            ruled[t] = False
            z[:, ruled] = NEG
        s["logits"], s["k"], s["tau"] = z.to(dt), k, 1.0
        del z
        t[torch.randperm(r, generator=g, device="cuda")[: int(r * case["out"])]] = -100
        s["targets"] = t
        if op == "top_bwd":
            f = _top(s)
            s["stats"], s["entropy"], s["ids"] = f["stats"], f["entropy"], f["top_ids"]
            scale = 1024.0 / r if dt is torch.float16 else 1.0 / r  # binary16 trains with a loss scale
            s["dlogp"], s["dentropy"], s["dtop"] = scale * randn(r), 0.1 * scale * randn(r), 0.3 * scale * randn(r, k)
        return s
    t, e = case["tokens"], case["experts"]
    s["logits"] = (1.5 * randn(t, e)).to(dt)
    s["bias"] = 0.05 * randn(e) if case["bias"] else None
    for name in ("k", "score", "groups", "top_groups", "group_top", "renorm"):
        s[name] = case[name]
    s["scale"] = 2.5 if case["renorm"] else 1.0
    if op == "route_bwd":
        s["ids"] = _route(s)["ids"]
        s["dweights"] = randn(t, case["k"])
        s["dscores"] = 0.01 * randn(t, e) if case["balance"] else None
    return s


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _turn(y, c, s, near):
    """The first 2 * c.shape[-1] entries of y turned by the angles of c and s."""
    h = c.shape[-1]
    rot = y[..., : 2 * h]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if near else (rot[..., :h], rot[..., h:])
    a, b = a * c - b * s, b * c + a * s
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if near else torch.cat([a, b], -1), y[..., 2 * h:]], -1)


def _angles(s):
    h = s["table"].shape[1] // 2
    live = (s["pos"] >= 0) & (s["pos"] < s["table"].shape[0])
    row = s["table"][s["pos"].clamp(0, s["table"].shape[0] - 1)]
    return row[:, None, :h], row[:, None, h:], live[:, None, None]


def _qk_one(x, w, s, c, sn, live):
    f = x.float()
    f = f / torch.sqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
    return torch.where(live, _turn(f, c, sn, s["near"]), 0.0).to(x.dtype)


def _qk_one_bwd(dy, x, w, s, c, sn, live):
    f = x.float()
    r = 1.0 / torch.sqrt(f.square().mean(-1, keepdim=True) + s["eps"])
    xhat = f * r
    g = torch.where(live, _turn(dy.float(), c, -sn, s["near"]), 0.0)
    u = g * w.float()
    dx = r * (u - xhat * (u * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xhat).sum((0, 1))


def _best(z, k):
    """Indices of the k largest of each row, the lowest index first among equals; where nothing is left, -1."""
    bits = (z.float() + 0.0).view(torch.int32)
    rank = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
    rank += torch.arange(z.shape[1] - 1, -1, -1, device="cuda")
    top = rank.topk(min(k, z.shape[1]), -1).values
    ids = z.shape[1] - 1 - (top & 0xFFFFFFFF)
    ids = torch.nn.functional.pad(ids, (0, k - ids.shape[1]))
    past = torch.arange(k, device="cuda") >= z.shape[1]
    return torch.where(past | (z.gather(-1, ids) == NEG), -1, ids)


def _top(s):
    z, t = s["logits"], s["targets"]
    live = (t >= 0) & (t < z.shape[1])
    x = z.float() * s["tau"]
    m = x.amax(-1, keepdim=True)
    logd = torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    x = x - m - logd  # log-probabilities
    entropy = -torch.where(x > NEG, torch.exp(x) * x, 0.0).sum(-1)
    ids = torch.where(live[:, None], _best(z, s["k"]), -1)
    top = torch.where(ids >= 0, x.gather(-1, ids.clamp(0)), NEG)
    out = {"logp": x.gather(-1, t.clamp(0, z.shape[1] - 1)[:, None])[:, 0], "entropy": entropy}
    out = {name: torch.where(live, v, 0.0) for name, v in out.items()}
    out["top_ids"], out["top_logp"] = ids, torch.where(live[:, None], top, 0.0)
    out["stats"] = torch.where(live[:, None], torch.cat([z.float().amax(-1, keepdim=True), logd], 1), 0.0)
    return out


def _top_bwd(s):
    z, t, tau = s["logits"], s["targets"], s["tau"]
    live = (t >= 0) & (t < z.shape[1])
    lp = (z.float() - s["stats"][:, :1]) * tau - s["stats"][:, 1:]
    p = torch.exp(lp)
    dtop = torch.where(s["ids"] >= 0, s["dtop"], 0.0)
    slope = (s["dlogp"] + dtop.sum(-1))[:, None] + s["dentropy"][:, None] * (torch.where(p > 0, lp, 0.0) + s["entropy"][:, None])
    d = -p * slope
    d.scatter_add_(-1, s["ids"].clamp(0), dtop)
    d.scatter_add_(-1, t.clamp(0, z.shape[1] - 1)[:, None], s["dlogp"][:, None])
    return torch.where(live[:, None], d * tau, 0.0).to(z.dtype)


def _scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _route(s):
    # the choice has borders: in 64 bits; the weights in 32
    x, k, g = s["logits"], s["k"], s["groups"]
    choice = _scores(x.double(), s["score"])
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    if s["top_groups"] < g:
        per = choice.unflatten(-1, (g, -1))
        worth = per.sort(dim=-1, descending=True).values[..., : s["group_top"]].sum(-1)
        kept = worth.sort(dim=-1, descending=True, stable=True).indices[:, : s["top_groups"]]
        keep = torch.zeros_like(worth, dtype=torch.bool).scatter_(-1, kept, True)
        choice = torch.where(keep[..., None], per, NEG).flatten(-2)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :k].contiguous()
    w = _scores(x.float(), s["score"]).gather(-1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"weights": w * s["scale"], "ids": ids}


def _route_bwd(s):
    x = s["logits"].float()
    sc = _scores(x, s["score"])
    w, d = sc.gather(-1, s["ids"]), s["dweights"] * s["scale"]
    if s["renorm"]:
        total = w.sum(-1, keepdim=True)
        d = (d - (d * w).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(x) if s["dscores"] is None else s["dscores"].clone()
    ds.scatter_add_(-1, s["ids"], d)
    dx = sc * (ds - (ds * sc).sum(-1, keepdim=True)) if s["score"] == "softmax" else ds * sc * (1.0 - sc)
    return dx.to(s["logits"].dtype)


def _plain(s):
    op = s["op"]
    if op == "qk_fwd":
        at = _angles(s)
        return {"q": _qk_one(s["q"], s["wq"], s, *at), "k": _qk_one(s["k"], s["wk"], s, *at)}
    if op == "qk_bwd":
        at = _angles(s)
        dq, dwq = _qk_one_bwd(s["dq"], s["q"], s["wq"], s, *at)
        dk, dwk = _qk_one_bwd(s["dk"], s["k"], s["wk"], s, *at)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    return {"top_fwd": _top, "top_bwd": _top_bwd, "route_fwd": _route, "route_bwd": _route_bwd}[op](s)


# ---------------------------------------------------------------------------
# The library's calls.
# ---------------------------------------------------------------------------
def _calls(s):
    import row_wise_normalization_reduce_gb300 as nrm
    op = s["op"]
    if op == "qk_fwd":
        q, k = nrm.qk_norm_rope_fwd(s["q"], s["k"], s["table"], s["pos"], s["wq"], s["wk"], s["eps"], interleaved=s["near"])
        return {"q": q, "k": k}
    if op == "qk_bwd":
        dq, dk, dwq, dwk = nrm.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["table"], s["pos"], s["wq"], s["wk"], s["eps"],
                                                interleaved=s["near"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if op == "top_fwd":
        logp, entropy, ids, top, stats = nrm.logprob_top_fwd(s["logits"], s["targets"], s["k"], s["tau"])
        return {"logp": logp, "entropy": entropy, "top_ids": ids, "top_logp": top, "stats": stats}
    if op == "top_bwd":
        return nrm.logprob_top_bwd(s["dlogp"], s["dentropy"], s["dtop"], s["logits"], s["targets"], s["stats"], s["entropy"], s["ids"],
                                   s["tau"])
    if op == "route_fwd":
        weights, ids, _ = nrm.route_fwd(s["logits"], s["k"], s["bias"], score=s["score"], groups=s["groups"], top_groups=s["top_groups"],
                                        group_top=s["group_top"], renormalize=s["renorm"], scale=s["scale"])
        return {"weights": weights, "ids": ids}
    return nrm.route_bwd(s["dweights"], s["logits"], s["ids"], score=s["score"], renormalize=s["renorm"], scale=s["scale"],
                         dscores=s["dscores"])


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _exact_qk(s, back):
    d, (most, rot) = s["q"].shape[-1], s["table"].shape
    i = torch.arange(d, device="cuda")
    # entry i turns with its partner by the angle of its pair: out_i = y_i cos + sign_i y_partner sin
    if s["near"]:
        partner, first, pair = i ^ 1, i % 2 == 0, i // 2
    else:
        partner, first, pair = torch.where(i < rot // 2, i + rot // 2, i - rot // 2), i < rot // 2, i % max(rot // 2, 1)
    still = i >= rot
    partner, pair = torch.where(still, i, partner), torch.where(still, 0, pair)
    ok = ((s["pos"] >= 0) & (s["pos"] < most)).double()[:, None]
    at = s["pos"].clamp(0, most - 1)
    tab = s["table"].double()[at]
    cos = torch.where(still, 1.0, tab[:, pair])[:, None]
    sin = torch.where(still, 0.0, tab[:, rot // 2 + pair])[:, None] * torch.where(first, -1.0, 1.0)
    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        norm = (x.pow(2).sum(-1, keepdim=True) / d + s["eps"]).rsqrt()
        if not back:
            y = x * norm * w
            out[name] = (y * cos + y[..., partner] * sin) * ok[..., None]
            continue
        dy = s["d" + name].double() * ok[..., None]
        g = dy * cos + (dy * sin)[..., partner]  # the transposed turn
        out["dw" + name] = torch.einsum("thd,thd->d", g, x * norm)
        u = g * w
        out["d" + name] = norm * u - norm.pow(3) / d * x * (u * x).sum(-1, keepdim=True)
    return {n: out[n] for n in (("dq", "dk", "dwq", "dwk") if back else ("q", "k"))}


def _exact_top(s, back):
    z, t, tau, k = s["logits"], s["targets"], s["tau"], s["k"]
    r, n = z.shape
    f64 = {"dtype": torch.float64, "device": "cuda"}
    if back:
        grad = torch.zeros(r, n, **f64)
    else:
        logp, ent, lp, stats = torch.zeros(r, **f64), torch.zeros(r, **f64), torch.zeros(r, k, **f64), torch.zeros(r, 2, **f64)
        ids = torch.full((r, k), -1, device="cuda")
    rows = torch.tensor([i for i, v in enumerate(t.tolist()) if 0 <= v < n], dtype=torch.long, device="cuda")
    for at in rows.split(max(1, 2 ** 26 // n)):  # some rows at a time: 64 bits of all logits are large
        x = z[at].double() * tau
        if back:
            l = (z[at].double() - s["stats"][at, :1].double()) * tau - s["stats"][at, 1:].double()
            p = l.exp()
            a = s["dtop"][at].double().masked_fill(s["ids"][at] < 0, 0.0)
            g, h = s["dlogp"][at].double()[:, None], s["dentropy"][at].double()[:, None]
            inner = (l + s["entropy"][at].double()[:, None]).masked_fill(p == 0, 0.0)
            d = -(g + a.sum(1, keepdim=True) + h * inner) * p
            d.scatter_add_(1, torch.cat([t[at, None], s["ids"][at].clamp(min=0)], 1), torch.cat([g, a], 1))
            grad[at] = d * tau
            continue
        lse = x.logsumexp(1, keepdim=True)
        l = x - lse
        logp[at] = l[torch.arange(len(at), device="cuda"), t[at]]
        ent[at] = -torch.special.xlogy(l.exp(), l.exp()).sum(1)
        stats[at, 0] = z[at].double().amax(1)
        stats[at, 1] = lse[:, 0] - x.amax(1)
        left = x.clone()
        i = torch.arange(n, device="cuda")
        for j in range(min(k, n)):
            top = left.amax(1, keepdim=True)
            first = torch.where(left == top, i, n).amin(1)
            none = top[:, 0] == NEG
            ids[at, j] = first.masked_fill(none, -1)
            lp[at, j] = l.gather(1, first[:, None])[:, 0].masked_fill(none, NEG)
            left.scatter_(1, first[:, None], NEG)
    return grad if back else {"logp": logp, "entropy": ent, "top_ids": ids, "top_logp": lp, "stats": stats}


def _exact_route(s, back):
    x = s["logits"].double()
    t, e = x.shape
    sc = (x - x.logsumexp(1, keepdim=True)).exp() if s["score"] == "softmax" else x.sigmoid()
    if not back:
        left = sc.clone() if s["bias"] is None else sc + s["bias"].double()
        size = e // s["groups"]
        worth = left.reshape(t, -1, size).topk(min(s["group_top"], size), 2).values.sum(2)
        place = torch.arange(s["groups"], device="cuda")
        # a group is in when fewer than top_groups are ahead of it
        ahead = (worth[:, None, :] > worth[:, :, None]) | ((worth[:, None, :] == worth[:, :, None]) & (place[None, :] < place[:, None]))
        left.masked_fill_((ahead.sum(2) >= s["top_groups"]).repeat_interleave(size, 1), NEG)
        ids = torch.empty(t, s["k"], dtype=torch.long, device="cuda")
        i = torch.arange(e, device="cuda")
        for j in range(s["k"]):
            ids[:, j] = torch.where(left == left.amax(1, keepdim=True), i, e).amin(1)
            left.scatter_(1, ids[:, j, None], NEG)
        w = sc.gather(1, ids)
        return {"weights": (w / w.sum(1, keepdim=True) if s["renorm"] else w) * s["scale"], "ids": ids}
    sc.requires_grad_()
    w = sc.gather(1, s["ids"])
    w = (w / w.sum(1, keepdim=True) if s["renorm"] else w) * s["scale"]
    loss = (w * s["dweights"].double()).sum()
    if s["dscores"] is not None:
        loss = loss + (sc * s["dscores"].double()).sum()
    ds, = torch.autograd.grad(loss, sc)
    p = sc.detach()
    return p * ds - p * (p * ds).sum(1, keepdim=True) if s["score"] == "softmax" else ds * p * (1 - p)


def exact(case, seed):
    s = prepare(case, seed)
    back = s["op"].endswith("bwd")
    return {"q": _exact_qk, "t": _exact_top, "r": _exact_route}[s["op"][0]](s, back)
