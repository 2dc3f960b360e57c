"""The training operators of the row library: dropout from a counter-based
generator (alone, and fused with the residual add and RMSNorm, forward and
backward), the log-probability of one target per row of logits with its
gradient, and the clipped policy loss with a KL term.

listed() and draw() give cases, prepare() their inputs, run() one call of an
operator: in plain torch operations, or (own) through the library's entry
points; exact() is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # dropout after a small projection: one launch, latency counts
        {"name": "dropout_fwd_f16_64x1024", "op": "dropout_fwd", "dtype": "f16", "rows": 64, "n": 1024, "p": 0.1},
        # gradient of the dropout on a long batch's activations
        {"name": "dropout_bwd_bf16_8192x8192", "op": "dropout_bwd", "dtype": "bf16", "rows": 8192, "n": 8192, "p": 0.1},
        # the residual stream of a short fine-tuning batch
        {"name": "drop_add_rms_fwd_f32_64x1024", "op": "drop_add_rms_fwd", "dtype": "f32", "rows": 64, "n": 1024, "p": 0.1},
        # the residual stream of an ordinary training batch
        {"name": "drop_add_rms_fwd_bf16_4096x4096", "op": "drop_add_rms_fwd", "dtype": "bf16", "rows": 4096, "n": 4096, "p": 0.1},
        # its backward, with the gradient that comes along the residual stream
        {"name": "drop_add_rms_bwd_bf16_4096x4096", "op": "drop_add_rms_bwd", "dtype": "bf16", "rows": 4096, "n": 4096, "p": 0.1, "up": True},
        # the last block of a ragged batch with an odd width: no gradient along the stream yet
        {"name": "drop_add_rms_bwd_f16_1999x5001", "op": "drop_add_rms_bwd", "dtype": "f16", "rows": 1999, "n": 5001, "p": 0.25, "up": False},
        # log-probabilities of a few generated tokens
        {"name": "logprob_fwd_bf16_16x32768", "op": "logprob_fwd", "dtype": "bf16", "rows": 16, "n": 32768, "masked": 0.0},
        # log-probabilities of a batch under the reference policy, a large vocabulary
        {"name": "logprob_fwd_bf16_4096x131072", "op": "logprob_fwd", "dtype": "bf16", "rows": 4096, "n": 131072, "masked": 0.25},
        # gradient of a loss on log-probabilities in binary32, an odd vocabulary
        {"name": "logprob_bwd_f32_513x50001", "op": "logprob_bwd", "dtype": "f32", "rows": 513, "n": 50001, "masked": 0.1},
        # the same for a training batch
        {"name": "logprob_bwd_bf16_2048x131072", "op": "logprob_bwd", "dtype": "bf16", "rows": 2048, "n": 131072, "masked": 0.25},
        # a policy step on a small batch with an odd vocabulary
        {"name": "policy_loss_f16_333x50001", "op": "policy_loss", "dtype": "f16", "rows": 333, "n": 50001, "masked": 0.2, "kl": 0.05},
        # a policy step on a training batch: prompts and padding take no part
        {"name": "policy_loss_bf16_4096x131072", "op": "policy_loss", "dtype": "bf16", "rows": 4096, "n": 131072, "masked": 0.3, "kl": 0.02},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; half of them multiples of 64 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["dropout_fwd", "dropout_bwd", "drop_add_rms_fwd", "drop_add_rms_bwd", "logprob_fwd", "logprob_bwd", "policy_loss"])
    c = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if op.startswith("drop"):
        c["n"] = _size(rng, 64, 16384)
        c["rows"] = _size(rng, 1, min(16384, 2 ** 25 // c["n"]))
        c["p"] = round(rng.uniform(0.01, 0.6), 3)
        if op == "drop_add_rms_bwd":
            c["up"] = rng.random() < 0.7
    else:
        c["n"] = _size(rng, 1000, 160000)
        c["rows"] = _size(rng, 1, min(8192, 2 ** 27 // c["n"]))
        c["masked"] = round(rng.uniform(0.0, 0.5), 2)
        if op == "policy_loss":
            c["kl"] = round(rng.uniform(0.0, 0.1), 3) if rng.random() < 0.7 else 0.0
    return c


def _live(case):
    return case["rows"] - int(case["rows"] * case.get("masked", 0.0))


def work(case):
    r, n, es, op = case["rows"], case["n"], SIZE[case["dtype"]], case["op"]
    if op in ("dropout_fwd", "dropout_bwd"):
        return {"bytes": 2 * r * n * es, "flops": r * n}
    if op == "drop_add_rms_fwd":
        return {"bytes": 4 * r * n * es + n * es + 4 * r, "flops": 6 * r * n}
    if op == "drop_add_rms_bwd":
        return {"bytes": (5 if case["up"] else 4) * r * n * es + n * es + 4 * r + 4 * n, "flops": 12 * r * n}
    live = _live(case)
    if op == "logprob_fwd":
        return {"bytes": live * n * es + 16 * r, "flops": 4 * live * n}
    if op == "logprob_bwd":
        return {"bytes": (live + r) * n * es + 16 * r, "flops": 5 * live * n}
    return {"bytes": (live + r) * n * es + 28 * r, "flops": 8 * live * n}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, r, n, op = DTYPES[case["dtype"]], case["rows"], case["n"], case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"op": op, "case": dict(case)}
    if op.startswith("drop"):
        # the generator's key and the call's place in the step, as a training loop numbers them
        s["p"], s["seed"], s["offset"] = case["p"], 0x9E3779B9 * (seed + 1) % 2 ** 63, 7 + seed % 1000
        if op in ("dropout_fwd", "dropout_bwd"):
            s["x"] = randn(r, n).to(dt)
            return s
        s["w"] = (1.0 + 0.05 * randn(n)).to(dt)
        s["eps"] = 1e-6
        if op == "drop_add_rms_fwd":
            s["x"], s["residual"] = randn(r, n).to(dt), (2.0 * randn(r, n)).to(dt)
            return s
        s["h"] = (2.0 * randn(r, n)).to(dt)
        s["rstd"] = 1.0 / torch.sqrt(s["h"].float().square().mean(-1) + s["eps"])
        s["dy"] = randn(r, n).to(dt)
        s["up"] = randn(r, n).to(dt) if case["up"] else None
        return s
    # logits with one likely token per row, the row's target
    t = torch.randint(0, n, (r,), generator=g, device="cuda")
    z = 2.5 * randn(r, n)
    z[torch.arange(r, device="cuda"), t] += 14.0 * torch.rand(r, generator=g, device="cuda")
    s["logits"] = z.to(dt)
    del z
    s["inv_temp"] = 1.0
    out = torch.randperm(r, generator=g, device="cuda")[: r - _live(case)]
    if op == "logprob_fwd":
        t[out] = -100
        s["targets"] = t
        return s
    logp, lse = _logprob(s["logits"], t, 1.0)
    if op == "logprob_bwd":
        t[out] = -100
        s["targets"], s["lse"], s["dlogp"] = t, lse, randn(r) / r
        s["lse"][out] = 0.0
        return s
    # the sampling policy and the reference policy are some steps away; prompt rows have weight 0, padded rows no target
    s["old"] = (logp + 0.15 * randn(r)).float()
    s["ref"] = (logp + 0.3 * randn(r)).float() if case["kl"] else None
    s["adv"] = randn(r)
    s["weights"] = torch.full((r,), 1.0 / max(1, _live(case)), device="cuda")
    s["weights"][out] = 0.0
    t[out[::2]] = -100
    s["targets"], s["kl"], s["clip"] = t, case["kl"], (0.2, 0.28)
    return s


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _philox(rows, n, seed, offset):
    """[rows, n] 16-bit random numbers: Philox4x32-10 of counter (col // 8, row, offset), key seed, eight numbers a block."""
    m = 0xFFFFFFFF
    a = torch.arange((n + 7) // 8, device="cuda").expand(rows, -1)
    b = torch.arange(rows, device="cuda")[:, None].expand_as(a)
    c, d = torch.full_like(a, offset & m), torch.full_like(a, offset >> 32)
    k0, k1 = seed & m, seed >> 32
    for _ in range(10):
        # the low 64 bits of the products: what >> carries in from the sign is masked away
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32 & m) ^ b ^ k0, q & m, (p >> 32 & m) ^ d ^ k1, p & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    u = torch.stack([a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16, c & 0xFFFF, c >> 16, d & 0xFFFF, d >> 16], -1)
    return u.reshape(rows, -1)[:, :n]


def _dropped(v, s):
    t = int(math.floor(s["p"] * 65536 + 0.5))
    keep = _philox(v.shape[0], v.shape[1], s["seed"], s["offset"]) >= t
    return torch.where(keep, v * (65536.0 / (65536 - t)), torch.zeros((), device="cuda"))


def _logprob(z, t, inv_temp):
    """log-softmax of each row's target and the row's log-sum-exp; the sum and what follows in 64 bits (the loss has a border)."""
    z = z.float() * inv_temp
    top = z.amax(-1, keepdim=True)
    lse = top[:, 0].double() + torch.log(torch.sum(torch.exp(z - top), -1, dtype=torch.float64))
    at = z.gather(-1, t.clamp(0, z.shape[1] - 1)[:, None])[:, 0].double()
    return at - lse, lse.float()


def _dlogits(z, t, lse, coef, inv_temp, dt):
    """coef * inv_temp * (onehot - softmax), rows without a coefficient 0."""
    g = (coef * inv_temp)[:, None]
    live = (g != 0)
    d = torch.where(live, -g * torch.exp(z.float() * inv_temp - lse[:, None]), torch.zeros((), device="cuda"))
    d.scatter_add_(-1, t.clamp(0, z.shape[1] - 1)[:, None], torch.where(live, g, torch.zeros((), device="cuda")))
    return d.to(dt)


def _plain(s):
    op = s["op"]
    if op in ("dropout_fwd", "dropout_bwd"):
        return _dropped(s["x"].float(), s).to(s["x"].dtype)
    if op == "drop_add_rms_fwd":
        h = (s["residual"].float() + _dropped(s["x"].float(), s)).to(s["x"].dtype)
        f = h.float()
        rstd = 1.0 / torch.sqrt(f.square().mean(-1) + s["eps"])
        return {"residual_out": h, "y": (f * rstd[:, None] * s["w"].float()).to(h.dtype), "rstd": rstd}
    if op == "drop_add_rms_bwd":
        dy, xhat = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        g = dy * s["w"].float()
        dh = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        if s["up"] is not None:
            dh = dh + s["up"].float()
        return {"dx": _dropped(dh, s).to(s["dy"].dtype), "dresidual": dh.to(s["dy"].dtype), "dw": (dy * xhat).sum(0)}
    z, t = s["logits"], s["targets"]
    valid = (t >= 0) & (t < z.shape[1])
    if op == "logprob_fwd":
        logp, lse = _logprob(z, t, s["inv_temp"])
        return {"logp": torch.where(valid, logp, 0.0).float(), "lse": torch.where(valid, lse, 0.0)}
    if op == "logprob_bwd":
        return _dlogits(z, t, s["lse"], torch.where(valid, s["dlogp"], 0.0), s["inv_temp"], z.dtype)
    logp, lse = _logprob(z, t, s["inv_temp"])
    live = valid & (s["weights"] != 0)
    adv, w, old = s["adv"].double(), s["weights"].double(), s["old"].double()
    ratio = torch.exp(logp - old)
    free, held = -adv * ratio, -adv * ratio.clamp(1 - s["clip"][0], 1 + s["clip"][1])
    loss, slope = torch.maximum(free, held), torch.where(free >= held, free, 0.0)
    if s["ref"] is not None:
        away = s["ref"].double() - logp
        loss = loss + s["kl"] * (torch.exp(away) - away - 1)
        slope = slope + s["kl"] * (1 - torch.exp(away))
    coef = torch.where(live, w * slope, 0.0).float()
    return {"loss": torch.where(live, w * loss, 0.0).sum().float(), "logp": torch.where(live, logp, 0.0).float(),
            "dlogits": _dlogits(z, t, lse, coef, s["inv_temp"], z.dtype)}


# ---------------------------------------------------------------------------
# The library's calls.
# ---------------------------------------------------------------------------
def _calls(s):
    import row_wise_normalization_reduce_gb300 as nrm
    op = s["op"]
    if op == "dropout_fwd":
        return nrm.dropout_fwd(s["x"], s["p"], s["seed"], s["offset"])
    if op == "dropout_bwd":
        return nrm.dropout_bwd(s["x"], s["p"], s["seed"], s["offset"])
    if op == "drop_add_rms_fwd":
        h, y, rstd = nrm.dropout_add_rms_fwd(s["x"], s["residual"], s["w"], s["p"], s["seed"], s["offset"], s["eps"])
        return {"residual_out": h, "y": y, "rstd": rstd}
    if op == "drop_add_rms_bwd":
        dx, dres, dw = nrm.dropout_add_rms_bwd(s["dy"], s["h"], s["rstd"], s["w"], s["p"], s["seed"], s["offset"], dresidual_out=s["up"])
        return {"dx": dx, "dresidual": dres, "dw": dw}
    if op == "logprob_fwd":
        logp, lse = nrm.logprob_fwd(s["logits"], s["targets"], s["inv_temp"])
        return {"logp": logp, "lse": lse}
    if op == "logprob_bwd":
        return nrm.logprob_bwd(s["dlogp"], s["logits"], s["targets"], s["lse"], s["inv_temp"])
    loss, logp, dlogits = nrm.policy_loss(s["logits"], s["targets"], s["old"], s["adv"], s["weights"], s["ref"], s["clip"][0],
                                          s["clip"][1], s["kl"], s["inv_temp"])
    return {"loss": loss, "logp": logp, "dlogits": dlogits}


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _kept(rows, n, p, seed, offset):
    """The mask from the generator's definition, in unsigned 64-bit host integers, and the scale of what is kept."""
    lo = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    nb = -(-n // 8)
    x = [np.tile(np.arange(nb, dtype=np.uint64), rows), np.repeat(np.arange(rows, dtype=np.uint64), nb)]
    x += [np.full(rows * nb, offset % 2 ** 32, np.uint64), np.full(rows * nb, offset // 2 ** 32, np.uint64)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for i in range(10):
        k = [np.uint64((key[0] + i * 0x9E3779B9) % 2 ** 32), np.uint64((key[1] + i * 0xBB67AE85) % 2 ** 32)]
        m0, m1 = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        x = [(m1 >> sh) ^ x[1] ^ k[0], m1 & lo, (m0 >> sh) ^ x[3] ^ k[1], m0 & lo]
    words = np.stack([v.astype("<u4") for v in x], -1)
    u = words.view("<u2").reshape(rows, nb * 8)[:, :n]
    bar = int(math.floor(p * 65536 + 0.5))
    return torch.from_numpy((u >= bar)).cuda(), 65536.0 / (65536 - bar)


def exact(case, seed):
    s = prepare(case, seed)
    r, n, op = case["rows"], case["n"], case["op"]
    if op.startswith("drop"):
        keep, scale = _kept(r, n, s["p"], s["seed"], s["offset"])
        if op in ("dropout_fwd", "dropout_bwd"):
            return (s["x"].double() * scale).masked_fill(~keep, 0.0)
        w = s["w"].double()
        if op == "drop_add_rms_fwd":
            # the norm is of the rounded stream: its value in the stream's type is part of the definition
            h = (s["x"].double() * scale).masked_fill(~keep, 0.0) + s["residual"].double()
            f = h.to(s["x"].dtype).double()
            rstd = (f.pow(2).sum(-1) / n + s["eps"]).rsqrt()
            return {"residual_out": h, "y": f * rstd[:, None] * w, "rstd": rstd}
        h, dy, k = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        g = dy * w
        dot = (g * h).sum(-1, keepdim=True)
        dh = k * g - k.pow(3) * h * dot / n
        if s["up"] is not None:
            dh += s["up"].double()
        return {"dx": (dh * scale).masked_fill(~keep, 0.0), "dresidual": dh, "dw": torch.einsum("ij,ij->j", dy, h * k)}
    logits, t, tau = s["logits"], s["targets"], s["inv_temp"]
    ok = [0 <= v < n for v in t.tolist()]
    logp, lse = torch.zeros(r, dtype=torch.float64, device="cuda"), torch.zeros(r, dtype=torch.float64, device="cuda")
    grad = None if op == "logprob_fwd" else torch.zeros(r, n, dtype=torch.float64, device="cuda")
    slope = torch.zeros(r, dtype=torch.float64, device="cuda")
    total = 0.0
    step = max(1, 2 ** 26 // n)
    for a in range(0, r, step):  # some rows at a time: 64 bits of all logits are large
        rows = [i for i in range(a, min(r, a + step)) if ok[i] and (op != "policy_loss" or float(s["weights"][i]) != 0.0)]
        if not rows:
            continue
        at = torch.tensor(rows, device="cuda")
        z = logits[at].double() * tau
        lse[at] = torch.logsumexp(z, -1)
        picked = z[torch.arange(len(rows), device="cuda"), t[at]]
        logp[at] = picked - lse[at]
        if op == "logprob_fwd":
            continue
        if op == "logprob_bwd":
            norm, g = s["lse"][at].double(), s["dlogp"][at].double()
        else:
            norm, lp = lse[at], logp[at]
            adv, wt, rho = s["adv"][at].double(), s["weights"][at].double(), (logp[at] - s["old"][at].double()).exp()
            low, high = 1 - s["clip"][0], 1 + s["clip"][1]
            # a positive advantage gains nothing above the upper bound, a negative one nothing below the lower
            inside = torch.where(adv > 0, rho <= high, rho >= low)
            term = -adv * torch.where(inside, rho, torch.where(adv > 0, high, low))
            g = torch.where(inside, -adv * rho, 0.0)
            if s["ref"] is not None:
                q = s["ref"][at].double() - lp
                term = term + s["kl"] * (torch.expm1(q) - q)
                g = g - s["kl"] * torch.expm1(q)
            g = wt * g
            total += float((wt * term).sum())
        soft = (z - norm[:, None]).exp_()
        soft[torch.arange(len(rows), device="cuda"), t[at]] -= 1.0
        grad[at] = soft.mul_(-(g * tau)[:, None])
    if op == "logprob_fwd":
        return {"logp": logp, "lse": lse}
    if op == "logprob_bwd":
        return grad
    return {"loss": torch.tensor(total, dtype=torch.float64), "logp": logp, "dlogits": grad}
