"""Plain 64-bit definitions of the operators inside a block and at a model's
end (head norms with the position rotation; log-probability with entropy and
top alternatives; routing to experts), and the bounds their tests use.

u = 2^-24 is the binary32 unit roundoff; an output in type t adds eps(t) / 2
relative (or half its smallest subnormal).

Head norms.  A row's sum of squares is at most 16 fused additions in a lane and
5 levels of the tree deep, halved by the root, + 2 ulp (4 u) of rsqrtf + 2 for
the mean and eps: r is good to 20 u, y = x r w to 22 u, and each of the two
products and the sum of a turn adds 1: 26 u (|y_a c| + |y_b s|).  Backward: a
turned gradient is good to 3 u of G = |da c| + |db s|; the row sum of u x to 27
u of sum G |w x|; with r^2 (40 u), three products and the last ones that makes
less than 128 u = 2^-17 of r (G |w| + |x| r^2 mean(G |w x|)).  dw adds at most 200
terms in a chain, each good to 25 u: 2^-16 of the sum of |terms|.
"""
import torch

U = 2.0 ** -24
EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def out_bound(dtype, ref, extra):
    """|got - ref| allowed for an output rounded to dtype whose unrounded value is within extra of ref."""
    return (ref.abs() + extra) * (EPS[dtype] / 2) + extra + TINY[dtype] / 2


def check(got, ref, bound, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    got, bound = got.double(), torch.as_tensor(bound, dtype=torch.float64, device=ref.device).expand(ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        at = bad.nonzero()[:3].tolist()
        raise AssertionError((what, int(bad.sum()), at, got[bad][:3].tolist(), ref[bad][:3].tolist(), bound[bad][:3].tolist()))


# --- head norms with the position rotation ----------------------------------
def angle_table(positions, rot, base=10000.0, device="cpu"):
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(y, table, pos, interleaved, back=False, magnitudes=False):
    """The rows y [tokens, heads, D] turned (back: by the negative angle); with
    magnitudes the sums of the products' absolute values."""
    rot = table.shape[1]
    a, b = (i.to(y.device) for i in pairs(rot, interleaved))
    t = table.double()[pos.clamp(0, max(table.shape[0] - 1, 0))][:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:] * (-1 if back else 1)
    out = y.clone()
    if magnitudes:
        y, c, s, out = y.abs(), c.abs(), s.abs(), out.abs()
        out[..., a], out[..., b] = y[..., a] * c + y[..., b] * s, y[..., b] * c + y[..., a] * s
    else:
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    return out


def live_tokens(table, pos):
    return (pos >= 0) & (pos < table.shape[0])


def head_norm(x, w, table, pos, eps, interleaved):
    """out [tokens, heads, D] in 64 bits, and the bound of its binary32 evaluation."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    live = live_tokens(table, pos)
    x = torch.where(live[:, None, None], x, 0.0)
    y = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w
    out = torch.where(live[:, None, None], turn(y, table, pos, interleaved), 0.0)
    return out, torch.where(live[:, None, None], 26 * U * turn(y, table, pos, interleaved, magnitudes=True), 0.0)


def head_norm_bwd(dout, x, w, table, pos, eps, interleaved):
    """dx, its bound, dw, its bound."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    live = live_tokens(table, pos)[:, None, None]
    d, x = torch.where(live, dout.double(), 0.0), torch.where(live, x, 0.0)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    g, big = turn(d, table, pos, interleaved, back=True), turn(d, table, pos, interleaved, back=True, magnitudes=True)
    u, mag = g * w, big * w.abs()
    dx = r * u - x * r ** 3 * (u * x).mean(-1, keepdim=True)
    slack = 2.0 ** -17 * r * (mag + x.abs() * r ** 2 * (mag * x.abs()).mean(-1, keepdim=True))
    dw = (g * x * r).sum((0, 1))
    return torch.where(live, dx, 0.0), torch.where(live, slack, 0.0), dw, 2.0 ** -16 * (big * x.abs() * r).sum((0, 1)) + 2.0 ** -149


# --- routing to experts -------------------------------------------------------
# Scores: expf and the division are good to 5 u of a sigmoid; a softmax adds the
# sum, at most 38 additions deep, of exponentials good to 4 u + 2 u |x - m|, and
# the rounding of x - m in its own: 128 u = 2^-17 while the weighed |x - m| stays
# below 32.  Underflow: 2^-126.
SCORE = 2.0 ** -17


def scores64(x, score):
    x = x.double()
    if score == "sigmoid":
        return torch.sigmoid(x)
    m = x.amax(-1, keepdim=True)
    e = torch.where(x == -float("inf"), 0.0, torch.exp(x - torch.where(m == -float("inf"), 0.0, m)))
    d = e.sum(-1, keepdim=True)
    return torch.where(d == 0, 0.0, e / d)


def route(x, k, bias=None, score="softmax", groups=1, top_groups=None, group_top=1, renormalize=True, scale=1.0):
    """weights (64 bits), ids: by the definition, a token at a time."""
    top_groups = groups if top_groups is None else top_groups
    s = scores64(x, score).cpu()
    c = s if bias is None else s + bias.double().cpu()
    if bias is None and (top_groups == groups or group_top == 1):
        c = x.double().cpu()  # the same order, and no two scores rounded to one
    c = torch.where((x.cpu() == -float("inf")) | torch.isnan(c), -float("inf"), c)
    tokens, experts = x.shape
    weights, ids = torch.zeros(tokens, k, dtype=torch.float64), torch.full((tokens, k), -1)
    size = experts // groups
    # stable: among equal ones the lowest index first
    order = c.sort(dim=-1, descending=True, stable=True)
    if top_groups < groups:
        top = c.view(tokens, groups, size).sort(dim=-1, descending=True).values[..., :group_top]
        worth = torch.where(top == -float("inf"), 0.0, top).sum(-1)
        worth = torch.where(top[..., 0] == -float("inf"), -float("inf"), worth)
        kept = worth.sort(dim=-1, descending=True, stable=True).indices[:, :top_groups]
        keep = torch.zeros(tokens, groups, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(size, 1)
        order = torch.where(keep, c, -float("inf")).sort(dim=-1, descending=True, stable=True)
    have = order.values[:, :k] > -float("inf")
    ids[have] = order.indices[:, :k][have]
    weights[have] = s.gather(1, order.indices[:, :k])[have]
    if renormalize and score == "softmax":  # exp(x_i) / sum exp(x_j) over the chosen: in this form nothing underflows
        z = torch.where(have, x.double().cpu().gather(1, order.indices[:, :k]), -float("inf"))
        weights = torch.where(have, torch.softmax(z, -1), 0.0)
    elif renormalize:
        total = weights.sum(-1, keepdim=True)
        weights = torch.where(total == 0, 0.0, weights / total)
    return weights * scale, ids


def route_grad(dweights, x, ids, score="softmax", renormalize=True, scale=1.0, dscores=None):
    """dx in 64 bits and the bound of its binary32 evaluation."""
    x, ids = x.double(), ids.clone()
    s = scores64(x, score)
    ok = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(ok, ids, 0)
    w = torch.where(ok, s.gather(1, at), 0.0)
    d = torch.where(ok, dweights.double() * scale, 0.0)
    mag = d.abs()
    if renormalize:
        total = w.sum(-1, keepdim=True)
        inv = torch.where(total == 0, 0.0, 1 / total)
        d, mag = (d - (d * w).sum(-1, keepdim=True) * inv) * inv, (mag + (mag * w).sum(-1, keepdim=True) * inv) * inv
    ds = torch.zeros_like(x) if dscores is None else dscores.double().clone()
    big = ds.abs()
    ds.scatter_add_(1, at, torch.where(ok, d, 0.0))
    big.scatter_add_(1, at, torch.where(ok, mag, 0.0))
    if score == "softmax":
        return s * (ds - (ds * s).sum(-1, keepdim=True)), 8 * SCORE * s * (big + (big * s).sum(-1, keepdim=True)) + 2.0 ** -126
    slope = s * torch.sigmoid(-x)
    return ds * slope, 8 * SCORE * big * slope + 2.0 ** -126


# --- rows of logits with entropy and alternatives ------------------------------
# log d: V / 512 additions in a thread and 20 merges of 5 u, exponentials good to
# 4 u and 3 roundings of their argument, which weigh |x| each (as train_ref.py).  The
# entropy adds sum p |x| times that, and sum p x^2 for the argument's roundings.
def logprob_top(z, t, k, s=1.0):
    """dict of logp, entropy, ids, top, stats in 64 bits, and of their bounds."""
    z, v = z.double(), z.shape[1]
    inf = float("inf")
    live = (t >= 0) & (t < v)
    x = z * s
    m = x.amax(-1, keepdim=True)
    none = m == -inf
    x = x - torch.where(none, 0.0, m)
    e = x.exp()
    d = e.sum(-1, keepdim=True)
    p = torch.where(none, 0.0, e / d)
    logd = torch.where(none, -inf, d.log())
    lp = torch.where(none, -inf, x - logd)
    fin = torch.where(p > 0, x, 0.0)
    b, c = (p * fin.abs()).sum(-1), (p * fin * fin).sum(-1)
    logd_slack = (v / 512 + 104 + 3 * b) * U
    out = {"logp": lp.gather(1, t.clamp(0, v - 1)[:, None])[:, 0], "entropy": -torch.where(p > 0, p * lp, 0.0).sum(-1)}
    bound = {"logp": logd_slack + U * torch.where(out["logp"] > -inf, out["logp"].abs(), 0.0),
             "entropy": logd_slack * (1 + 2 * b) + U * (8 * b + 3 * c + 4)}
    order = torch.where(torch.isnan(z), -inf, z).sort(dim=-1, descending=True, stable=True)
    ids = torch.full((len(z), k), -1, device=z.device)
    n = min(k, v)
    ids[:, :n] = torch.where(order.values[:, :n] > -inf, order.indices[:, :n], -1)
    out["ids"] = ids
    out["top"] = torch.where(ids >= 0, lp.gather(1, ids.clamp(0)), -inf)
    bound["top"] = logd_slack[:, None] + U * torch.where(ids >= 0, out["top"], 0.0).abs()
    out["stats"] = torch.cat([z.amax(-1, keepdim=True), logd], 1)
    bound["stats"] = torch.stack([0 * b, logd_slack + U * torch.where(none, 0.0, logd)[:, 0].abs()], 1)
    for name in ("logp", "entropy", "stats", "top"):
        dead = ~live if out[name].dim() == 1 else ~live[:, None]
        out[name] = torch.where(dead, 0.0, out[name])
    out["ids"] = torch.where(live[:, None], ids, -1)
    out["entropy"] = torch.where(none[:, 0], 0.0, out["entropy"])
    return out, bound


def logprob_top_grad(z, t, stats, entropy, ids, g, h, a, s=1.0):
    """dlogits in 64 bits for the given statistics, and the bound of their binary32 evaluation."""
    z, v = z.double(), z.shape[1]
    live = ((t >= 0) & (t < v) & (stats[:, 1] > -float("inf")))[:, None]
    lp = (z - torch.where(live, stats[:, :1].double(), 0.0)) * s - torch.where(live, stats[:, 1:].double(), 0.0)
    p = lp.exp()
    lp = torch.where(p > 0, lp, 0.0)
    zero = torch.zeros(len(z), 1, dtype=torch.float64, device=z.device)
    g = zero if g is None else g.double()[:, None]
    h, H = (zero, zero) if h is None else (h.double()[:, None], entropy.double()[:, None])
    if a is None:
        a, ids = zero[:, :0], torch.zeros(len(z), 0, dtype=torch.int64, device=z.device)
    ok = (ids >= 0) & (ids < v)
    a = torch.where(ok, a.double(), 0.0)
    dz = -p * (g + a.sum(1, keepdim=True) + h * (lp + H))
    mag = g.abs() + a.abs().sum(1, keepdim=True) + h.abs() * (lp.abs() + H.abs())
    slack = p * mag * U * (48 + 4 * (lp.abs() + stats[:, 1:].double().abs().clamp_max(1e30)))
    at = torch.cat([t.clamp(0, v - 1)[:, None], torch.where(ok, ids, 0)], 1)
    dz.scatter_add_(1, at, torch.cat([g, a], 1))
    slack.scatter_add_(1, at, 40 * U * torch.cat([g, a], 1).abs())
    return torch.where(live, dz * s, 0.0), torch.where(live, slack * s, 0.0) + 2.0 ** -126
