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
