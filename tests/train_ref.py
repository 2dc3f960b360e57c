"""Plain 64-bit definitions of the training operators (numpy), and the bounds
their tests use.

Roundings: u = 2^-24 is the binary32 unit roundoff; an output in type t adds
eps(t) / 2 relative (or half its smallest subnormal).  The other terms count
the binary32 operations between input and output:

* dropout: the scale's own rounding and one product: 2 u.
* residual_out: the same binary32 operations in numpy, so equal bits.
* rstd: a sum of positive terms, at most 64 additions deep (16 in a thread and
  10 levels of the tree in the register plan, N / 4096 + 16 in the long-row
  plan), halved by the root, + 2 ulp (4 u) of rsqrtf + 2 for the mean and eps:
  40 u.  y adds two products: 44 u < 2^-18.
* dh = rstd g + k h + up: 4 roundings of rstd g; k carries the row sum's error,
  at most 64 u of sum |g h|, and 5 products (a bound of 2^-17 of the same sum
  with absolute values); the additions 3 u of their operands.
* dw: at most 128 additions deep: 2^-16 sum |dy xhat|.
* d of a row of logits: V / 512 additions in a thread and 20 merges (an
  addition, a product and an exponential each: 5 u); each exponential 4 u and
  its argument 3 roundings, which weigh |x| u each.
"""
import numpy as np
import torch

U = 2.0 ** -24
EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
M32 = np.uint64(0xFFFFFFFF)


def philox(ctr, key):
    """Philox4x32-10 of counters [..., 4] and one key (two words): [..., 4] words."""
    c = [np.asarray(ctr[..., i], np.uint64) for i in range(4)]
    for r in range(10):
        k0 = np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ k0, b & M32, (a >> np.uint64(32)) ^ c[3] ^ k1, a & M32]
    return np.stack(c, -1)


def bar_scale(p):
    t = int(np.floor(p * 65536 + 0.5))
    return t, (65536.0 / (65536 - t) if t < 65536 else 0.0)


def keep(rows, n, p, seed, offset=0):
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    nb = -(-n // 8)
    ctr = np.zeros((rows, nb, 4), np.uint64)
    ctr[..., 0] = np.arange(nb)
    ctr[..., 1] = np.arange(rows)[:, None]
    ctr[..., 2] = offset & 0xFFFFFFFF
    ctr[..., 3] = offset >> 32
    w = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(rows, nb * 8)[:, :n]
    return u >= np.uint64(bar_scale(p)[0])


def f64(t):
    return t.detach().cpu().double().numpy()


def out_bound(dtype, ref, extra):
    """|got - ref| allowed for an output rounded to dtype whose unrounded value is within extra of ref."""
    return (np.abs(ref) + extra) * (EPS[dtype] / 2) + extra + TINY[dtype] / 2


def check(got, ref, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], ref[bad][:3],
                           np.broadcast_to(bound, ref.shape)[bad][:3])


# --- dropout and the residual path -----------------------------------------
def drop(v, mask, p):
    return np.where(mask, v * bar_scale(p)[1], 0.0)


def stream(x, residual, mask, p):
    """residual_out in the tensors' type, by the binary32 operations that define it (torch, on the CPU)."""
    s = torch.tensor(bar_scale(p)[1], dtype=torch.float32)
    d = torch.where(torch.from_numpy(mask), x.cpu().float() * s, torch.zeros(()))
    return (residual.cpu().float() + d).to(x.dtype)


def norm(h, w, eps):
    rstd = 1.0 / np.sqrt(np.mean(h * h, -1) + eps)
    return h * rstd[:, None] * w, rstd


def add_rms_bwd(dy, h, rstd, w, up):
    """dh, dw and the bounds of their binary32 evaluation."""
    n = h.shape[1]
    r = rstd[:, None]
    g = dy * w
    xhat = h * r
    dh = r * (g - xhat * np.mean(g * xhat, -1, keepdims=True)) + up
    slack = 4 * U * np.abs(r * g) + 2.0 ** -17 * np.abs(h) * r ** 3 * np.mean(np.abs(g * h), -1, keepdims=True)
    slack = slack + 3 * U * np.abs(up)
    return dh, slack, np.sum(dy * xhat, 0), 2.0 ** -16 * np.sum(np.abs(dy * xhat), 0) + 2.0 ** -149


# --- rows of logits ---------------------------------------------------------
def logprob(z, t, s):
    """logp, lse per row, and the bound of the error of log d (rows without a target: 0)."""
    rows, v = z.shape
    logp, lse, slack = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    for r in range(rows):
        if not 0 <= t[r] < v:
            continue
        x = s * z[r]
        m = x.max()
        if m == -np.inf:
            logp[r] = lse[r] = -np.inf
            continue
        with np.errstate(invalid="ignore"):
            e = np.exp(x - m)
        lse[r] = m + np.log(e.sum())
        logp[r] = x[t[r]] - lse[r]
        with np.errstate(invalid="ignore"):
            arg = np.where(e > 0, np.abs(x - m) * e, 0.0).sum() / e.sum()
        slack[r] = (v / 512 + 104 + 3 * arg) * U
    return logp, lse, slack


def grad(z, t, lse, g, s):
    """dlogits for the slopes g and the given lse, and per element |x - lse|."""
    out, arg = np.zeros_like(z), np.zeros_like(z)
    for r in range(z.shape[0]):
        if not 0 <= t[r] < z.shape[1] or g[r] == 0 or lse[r] == -np.inf:
            continue
        d = s * z[r] - lse[r]
        p = np.exp(d)
        out[r] = -g[r] * s * p
        out[r, t[r]] += g[r] * s
        arg[r] = np.where(p > 0, np.abs(d), 0.0)
    return out, arg


def policy(z, t, old, adv, weight, ref, lo, hi, beta, s):
    """loss, logp, slope of the loss in each logp."""
    logp, lse, slack = logprob(z, t, s)
    live = np.array([0 <= t[r] < z.shape[1] and weight[r] != 0 for r in range(len(t))])
    total, slope, room = 0.0, np.zeros(len(t)), 0.0
    for r in np.flatnonzero(live):
        if lse[r] == -np.inf:
            continue
        ratio = np.exp(logp[r] - old[r])
        free, held = -adv[r] * ratio, -adv[r] * np.clip(ratio, 1 - lo, 1 + hi)
        term, g = max(free, held), free if free >= held else 0.0
        if beta:
            q = ref[r] - logp[r]
            term += beta * (np.exp(q) - q - 1)
            g += beta * (1 - np.exp(q))
            room += abs(weight[r]) * beta * (np.exp(q) + 1) * (slack[r] + 8 * U * (1 + abs(q)))
        total += weight[r] * term
        slope[r] = weight[r] * g
        room += abs(weight[r] * free) * (slack[r] + 10 * U * (1 + abs(logp[r] - old[r])))
    return total, np.where(live, logp, 0.0), slope, lse, slack, room + 4 * U * abs(total)
