"""Many rows of logits of mixed kinds (live, clipped, without a target, without
a weight, without a finite logit) through every kernel that takes them, against
the 64-bit definitions, and in place against out of place.  The definitions are
those of train_ref.py in torch on the GPU, a part of the rows at a time."""
import numpy as np
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

INF = float("inf")
LO, HI = 0.2, 0.3
# distances of log(ratio) from 0: on both sides of both bounds (-0.22 and 0.26)
STEPS = [-0.6, -0.1, 0.0, 0.1, 0.2, 0.6]


@pytest.fixture(autouse=True)
def _setup():
    nrm.build()
    nrm.force_plan(nrm.PLAN_AUTO)
    yield
    nrm.force_plan(nrm.PLAN_AUTO)


def packs(n, dtype, more=3):
    """Columns of n packs of 16 bytes and a few more."""
    return n * (4 if dtype == torch.float32 else 8) + more


def parts(rows, v):
    step = max(1, 2 ** 24 // v)
    return [slice(a, min(a + step, rows)) for a in range(0, rows, step)]


def logsoftmax64(z, s):
    """s z less the row's log-sum-exp (as its maximum and log d: their sum loses log d at large logits), lse, and the bound
    of log d (train_ref.logprob); rows without a finite logit -inf."""
    z = z.double()
    m = z.amax(-1, keepdim=True)
    none = m == -INF
    x = (z - torch.where(none, 0.0, m)) * s
    d = torch.exp(x).sum(-1, keepdim=True)
    arg = torch.where(torch.exp(x) > 0, x.abs() * torch.exp(x), 0.0).sum(-1) / torch.where(none, 1.0, d)[:, 0]
    logd = torch.log(d)
    return torch.where(none, -INF, x - logd), (m * s)[:, 0], logd[:, 0], (z.shape[1] / 512 + 104 + 3 * arg) * R.U


def logprob64(z, t, s):
    x, top, logd, slack = logsoftmax64(z, s)
    return x.gather(-1, t[:, None])[:, 0], top + logd, slack


def away64(zt, top, logd, other):
    """zt - top - logd - other; where zt and other are large (a masked target: -1e30 each), what 64 bits keep of
    zt - top alone is not enough, so the two that are nearest cancel first."""
    return torch.where((zt - top).abs() <= (zt - other).abs(), zt - top - other, zt - other - top) - logd


def mixed(rows, v, dtype, seed, s=1.0, scale=2.5, low=None):
    """Logits, targets and a policy's other inputs; of 16 rows two have no target, one no weight, one no finite logit; the
    others are live, some of them clipped.  low: the value of masked logits of some live rows: a third in one piece, every
    third, all of them; and a logit of -low."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.empty(rows, v, dtype=dtype, device="cuda")
    t = torch.randint(0, v, (rows,), generator=g, device="cuda")
    logp = torch.empty(rows, dtype=torch.float64, device="cuda")
    kind = torch.randint(0, 16, (rows,), generator=g, device="cuda")
    for p in parts(rows, v):
        x = scale * torch.randn(p.stop - p.start, v, generator=g, device="cuda")
        x[torch.arange(len(x), device="cuda"), t[p]] += 6 * torch.rand(len(x), generator=g, device="cuda")
        x[kind[p] == 3] = -INF
        if low is not None:
            one, every, whole, hot = ((kind[p] == k) for k in (4, 5, 6, 7))
            x[one, v // 3:2 * v // 3] = low
            t[p][one] %= max(1, v // 3)
            x[every, ::3] = low
            t[p][every] = (t[p][every] // 3 * 3 + 1).clamp(max=v - 1)
            x[whole] = low
            x[hot, t[p][hot]] = -low
        z[p] = x.to(dtype)
        logp[p] = logprob64(z[p], t[p], s)[0]
    step = torch.tensor(STEPS, device="cuda")[torch.randint(0, len(STEPS), (rows,), generator=g, device="cuda")]
    logp = torch.where(kind == 3, -3.0, logp).float()
    old, ref = logp - step, logp + 0.4 * torch.randn(rows, generator=g, device="cuda")
    adv, wt = torch.randn(rows, generator=g, device="cuda"), (0.5 + torch.rand(rows, generator=g, device="cuda")) / rows
    t[kind == 0], t[kind == 1], wt[kind == 2] = -100, v + 5, 0.0
    # what rows that take no part hold is not read
    old[kind == 0] = adv[kind == 1] = float("nan")
    return z, t, old, adv, wt, ref


def near(got, want, room, what):
    bad = ~((got.double() - want).abs() <= room)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist())


def out_room(dtype, want, extra):
    return (want.abs() + extra) * (R.EPS[dtype] / 2) + extra + R.TINY[dtype] / 2


def check_logprob(z, t, s, got):
    v = z.shape[1]
    ok = (t >= 0) & (t < v)
    assert not got[0][~ok].any() and not got[1][~ok].any()
    for p in parts(*z.shape):
        o = ok[p]
        logp, lse, slack = logprob64(z[p][o], t[p][o], s)
        fin = torch.isfinite(logp)
        for a, want in ((got[0][p][o], logp), (got[1][p][o], lse)):
            assert (a[~fin] == -INF).all()
            near(a[fin], want[fin], (slack + R.U * want.abs())[fin] + 1e-45, "logp, lse")


def check_policy(z, t, old, adv, wt, ref, kl, s, got, scale=1.0):
    """The bounds of check_policy in test_gpu_logits.py, over all rows."""
    dtype, v = z.dtype, z.shape[1]
    live = (t >= 0) & (t < v) & (wt != 0)
    assert not got[1][~live].any()
    total = room = 0.0
    for p in parts(*z.shape):
        i = torch.nonzero(live[p])[:, 0]
        assert not (got[2][p][~live[p]] != 0).any()
        x, a = z[p][i], t[p][i]
        zt = x.gather(-1, a[:, None])[:, 0].double() * s
        x, top, logd, slack = logsoftmax64(x, s)
        logp = x.gather(-1, a[:, None])[:, 0]
        none = logp == -INF
        assert (got[1][p][i][none] == -INF).all() and not (got[2][p][i][none] != 0).any()
        i, x, a, logp, zt, top, logd, slack = (q[~none] for q in (i, x, a, logp, zt, top, logd, slack))
        near(got[1][p][i], logp, slack + R.U * logp.abs() + 1e-45, "logp")
        o, A, w, r = (q[p][i].double() for q in (old, adv, wt, ref))
        d, e = away64(zt, top, logd, o), -away64(zt, top, logd, r)
        ratio = torch.exp(d)
        free, held = -A * ratio, -A * ratio.clamp(1 - LO, 1 + HI)
        clipped = held > free
        term, g = torch.maximum(free, held), torch.where(clipped, 0.0, free)
        wrong = (w * free).abs() * (slack + 16 * R.U * (1 + d.abs()))
        room += float(((w * free).abs() * (slack + 10 * R.U * (1 + d.abs()))).sum())
        if kl:
            term, g = term + kl * (torch.exp(e) - e - 1), g + kl * (1 - torch.exp(e))
            wrong += w.abs() * kl * torch.exp(e) * (slack + 16 * R.U * (1 + e.abs()))
            room += float((w.abs() * kl * (torch.exp(e) + 1) * (slack + 8 * R.U * (1 + e.abs()))).sum())
        else:
            assert not (got[2][p][i][clipped] != 0).any()
        total += float((w * term).sum())
        g = w * g * scale * s
        wrong = wrong * abs(scale) * s
        soft = torch.exp(x)
        out = -g[:, None] * soft
        out.scatter_add_(-1, a[:, None], g[:, None])
        mag = out.abs()
        mag.scatter_(-1, a[:, None], g.abs()[:, None])
        soft.scatter_(-1, a[:, None], 1.0)
        arg = torch.where(soft > 0, x.abs(), 0.0)
        extra = mag * ((3 * arg + 16) * R.U + slack[:, None]) + wrong[:, None] * soft.clamp(min=1e-30)
        near(got[2][p][i], out, out_room(dtype, out, extra), "dlogits")
    assert abs(float(got[0]) - total) <= room + 5 * R.U * abs(total) + 1e-45


# --- in place ----------------------------------------------------------------
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,n,cs", [(3001, 2100, 2), (2003, 5000, 4), (2003, 10000, 8), (613, 19000, 8), (311, 5000, 4)])
def test_policy_loss_in_place_where_a_row_takes_a_cluster(rows, n, cs, dtype):
    # every CTA of the cluster overwrites its slice while others may be a step
    # behind: the same bits as out of place, everywhere
    v = packs(n, dtype)
    z, t, old, adv, wt, ref = mixed(rows, v, dtype, n)
    want = nrm.policy_loss(z, t, old, adv, wt, ref, LO, HI, 0.1, out=torch.full_like(z, 3.0))
    plan = nrm.last_plan()
    assert plan[0] == nrm.PLAN_CLUSTER and plan[4] == cs
    for _ in range(3):
        x = z.clone()
        got = nrm.policy_loss(x, t, old, adv, wt, ref, LO, HI, 0.1, out=x)
        assert got[2].data_ptr() == x.data_ptr()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert torch.isfinite(want[0]) and (want[2] != 0).any(-1).sum() > rows / 2
    # targets at the row's ends and at the borders of the CTAs' slices
    edge = torch.tensor([0, 1, v - 1, v - 2, *(v * q // cs + k for q in range(1, cs) for k in (-9, -1, 0, 1, 9))], device="cuda")
    t = edge[torch.arange(rows, device="cuda") % len(edge)]
    want = nrm.policy_loss(z, t, old.nan_to_num(-9.0), adv.nan_to_num(1.0), wt, None, LO, 9.0)
    x = z.clone()
    got = nrm.policy_loss(x, t, old.nan_to_num(-9.0), adv.nan_to_num(1.0), wt, None, LO, 9.0, out=x)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    live = torch.nonzero((wt != 0) & torch.isfinite(want[1]))[:, 0]
    logp = torch.cat([logprob64(z[live[q]], t[live[q]], 1.0)[0] for q in torch.arange(len(live)).split(64)])
    near(want[1][live], logp, (v / 512 + 150) * R.U + R.U * logp.abs(), "logp")


# --- masked logits that are finite -------------------------------------------
# one of each kernel: rows by warps, by CTAs, by clusters, in segments (the
# log-probability of many long rows), and forced through the streaming plan
KINDS = [(400, 20, 0), (310, 500, 0), (400, 900, 0), (310, 1900, 0), (24, 1500, 0), (24, 3000, 0), (20, 20000, 0),
         (310, 2500, 0), (24, 5000, 1), (310, 1500, 1)]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("low", [-1e4, -1e9, -1e10, -1e30, None])
@pytest.mark.parametrize("rows,n,stream", KINDS)
def test_masks_of_large_finite_values(rows, n, stream, low, dtype):
    if low is not None and abs(low) > torch.finfo(dtype).max:
        low = -5e4
    low = torch.finfo(dtype).min if low is None else low
    v = packs(n, dtype)
    z, t, old, adv, wt, ref = mixed(rows, v, dtype, n, low=low)
    if stream:
        nrm.force_plan(nrm.PLAN_GENERIC)
    check_logprob(z, t, 1.0, nrm.logprob_fwd(z, t))
    check_policy(z, t, old, adv, wt, ref, 0.1, 1.0, nrm.policy_loss(z, t, old, adv, wt, ref, LO, HI, 0.1))


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("s", [0.5, 1.0, 1.4, 3.0, 1e6])
@pytest.mark.parametrize("rows,n,stream", [(40, 5, 0), (400, 900, 0), (24, 5000, 0), (310, 2500, 0), (24, 5000, 1)])
def test_a_masked_target_at_any_temperature(rows, n, stream, s, dtype):
    # s (z - max) of a target at the type's lowest value can leave binary32: its
    # log-probability is -inf then, not NaN, and the ratio 0
    v = packs(n, dtype)
    z, t, old, adv, wt, _ = mixed(rows, v, dtype, n, s=s)
    z[::5] = z[::5].clamp(-20, 20)
    at = torch.arange(0, rows, 5, device="cuda")
    t[at] = at % v
    z[at, t[at]] = torch.finfo(dtype).min
    old, adv, wt = old.nan_to_num(-1.0), adv.nan_to_num(1.0).abs(), wt.clamp(min=0.1 / rows)
    if stream:
        nrm.force_plan(nrm.PLAN_GENERIC)
    logp, lse = nrm.logprob_fwd(z, t, s)
    want, lse64, slack = logprob64(z[at], t[at], s)
    # the type's lowest value times s beyond binary32: rounds to -inf
    over = want < -(2.0 - 2.0 ** -24) * 2.0 ** 127
    assert over.any() == (dtype != torch.float16 and s > 1)
    assert (logp[at][over] == -INF).all()
    near(logp[at][~over], want[~over], (slack + R.U * want.abs())[~over], "logp")
    near(lse[at], lse64, slack + R.U * lse64.abs(), "lse")
    # nothing of such a row is left for a positive advantage: as without it
    got = nrm.policy_loss(z, t, old, adv, wt, None, LO, HI, 0.0, s)
    w0 = wt.clone()
    w0[at] = 0.0
    ref = nrm.policy_loss(z, t, old, adv, w0, None, LO, HI, 0.0, s)
    assert torch.isfinite(got[0]) and torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])
    # the log-probability of many long rows sums in another order (segments): each is within its bound of the exact value
    assert torch.equal(got[1][at] == -INF, logp[at] == -INF)
    fin = torch.isfinite(logp[at])
    near(got[1][at][fin], logp[at][fin].double(), 2 * (slack + R.U * want.abs())[fin], "logp of both")


# --- the log-probability's two parts -----------------------------------------
# sums of 1 to 98305 ones: around the powers of two, 0.75 and 1.5 times one and
# sqrt(2) times one
ONES = sorted({max(1, int(f * 2 ** k) + e) for k in (0, 1, 2, 3, 5, 8, 10, 13, 16) for f in (1, 1.5, 2 ** 0.5) for e in (-1, 0, 1)})


@pytest.mark.parametrize("dtype", R.DTYPES)
def test_log_probability_of_equal_logits(dtype):
    # every exponential is 1 and their sum v exactly, so logp = -log v with the
    # error of the logarithm alone: log f (at most 1 ulp of a value below 0.35:
    # 2^-25) and the roundings of two sums of that size (2^-26 each) make 2^-24
    # in the low part, and the high part is the sum's rounding
    for v in ONES:
        z = torch.zeros(2, v, dtype=dtype, device="cuda")
        t = torch.tensor([0, v - 1], device="cuda")
        logp, lse = nrm.logprob_fwd(z, t)
        want = -np.log(v)
        ulp = float(np.spacing(np.float32(abs(want)))) if v > 1 else 0.0
        assert abs(R.f64(logp) - want).max() <= ulp / 2 + 2.0 ** -24 * (v > 1), v
        assert abs(R.f64(lse) + want).max() <= ulp / 2 + 2.0 ** -24 * (v > 1), v
        # the low part: with clip bounds of 0, old = the rounded log-probability
        # and advantages of both signs, the side of the border that the exact
        # remainder lies on decides which row has a gradient
        old = np.float32(want)
        rest = want - float(old)
        if abs(rest) > 2.0 ** -24:
            olds = torch.full((2,), float(old), device="cuda")
            dz = nrm.policy_loss(z, t, olds, torch.tensor([1.0, -1.0], device="cuda"), clip_low=0.0, clip_high=0.0)[2]
            has = (dz != 0).any(-1).tolist()
            assert has == [rest < 0, rest > 0], (v, rest, has)


def test_equal_logits_reach_the_low_part():
    # the test above says something: of its sums more than half have a remainder that decides
    rest = [abs(-np.log(v) - float(np.float32(-np.log(v)))) for v in ONES if v > 1]
    assert sum(r > 2.0 ** -24 for r in rest) > len(rest) / 2


# --- the gradient end to end, from the forward's stats -----------------------
def check_logprob_bwd(z, t, g, s, dz):
    """dz against g s (onehot - softmax(s z)) of the logits themselves, with the bounds of check_policy."""
    v = z.shape[1]
    ok = (t >= 0) & (t < v) & (g != 0)
    for p in parts(*z.shape):
        assert not (dz[p][~ok[p]] != 0).any()
        i = torch.nonzero(ok[p])[:, 0]
        x, _, _, slack = logsoftmax64(z[p][i], s)
        none, nan = x.amax(-1) == -INF, x.isnan().any(-1)  # no finite logit; an infinite one (NaN as anywhere)
        assert not (dz[p][i][none] != 0).any() and dz[p][i][nan].isnan().all()
        i, x, slack = (q[~none & ~nan] for q in (i, x, slack))
        k, a = g[p][i].double()[:, None] * s, t[p][i][:, None]
        soft = torch.exp(x)
        out = (-k * soft).scatter_add_(-1, a, k)
        mag = out.abs().scatter_(-1, a, k.abs())
        arg = torch.where(soft > 0, x.abs(), 0.0)
        near(dz[p][i], out, out_room(z.dtype, out, mag * ((3 * arg + 16) * R.U + slack[:, None])), "dlogits")


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("s", [1.0, 0.7, 2.5])
@pytest.mark.parametrize("rows,n,stream", [(40, 1, 0), (400, 20, 0), (310, 900, 0), (24, 5000, 0), (310, 2500, 0), (24, 5000, 1)])
def test_gradient_from_stats(rows, n, stream, s, dtype):
    # rows with a common offset of up to 1e4 and rows masked as a whole by
    # finite values, the type's lowest among them: what one binary32 lse loses
    v = packs(n, dtype)
    z, t = mixed(rows, v, dtype, n, low=torch.finfo(dtype).min)[:2]
    for i, off in enumerate((1e3, -1e3, 1e4, -1e4)):
        z[8 + i::12] = (z[8 + i::12].float() + off).to(dtype)
    if dtype != torch.float16:
        z[3::12] = -1e30
    if stream:
        nrm.force_plan(nrm.PLAN_GENERIC)
    plain = nrm.logprob_fwd(z, t, s)
    stats = torch.full((rows, 2), 7.0, device="cuda")
    logp, lse = nrm.logprob_fwd(z, t, s, stats=stats)
    same = lambda a, b: torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))  # noqa: E731  (binary16's largest + 1e4: NaN rows)
    assert same(logp, plain[0]) and same(lse, plain[1])
    ok = (t >= 0) & (t < v)
    assert not stats[~ok].any() and torch.equal(stats[ok][:, 0], z[ok].amax(-1).float())
    g = torch.linspace(-1.0, 1.0, rows, device="cuda")
    g[rows // 2] = 0.0
    dz = nrm.logprob_bwd(g, z, t, None, s, stats=stats)
    check_logprob_bwd(z, t, g, s, dz)
    # rows at another alignment, and in place
    flat = torch.empty(rows * (v + 1) + 1, dtype=dtype, device="cuda")
    other = flat[1:].view(rows, v + 1)[:, :v]
    other.copy_(z)
    assert same(nrm.logprob_bwd(g, other, t, None, s, stats=stats), dz)
    x = z.clone()
    got = nrm.logprob_bwd(g, x, t, None, s, stats=stats, out=x)
    assert got.data_ptr() == x.data_ptr() and same(x, dz)


def test_stats_are_refused_in_other_forms():
    z, t, old = (q.cuda() for q in (torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)))
    good = torch.zeros(4, 2, device="cuda")
    for bad in (good.half(), good[:3], good.t().contiguous(), torch.zeros(4, 4, device="cuda")[:, ::2], good.cpu()):
        with pytest.raises(ValueError):
            nrm.logprob_fwd(z, t, stats=bad)
        with pytest.raises(ValueError):
            nrm.logprob_bwd(old, z, t, None, stats=bad)
    with pytest.raises(ValueError):
        nrm.logprob_bwd(old, z, t, None)
    with pytest.raises(nrm.NrmError) as e:
        nrm.logprob_fwd(z, t, stats=z.view(-1)[:8].view(4, 2))
    assert e.value.status == 4


# --- the loss' gradient against differences ----------------------------------
@pytest.mark.parametrize("kl", [0.0, 0.1])
@pytest.mark.parametrize("rows,v", [(10, 700), (6, 5003), (5, 40001)])
def test_gradient_against_differences_along_itself(rows, v, kl):
    # along the gradient's signs the slope is its 1-norm, the largest there is.
    # Central differences of the library's loss differ from it by the formula's
    # own truncation at this step (taken in 64 bits, from the same two points),
    # by the loss' bound at either point over 2 h and by the gradient's bound
    g = torch.Generator().manual_seed(rows)
    z = 2 * torch.randn(rows, v, generator=g)
    t = torch.randint(0, v, (rows,), generator=g)
    z[torch.arange(rows), t] += 8
    logp = torch.from_numpy(R.logprob(z.double().numpy(), t.numpy(), 1.0)[0]).float()
    old = logp - torch.tensor([-0.6, -0.1, 0.1, 0.6, 0.0])[torch.arange(rows) % 5]
    adv = torch.where(torch.arange(rows) % 2 == 0, 1.0, -1.0) * (0.5 + torch.rand(rows, generator=g))
    ref, wt = logp + 0.4 * torch.randn(rows, generator=g), 0.5 + torch.rand(rows, generator=g)
    rest = [x.cuda() for x in (t, old, adv, wt, ref)]
    rest64 = [t.numpy(), *(x.double().numpy() for x in (old, adv, wt, ref))]
    loss = lambda q: float(nrm.policy_loss(q, *rest, LO, HI, kl, want_grad=False)[0])  # noqa: E731
    exact = lambda q: R.policy(R.f64(q), *rest64, LO, HI, kl, 1.0)  # noqa: E731
    dz = nrm.policy_loss(z.cuda(), *rest, LO, HI, kl)[2]
    h = 2.0 ** -5
    hi, lo = z.cuda() + h * dz.sign(), z.cuda() - h * dz.sign()
    # the step that binary32 took, and the slope along it
    d = (hi.double() - lo.double()) / (2 * h)
    slope = float((dz.double() * d).sum())
    out64 = exact(z)
    dz64 = torch.from_numpy(R.grad(z.double().numpy(), rest64[0], out64[3], out64[2], 1.0)[0])
    e_hi, e_lo = exact(hi), exact(lo)
    truncation = abs((e_hi[0] - e_lo[0]) / (2 * h) - float((dz64 * d.cpu()).sum()))
    room = truncation + (e_hi[5] + e_lo[5] + R.U * (abs(e_hi[0]) + abs(e_lo[0]))) / (2 * h) + 512 * R.U * float(dz.double().abs().sum())
    assert room < 0.01 * slope  # nothing less than the whole gradient passes
    assert abs((loss(hi) - loss(lo)) / (2 * h) - slope) <= room


# --- batches of rows ---------------------------------------------------------
# A group (warp, CTA, cluster) takes a batch of up to 32 rows and fetches the
# next live one ahead: live, dead, clipped and empty rows side by side, in each
# kernel, batches of two and more.  (rows, packs, plan, threads, packs a thread)
BATCHES = [(950_001, 3, "warp", 128, 4), (30_011, 100, "warp", 128, 4), (22_003, 250, "warp", 128, 8),
           (15_001, 380, "warp", 128, 12), (15_001, 500, "warp", 128, 16), (7_501, 600, "cta", 128, 8),
           (5_603, 1200, "cta", 160, 8), (4_703, 1500, "cta", 192, 8), (3_701, 1700, "cta", 224, 8),
           (3_701, 1900, "cta", 256, 8), (2_903, 2400, "cluster", 160, 8), (1_201, 6000, "cluster", 192, 8),
           (483, 14000, "cluster", 224, 8), (353, 19000, "cluster", 256, 10)]
KIND = {"warp": nrm.PLAN_WARP, "cta": nrm.PLAN_CTA, "cluster": nrm.PLAN_CLUSTER}


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,n,kind,threads,per", BATCHES)
def test_batches_of_mixed_rows(rows, n, kind, threads, per, dtype):
    v = packs(n, dtype)
    z, t, old, adv, wt, ref = mixed(rows, v, dtype, n + 1)
    z[(t < 0) | (t >= v)] = float("nan")  # not read
    got = nrm.policy_loss(z, t, old, adv, wt, ref, LO, HI, 0.1)
    assert nrm.last_plan()[:3] == (KIND[kind], threads, per)
    check_policy(z, t, old, adv, wt, ref, 0.1, 1.0, got)
    x = z.clone()
    for a, b in zip(nrm.policy_loss(x, t, old, adv, wt, ref, LO, HI, 0.1, out=x), got):
        assert torch.equal(a, b)
    # at another temperature, without the KL term, the gradient scaled
    z, t, old, adv, wt, ref = mixed(rows, v, dtype, n + 2, s=0.6)
    gs = torch.tensor(-3.0, device="cuda")
    check_policy(z, t, old, adv, wt, ref, 0.0, 0.6, nrm.policy_loss(z, t, old, adv, wt, None, LO, HI, 0.0, 0.6, grad_scale=gs), -3.0)
    check_logprob(z, t, 0.6, nrm.logprob_fwd(z, t, 0.6))


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,n", [(7_401, 2300), (3_701, 5001)])
def test_batches_of_rows_in_segments(rows, n, dtype):
    # the log-probability alone, rows longer than a CTA's registers, batches of two and of one
    v = packs(n, dtype)
    z, t = mixed(rows, v, dtype, n + 1, s=1.3)[:2]
    z[(t < 0) | (t >= v)] = float("nan")
    got = nrm.logprob_fwd(z, t, 1.3)
    assert nrm.last_plan()[:3] == (nrm.PLAN_CTA, 256, 8)
    check_logprob(z, t, 1.3, got)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,n,cs", [(1009, 300, 1), (311, 1500, 1), (200, 1300, 2), (100, 2500, 4), (20, 5000, 8), (70, 4200, 8)])
def test_the_streaming_plan(rows, n, cs, dtype):
    # forced: a row by one, two, four and eight CTAs, also in place
    v = packs(n, dtype)
    z, t, old, adv, wt, ref = mixed(rows, v, dtype, n + 1, s=1.2)
    z[(t < 0) | (t >= v)] = float("nan")
    nrm.force_plan(nrm.PLAN_GENERIC)
    got = nrm.logprob_fwd(z, t, 1.2)
    assert nrm.last_plan()[0] == nrm.PLAN_GENERIC and max(1, nrm.last_plan()[4]) == cs
    check_logprob(z, t, 1.2, got)
    got = nrm.policy_loss(z, t, old, adv, wt, ref, LO, HI, 0.1, 1.2)
    assert nrm.last_plan()[0] == nrm.PLAN_GENERIC and max(1, nrm.last_plan()[4]) == cs
    check_policy(z, t, old, adv, wt, ref, 0.1, 1.2, got)
    for _ in range(2):
        x = z.clone()
        for a, b in zip(nrm.policy_loss(x, t, old, adv, wt, ref, LO, HI, 0.1, 1.2, out=x), got):
            assert torch.equal(a, b)
