"""Target log-probabilities, their gradient and the policy loss on the GPU
against the 64-bit definitions of train_ref.py."""
import numpy as np
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

INF = float("inf")


@pytest.fixture(autouse=True)
def _setup():
    nrm.build()
    yield


def make(rows, v, dtype, seed=0, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    z = scale * torch.randn(rows, v, generator=g)
    t = torch.randint(0, v, (rows,), generator=g)
    z[torch.arange(rows), t] += 6 * torch.rand(rows, generator=g)
    return z.to(dtype).cuda(), t.cuda()


def place(z, pad, shift):
    """The same rows in a buffer with `pad` columns behind each and `shift` elements before the first."""
    rows, v = z.shape
    flat = torch.full((rows * (v + pad) + shift,), 7.0, dtype=z.dtype, device="cuda")
    view = flat[shift:].view(rows, v + pad)[:, :v]
    view.copy_(z)
    return view, flat


def rest_untouched(flat, rows, v, pad, shift):
    return (flat[:shift] == 7.0).all() and (flat[shift:].view(rows, v + pad)[:, v:] == 7.0).all()


def check_logprob(z, t, s, got):
    logp, lse, slack = R.logprob(R.f64(z), t.cpu().numpy(), s)
    for a, ref, what in ((got[0], logp, "logp"), (got[1], lse, "lse")):
        fin = np.isfinite(ref)
        a = R.f64(a)
        assert np.array_equal(a[~fin], ref[~fin]), what
        R.check(a[fin], ref[fin], (slack + R.U * np.abs(ref))[fin] + 1e-45, what)
    return lse


# one pack, ragged ends, one row and many, one CTA and clusters
SIZES = [(1, 1), (3, 2), (5, 7), (4, 8), (2, 65), (700, 33), (9, 1000), (3, 4096), (2, 8191), (300, 8193),
         (310, 16384), (1, 40000), (17, 50001), (2, 131072)]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", SIZES)
def test_logprob(rows, v, dtype):
    z, t = make(rows, v, dtype, v)
    got = nrm.logprob_fwd(z, t)
    check_logprob(z, t, 1.0, got)
    dlogp = torch.linspace(-1, 1, rows).cuda()
    dz = nrm.logprob_bwd(dlogp, z, t, got[1])
    check_grad(z, t, got[1], dlogp, 1.0, dz)


def check_grad(z, t, lse, g, s, dz, d_slack=0.0):
    """d_slack: the relative error of each row's exp(-lse), where it is not given but computed."""
    g64 = R.f64(g)
    ref, arg = R.grad(R.f64(z), t.cpu().numpy(), R.f64(lse), g64, s)
    p = np.abs(ref)
    tt = t.cpu().numpy()
    ok = (tt >= 0) & (tt < z.shape[1])
    gs = np.abs(g64 * s)
    p[ok, tt[ok]] = gs[ok]  # at the target: a difference of two terms of at most |g s|
    extra = p * ((3 * arg + 12) * R.U + d_slack)
    R.check(dz, ref, R.out_bound(z.dtype, ref, extra), "dlogits")


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("v,pad,shift", [(64, 0, 1), (1003, 1, 0), (1003, 5, 3), (8200, 8, 0), (8200, 8, 8), (20011, 2, 5)])
def test_logprob_strides_alignment_in_place(v, pad, shift, dtype):
    rows = 6
    z0, t = make(rows, v, dtype, v + pad)
    t[0], t[1] = 0, v - 1
    z, flat = place(z0, pad, shift)
    got = nrm.logprob_fwd(z, t, 0.7)
    check_logprob(z0, t, 0.7, got)
    dlogp = torch.tensor([1.0, -2.0, 0.5, 0.0, 3.0, -0.1]).cuda()
    other, oflat = place(torch.zeros_like(z0), pad + 1, shift + 1)  # rows of another alignment
    dz = nrm.logprob_bwd(dlogp, z, t, got[1], 0.7, out=other)
    check_grad(z0, t, got[1], dlogp, 0.7, dz)
    assert rest_untouched(oflat, rows, v, pad + 1, shift + 1)
    dz2 = nrm.logprob_bwd(dlogp, z, t, got[1], 0.7, out=z)
    assert dz2.data_ptr() == z.data_ptr()
    assert torch.equal(dz2, dz) and rest_untouched(flat, rows, v, pad, shift)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("v", [9, 1000, 30001])
def test_rows_that_take_no_part_and_masked_entries(v, dtype):
    z, t = make(8, v, dtype, 5)
    z[0, 1:] = -INF          # one finite logit, the target
    t[0] = 0
    z[1, 0::2] = -INF        # half masked
    t[1] = 1
    z[2] = -INF              # nothing left
    t[3], t[4] = -100, v     # no target
    z[3], z[4] = float("nan"), INF
    t[5] = 2
    z[5, 2] = -INF           # an impossible target
    z[6, 1] = 1e4 if dtype != torch.float16 else 6e4
    logp, lse = nrm.logprob_fwd(z, t)
    check_logprob(z, t, 1.0, (logp, lse))
    assert logp[0] == 0 and logp[2] == -INF and lse[2] == -INF and logp[5] == -INF
    assert logp[3] == logp[4] == lse[3] == lse[4] == 0
    dlogp = torch.ones(8, device="cuda")
    dlogp[7] = 0.0
    z[7, 3] = float("nan")   # a row without a slope is not read
    dz = nrm.logprob_bwd(dlogp, z, t, lse)
    for r in (2, 3, 4, 7):
        assert not (dz[r] != 0).any(), r
    live = [0, 1, 5, 6]
    check_grad(z[live], t[live], lse[live], dlogp[live], 1.0, dz[live])


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", [(6, 40), (6, 1003), (6, 5000), (3, 40001), (2, 300001)])
def test_masks_of_the_lowest_value(rows, v, dtype):
    # the type's lowest value instead of -inf: where it is all a row has, the
    # row is uniform; elsewhere it has probability 0
    low = torch.finfo(dtype).min
    z, t = make(rows, v, dtype, 8)
    z[0] = low
    z[1, ::3] = low
    t[1] = 1
    logp, lse = nrm.logprob_fwd(z, t)
    # -log v at a lse of -3.4e38 is all rounding there; logp keeps it
    assert abs(float(logp[0]) + np.log(v)) < (v / 512 + 120) * R.U + 1e-6
    check_logprob(z[1:], t[1:], 1.0, (logp[1:], lse[1:]))
    one = torch.ones(rows, device="cuda")
    loss, lp, dz = nrm.policy_loss(z, t, logp, -one, one)
    assert torch.equal(lp, logp)
    ref = np.full(v, -1.0 / v)
    ref[int(t[0])] += 1.0
    R.check(dz[0], ref, R.out_bound(dtype, ref, np.abs(ref) * (v / 512 + 200) * R.U), "dlogits")
    assert not (dz[1, ::3] != 0).any()


def test_nan_and_infinite_logits_are_not_hidden():
    z, t = make(4, 5000, torch.float32)
    z[0, 4000] = float("nan")
    z[1] = -INF
    z[1, 17] = float("nan")
    z[2, 100] = INF
    logp, lse = nrm.logprob_fwd(z, t)
    assert torch.isnan(logp[:3]).all() and torch.isnan(lse[:3]).all() and torch.isfinite(logp[3])


def policy_inputs(rows, v, dtype, seed=0, s=1.0):
    """Ratios at fixed distances from the clip bounds (0.8 and 1.3), on both sides of each."""
    z, t = make(rows, v, dtype, seed)
    logp = R.logprob(R.f64(z), t.cpu().numpy(), s)[0]
    g = torch.Generator().manual_seed(seed + 1)
    step = torch.tensor([-0.6, -0.1, 0.0, 0.1, 0.2, 0.6])[torch.randint(0, 6, (rows,), generator=g)]
    logp = torch.from_numpy(logp).float()
    old, ref = logp - step, logp + 0.4 * torch.randn(rows, generator=g)
    adv, wt = torch.randn(rows, generator=g), torch.rand(rows, generator=g) / rows
    if rows > 3:
        t[1], t[3] = -100, v + 5
        wt[2] = 0.0
        adv[1] = old[2] = ref[3] = float("nan")
    return [x.cuda() for x in (z, t, old, adv, wt, ref)]


def check_policy(z, t, old, adv, wt, ref, lo, hi, kl, s, got, scale=1.0):
    n = [R.f64(x) if x.is_floating_point() else x.cpu().numpy() for x in (z, t, old, adv, wt, ref)]
    loss, logp, slope, lse, slack, room = R.policy(*n, lo, hi, kl, s)
    fin = np.isfinite(logp)
    R.check(R.f64(got[1])[fin], logp[fin], (slack + R.U * np.abs(logp))[fin] + 1e-45, "logp")
    assert np.array_equal(R.f64(got[1])[~fin], logp[~fin])
    R.check(np.array(R.f64(got[0])), np.array(loss), room + R.U * abs(loss) + 1e-45, "loss")
    if got[2] is None:
        return
    # the slope's own error: that of logp (its argument) and a few operations
    g = torch.from_numpy(slope * scale)
    d, e = (np.nan_to_num(x) for x in (logp - n[2], n[5] - logp))
    free = np.nan_to_num(np.abs(n[4] * n[3]) * np.exp(np.clip(d, -50, 50)))
    klm = np.nan_to_num(np.abs(n[4]) * kl * np.exp(np.clip(e, -50, 50)))
    wrong = (free + klm) * (slack + 16 * R.U * (1 + np.abs(d) + np.abs(e))) * abs(scale) * s
    out, arg = R.grad(n[0], n[1], lse, R.f64(g), s)
    p = np.abs(out)
    ok = (n[1] >= 0) & (n[1] < z.shape[1])
    gs = np.abs(R.f64(g) * s)
    p[ok, n[1][ok]] = gs[ok]
    extra = p * ((3 * arg + 16) * R.U + slack[:, None])
    soft = np.where(gs[:, None] > 0, p / np.maximum(gs, 1e-300)[:, None], 0.0)
    extra = extra + wrong[:, None] * np.maximum(soft, 1e-30)
    none = ~np.array([0 <= a < z.shape[1] for a in n[1]]) | (n[4] == 0)
    assert not (got[2][torch.from_numpy(none).cuda()] != 0).any()
    R.check(got[2], out, R.out_bound(z.dtype, out, extra), "dlogits")


@pytest.mark.parametrize("kl", [0.0, 0.1])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", SIZES)
def test_policy_loss(rows, v, dtype, kl):
    args = policy_inputs(rows, v, dtype, rows)
    z, t, old, adv, wt, ref = args
    got = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, kl)
    check_policy(*args, 0.2, 0.3, kl, 1.0, got)
    fwd = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, kl, want_grad=False)
    assert fwd[2] is None and torch.equal(fwd[0], got[0]) and torch.equal(fwd[1], got[1])


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("v,pad,shift", [(1003, 1, 0), (1003, 5, 3), (8200, 8, 0), (20011, 2, 5)])
def test_policy_loss_strides_in_place_and_scale(v, pad, shift, dtype):
    args = policy_inputs(12, v, dtype, 3, 1.4)
    z0, t, old, adv, wt, ref = args
    z, flat = place(z0, pad, shift)
    gs = torch.tensor(2.5, device="cuda")
    other, oflat = place(torch.zeros_like(z0), pad + 1, shift + 1)
    got = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.05, 1.4, grad_scale=gs, out=other)
    check_policy(*args, 0.2, 0.3, 0.05, 1.4, got, 2.5)
    assert rest_untouched(oflat, 12, v, pad + 1, shift + 1)
    inp = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.05, 1.4, grad_scale=gs, out=z)
    assert inp[2].data_ptr() == z.data_ptr() and torch.equal(inp[2], got[2]) and torch.equal(inp[0], got[0])
    assert rest_untouched(flat, 12, v, pad, shift)


def test_policy_loss_masked_rows_and_edges():
    z, t, old, adv, wt, ref = policy_inputs(8, 5003, torch.bfloat16, 4)
    z[4] = -INF                      # a live row with nothing left
    z[5, 100:] = -INF
    t[5] = 3
    z[1], z[2], z[3] = float("nan"), INF, float("nan")   # rows that take no part
    logp = torch.from_numpy(R.logprob(R.f64(z), t.cpu().numpy(), 1.0)[0]).float().cuda()
    old[5], ref[5] = logp[5] - 0.1, logp[5] + 0.2
    got = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1)
    assert got[1][4] == -INF and torch.isfinite(got[0]) and torch.isfinite(got[2]).all()
    for r in (1, 2, 3, 4):
        assert not (got[2][r] != 0).any()
    assert got[1][1] == got[1][2] == got[1][3] == 0
    zz = z.clone()
    zz[1:4] = 0
    wt4 = wt.clone()
    wt4[4] = 0
    logp4 = got[1].clone()
    logp4[4] = 0
    check_policy(zz, t, old, adv, wt4, ref, 0.2, 0.3, 0.1, 1.0, (got[0], logp4, got[2]))
    # no row takes part; no row at all; no weights
    none = nrm.policy_loss(z, torch.full_like(t, -100), old, adv, wt, ref, 0.2, 0.3, 0.1)
    assert none[0] == 0 and not (none[2] != 0).any()
    e = nrm.policy_loss(z[:0], t[:0], old[:0], adv[:0])
    torch.cuda.synchronize()
    assert e[0] == 0 and e[2].shape == (0, 5003)
    live = [0, 5, 6, 7]
    one = torch.ones(4, device="cuda")
    sub = [z[live], t[live], old[live], adv[live]]
    check_policy(*sub, one, ref[live], 0.2, 0.3, 0.0, 1.0, nrm.policy_loss(*sub, clip_high=0.3))


# rows by warps at each of their register budgets, and the cluster's from its
# smallest to the rows it has no room for; the last of a budget and the first
# of the next
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,packs", [(305, 128), (305, 129), (304, 257), (307, 385), (305, 512), (303, 300),
                                        (2433, 1100), (1217, 2100), (1217, 2600), (1217, 3400),
                                        (3, 16385), (2, 20481), (2, 24577), (2, 32768), (1, 32769), (2, 40959), (1, 41000)])
def test_every_budget_of_packs(rows, packs, dtype):
    v = packs * (4 if dtype == torch.float32 else 8) + 3
    args = policy_inputs(rows, v, dtype, packs)
    z, t, old, adv, wt, ref = args
    check_policy(*args, 0.2, 0.3, 0.1, 1.0, nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1))
    got = nrm.logprob_fwd(z, t)
    live = (t >= 0) & (t < v)
    check_logprob(z[live], t[live], 1.0, [x[live] for x in got])
    dlogp = torch.linspace(-1, 1, rows).cuda()
    check_grad(z[live], t[live], got[1][live], dlogp[live], 1.0, nrm.logprob_bwd(dlogp, z, t, got[1])[live])


def test_the_loss_of_many_rows_that_cancel():
    # one logit a row: its log-probability is 0 and the ratio 1, exactly, so the
    # loss is -sum(adv) with nothing but the sum's own rounding.  A thread adds
    # rows / 1024 terms; each addition's error is kept, at most u A of the sum A
    # of the magnitudes, and what adding those up loses is (rows / 1024)^2 2 u^2 A
    rows = 300_001
    g = torch.Generator().manual_seed(3)
    adv = torch.randn(rows, generator=g)
    adv[1000], adv[250_000] = 3e6, -3e6
    zero = torch.zeros(rows, device="cuda")
    z, t = torch.ones(rows, 1, device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda")
    loss, logp, _ = nrm.policy_loss(z, t, zero, adv.cuda())
    assert not logp.any()
    want, total = float(-adv.double().sum()), float(adv.double().abs().sum())
    assert abs(float(loss) - want) <= R.U * abs(want) + ((rows / 1024) ** 2 + 64) * 2 * R.U ** 2 * total
    for bad in (INF, -INF, float("nan")):
        adv[77] = bad
        got = float(nrm.policy_loss(z, t, zero, adv.cuda())[0])
        assert got == -bad or (bad != bad and got != got)


def test_clipped_rows_have_no_gradient_without_kl():
    z, t = make(6, 3000, torch.float32, 9)
    logp, _ = nrm.logprob_fwd(z, t)
    old = logp - torch.tensor([0.5, -0.5, 0.5, -0.5, 0.0, 0.1], device="cuda")
    adv = torch.tensor([1.0, -1.0, -1.0, 1.0, 1.0, -1.0], device="cuda")
    loss, _, dz = nrm.policy_loss(z, t, old, adv)
    norms = dz.abs().sum(-1)
    assert (norms[:2] == 0).all() and (norms[2:] > 0).all()
    want = -(1.2 + -0.8 + -np.exp(0.5) + np.exp(-0.5) + 1.0 - np.exp(0.1))
    # six ratios of at most 1.7, each within (3000 / 512 + 110 + 3 * 20) u of its value
    assert abs(float(loss) - want) < 6 * 1.7 * 200 * R.U


def test_gradient_against_differences_of_the_library():
    # the loss along a random direction, binary32 logits; central differences of
    # step h err by h^2/6 |f'''| (|direction| <= 1, values O(1)) and by the loss'
    # own rounding over h
    z, t, old, adv, wt, ref = policy_inputs(10, 700, torch.float32, 2)
    loss, _, dz = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1)
    g = torch.Generator().manual_seed(7)
    d = torch.randn(z.shape, generator=g).cuda()
    d /= d.abs().max()
    h = 2.0 ** -6
    hi = nrm.policy_loss(z + h * d, t, old, adv, wt, ref, 0.2, 0.3, 0.1, want_grad=False)[0].double()
    lo = nrm.policy_loss(z - h * d, t, old, adv, wt, ref, 0.2, 0.3, 0.1, want_grad=False)[0].double()
    slope = float((dz.double() * d.double()).sum())
    # the rows' weights sum to at most 1, |A| <= 4, ratios <= 2: values and third derivatives below 16
    assert abs(float(hi - lo) / (2 * h) - slope) < 16 * h * h / 6 + 16 * 300 * R.U / h


def test_leading_dimensions_stream_and_graph():
    z, t, old, adv, wt, ref = (x.view(2, 6, *x.shape[1:]) for x in policy_inputs(12, 4099, torch.bfloat16, 6))
    want = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1)
    assert want[1].shape == (2, 6) and want[2].shape == z.shape and want[0].shape == ()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, ws = torch.zeros_like(z), torch.zeros(64, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = nrm.policy_loss(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1, out=out, workspace=ws)
    for _ in range(2):
        out.fill_(3.0)
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(cap, want))


def test_more_than_2_to_the_31_logits():
    rows, v = 21000, 110001
    z = torch.zeros(rows, v, dtype=torch.bfloat16, device="cuda")
    z[:, 5] = 3.0
    t = torch.full((rows,), 5, device="cuda")
    old = torch.full((rows,), np.log(np.exp(3.0) / (v - 1 + np.exp(3.0))), device="cuda")
    adv = torch.full((rows,), -1.0, device="cuda")
    loss, logp, dz = nrm.policy_loss(z, t, old, adv, out=z)  # ratio 1: the slope is 1 everywhere
    prob = np.exp(3.0) / (v - 1 + np.exp(3.0))
    lp, slack = np.log(prob), (v / 512 + 130) * R.U
    assert float((logp.double() - lp).abs().max()) <= slack + 12 * R.U
    assert abs(float(loss) - rows) <= rows * (2 * slack + 16 * R.U)
    for r in (0, 1, 11000, rows - 2, rows - 1):
        row = dz[r].double().cpu().numpy()
        ref = np.full(v, -1.0 / (v - 1 + np.exp(3.0)))
        ref[5] = 1 - prob
        R.check(row, ref, R.out_bound(torch.bfloat16, ref, np.abs(ref) * 4 * slack), "dlogits")


def test_bounded_waits_give_up_and_report():
    # wait limit 0: every wait for a peer's pair gives up at once, raises the
    # fault bit and the kernel ends; the next call is unaffected
    args = policy_inputs(5, 50001, torch.bfloat16, 6)
    assert nrm.device_fault(clear=True) == 0
    old = nrm.set_wait_limit(0)
    try:
        nrm.policy_loss(*args, 0.2, 0.3, 0.1)
        plan = nrm.last_plan()
        torch.cuda.synchronize()
        bits = nrm.device_fault(clear=True)
    finally:
        nrm.set_wait_limit(old)
    assert plan[0] == nrm.PLAN_CLUSTER and bits & 1
    check_policy(*args, 0.2, 0.3, 0.1, 1.0, nrm.policy_loss(*args, 0.2, 0.3, 0.1))
    assert nrm.device_fault(clear=True) == 0


def test_refused_tensors():
    z, t, old, adv, wt, ref = policy_inputs(8, 64, torch.float16)
    for call in (lambda: nrm.logprob_fwd(z, t.int()), lambda: nrm.logprob_fwd(z, t[:4]), lambda: nrm.logprob_fwd(z.t(), t),
                 lambda: nrm.logprob_bwd(old.half(), z, t, old), lambda: nrm.logprob_bwd(old, z, t, old, out=z.float()),
                 lambda: nrm.policy_loss(z, t, old[:3], adv), lambda: nrm.policy_loss(z, t, old, adv.cpu()),
                 lambda: nrm.policy_loss(z, t, old, adv, grad_scale=old)):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: nrm.logprob_fwd(z, t, 0.0), 5), (lambda: nrm.policy_loss(z, t, old, adv, clip_low=2.0), 5),
                         (lambda: nrm.policy_loss(z, t, old, adv, kl_coef=0.1), 1),
                         (lambda: nrm.policy_loss(z, t, old, adv, logp=old), 4)):
        with pytest.raises(nrm.NrmError) as e:
            call()
        assert e.value.status == status
