"""The gradient of renormalised routing weights where the chosen scores are far
below the row's largest or below binary32's range, on the GPU against the
weights' own form: softmax, or sigmoids' ratios, over the chosen alone in 64
bits.

u = 2^-24.  A weight is exp of a difference of at most 104 (below that it is 0 in
binary32: 2^-126 of |d|), whose rounding weighs as much in u, + 16 u for the
exponential, the sum over at most 32 and the division: 120 u < 2^-17.  The mean of d
and d less the mean are good to that of |d| + sum w |d|, so the product to 4 2^-17 of
w (|d| + sum w |d|).  Scores with their gradients as in block_ref.py.
"""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

INF = float("inf")


@pytest.fixture(autouse=True, scope="module")
def _built():
    nrm.build()


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return scale * torch.randn(*shape, generator=g, device="cuda")


def renormalised(dw, x, ids, score, scale, dscores=None):
    """dx in 64 bits, its bound, and the weights that the forward gives."""
    x = x.double()
    ok = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(ok, ids, 0)
    log = x if score == "softmax" else torch.nn.functional.logsigmoid(x)  # of the scores, but for a constant
    log = torch.where(ok, log.gather(1, at), -INF)
    w = torch.where(ok.any(1, keepdim=True), torch.softmax(log, -1), 0.0)
    d = torch.where(ok, dw.double() * scale, 0.0)
    part = w * (d - (w * d).sum(1, keepdim=True))
    mag = w * (d.abs() + (w * d.abs()).sum(1, keepdim=True))
    if score == "sigmoid":
        rest = torch.where(ok, torch.sigmoid(-x).gather(1, at), 0.0)
        part, mag = part * rest, mag * rest
    dx, big = torch.zeros_like(x).scatter_add_(1, at, part), torch.zeros_like(x).scatter_add_(1, at, mag)
    bound = 4 * R.SCORE * big + 2.0 ** -126 * (1 + d.abs().sum(1, keepdim=True))
    if dscores is not None:
        ref, slack = R.route_grad(torch.zeros_like(dw), x, ids, score=score, renormalize=False, dscores=dscores)
        dx, bound = dx + ref, bound + slack
    return dx, bound, w * scale


def check(dw, x, ids, score, scale=1.7, dscores=None):
    ref, slack, w = renormalised(dw, x, ids, score, scale, dscores)
    how = dict(score=score, renormalize=True, scale=scale, dscores=dscores)
    dx = nrm.route_bwd(dw, x, ids, **how)
    R.check(dx, ref, R.out_bound(x.dtype, ref, slack), "dx")
    out = x.clone()
    assert nrm.route_bwd(dw, out, ids, out=out, **how) is out and torch.equal(out, dx)
    return w


def some_ids(tokens, experts, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(tokens, experts, generator=g, device="cuda").topk(k, -1).indices


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("balance", [False, True])
@pytest.mark.parametrize("below", [0.0, 30.0, 80.0, 88.0, 90.0, 97.0, 103.0, 120.0, 700.0, 6e4])
@pytest.mark.parametrize("experts,k", [(64, 1), (64, 6), (160, 8), (1000, 32)])
def test_softmax_far_below_the_largest(experts, k, below, balance, dtype):
    tokens = 50
    ids = some_ids(tokens, experts, k, 1)
    x = randn(tokens, experts, seed=2)
    if below:
        x.scatter_(1, ids, x.gather(1, ids) - below)
    x = x.to(dtype)
    check(randn(tokens, k, seed=3), x, ids, "softmax", dscores=randn(tokens, experts, seed=4, scale=0.1) if balance else None)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("balance", [False, True])
@pytest.mark.parametrize("below", [0.0, 30.0, 80.0, 87.0, 90.0, 97.0])
@pytest.mark.parametrize("experts,k", [(64, 1), (64, 6), (160, 8), (1000, 32)])
def test_small_sigmoids(experts, k, below, balance, dtype):
    tokens = 50
    ids = some_ids(tokens, experts, k, 1)
    x = randn(tokens, experts, seed=2)
    x = x.scatter_(1, ids, x.gather(1, ids) - below).to(dtype)
    check(randn(tokens, k, seed=3), x, ids, "sigmoid", dscores=randn(tokens, experts, seed=4, scale=0.1) if balance else None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [30.0, 1000.0])
def test_chosen_by_a_large_bias(score, scale):
    # the forward's own choice against the scores; its weights have this gradient.
    # Sigmoids that are all 0 in binary32 have weights of 0, and their gradient is 0
    x = randn(50, 128, seed=8, scale=scale)
    w, ids, _ = nrm.route_fwd(x, 8, randn(128, seed=9, scale=50.0), score=score)
    dw = randn(50, 8, seed=1)
    none = (w == 0).all(1)
    assert torch.isfinite(nrm.route_bwd(dw, x, ids, score=score)).all()
    want = check(dw[~none], x[~none], ids[~none], score, scale=1.0)
    # a sigmoid below the normal range is off by up to 2^-149 of their sum
    total = R.scores64(x, "sigmoid").gather(1, ids).sum(1, keepdim=True)[~none].clamp_min(2.0 ** -149)
    R.check(w[~none], want, 2 * R.SCORE * want + (2.0 ** -126 + (2.0 ** -126 / total if score == "sigmoid" else 0.0)), "weights")
    x = x * 0 - 1000.0
    assert not nrm.route_bwd(dw, x, ids, score="sigmoid").any()
    x[0] = -INF
    assert not nrm.route_bwd(dw, x, ids, score="sigmoid").any() and not nrm.route_bwd(dw, x, ids)[0].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_listed_twice_and_missing_far_below(score):
    x = randn(6, 64, seed=1)
    x[:, 10:] -= 95.0
    ids = some_ids(6, 54, 6, 2) + 10
    ids[0, 3] = ids[0, 1]
    ids[1] = 19
    ids[2, 1:] = -1
    ids[3] = torch.tensor([64, -1, -5, 1 << 40, 20, 63])
    ids[4] = -1
    for dscores in (None, randn(6, 64, seed=3)):
        check(randn(6, 6, seed=2), x, ids, score, dscores=dscores)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_below_against_differences(score):
    # central differences of the forward's weights in 64 bits, through the choice held
    x = randn(5, 32, seed=1)
    x[:, 8:] -= 92.0
    ids, dw, step = some_ids(5, 24, 4, 2) + 8, randn(5, 4, seed=3), 2.0 ** -10
    dx = nrm.route_bwd(dw, x, ids, score=score).double()
    for j in range(4):
        hi, lo = x.double(), x.double()
        hi.scatter_add_(1, ids[:, j:j + 1], torch.full((5, 1), step, dtype=torch.float64, device="cuda"))
        lo.scatter_add_(1, ids[:, j:j + 1], torch.full((5, 1), -step, dtype=torch.float64, device="cuda"))
        d = sum(s * (renormalised(dw, v, ids, score, 1.0)[2] * dw).sum(1) for s, v in ((1, hi), (-1, lo))) / (2 * step)
        # third derivatives of a softmax are below 1: step^2 / 6 of sum |dw|
        assert ((d - dx.gather(1, ids[:, j:j + 1])[:, 0]).abs() <= (step ** 2 / 6 + 2.0 ** -14) * dw.abs().sum(1)).all()


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_expert_alone(score, dtype):
    # its weight is the scale, whatever its logit
    x = randn(500, 96, seed=1, scale=4.0).to(dtype)
    ids = some_ids(500, 96, 3, 2)
    assert not nrm.route_bwd(randn(500, 1, seed=3), x, ids[:, :1].contiguous(), score=score).any()
    ids[:, 0] = ids[:, 2] = -1
    assert not nrm.route_bwd(randn(500, 3, seed=3), x, ids, score=score).any()
