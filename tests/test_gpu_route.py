"""Routing to experts, forward and backward, on the GPU against the 64-bit
definition of block_ref.py.  The chosen experts have to be equal, whatever the
distance between them."""
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


def check(x, k, bias=None, **how):
    want, ids = R.route(x, k, bias, **how)
    # a sigmoid below binary32's range is off by up to 2^-126, and as much of the
    # sum that it is divided by; a renormalised softmax does not underflow
    low = torch.tensor(2.0 ** -126, dtype=torch.float64)
    if how.get("renormalize", True) and how.get("score") == "sigmoid":
        total = R.route(x, k, bias, **dict(how, renormalize=False, scale=1.0))[0].sum(-1, keepdim=True)
        low = low * how.get("scale", 1.0) / total.clamp_min(2.0 ** -500)
    w, got, sc = nrm.route_fwd(x, k, bias, want_scores=True, **how)
    assert torch.equal(got.cpu(), ids), (got.cpu() != ids).nonzero()[:5].tolist()
    R.check(w.cpu(), want, R.SCORE * want.abs() * 2 + low, "weights")
    ref = R.scores64(x, how.get("score", "softmax"))
    R.check(sc, ref, R.SCORE * ref + 2.0 ** -126, "scores")
    w2, got2, none = nrm.route_fwd(x, k, bias, **how)  # without the scores the sum may be another
    assert none is None and torch.equal(got2, got)
    R.check(w2.cpu(), want, R.SCORE * want.abs() * 2 + low, "weights")


FORMS = [  # experts, k, groups, top_groups, group_top
    (1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (3, 1, 1, 1, 1), (8, 2, 1, 1, 1), (33, 8, 1, 1, 1), (64, 6, 1, 1, 1), (64, 32, 1, 1, 1),
    (128, 8, 1, 1, 1), (160, 6, 8, 3, 1), (160, 6, 8, 3, 2), (256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (255, 8, 1, 1, 1),
    (255, 8, 3, 2, 2), (512, 10, 4, 1, 2), (500, 10, 1, 1, 1), (1024, 32, 1, 1, 1), (1024, 32, 32, 7, 2), (1023, 4, 1, 1, 1),
    (96, 3, 12, 5, 2), (32, 4, 32, 6, 2), (40, 4, 20, 3, 1), (256, 8, 8, 8, 2), (768, 8, 3, 2, 1), (24, 6, 8, 2, 2),
]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts,k,groups,top_groups,group_top", FORMS)
def test_against_the_definition(experts, k, groups, top_groups, group_top, with_bias, score, dtype):
    x = randn(203, experts, seed=experts + k, scale=1.5).to(dtype)
    bias = randn(experts, seed=3, scale=0.05) if with_bias else None
    renorm = (experts + k) % 2 == 0
    check(x, k, bias, score=score, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm,
          scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups,group_top", [(256, 8, 4, 2), (256, 1, 1, 1), (64, 1, 1, 1), (160, 8, 3, 1)])
def test_many_tokens(experts, groups, top_groups, group_top, score):
    x = randn(20000, experts, seed=1, scale=1.5)
    check(x, 8 if experts > 64 else 6, randn(experts, seed=3, scale=0.05), score=score, groups=groups, top_groups=top_groups,
          group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,k", [(64, 6), (128, 8), (256, 20), (256, 32), (700, 9)])
def test_choices_a_rounding_apart(experts, k, score):
    # biases that make every expert of a token equal up to the bias' own rounding,
    # in which the order in binary32 is that of the last bits
    x = randn(32, experts, seed=4)
    s = R.scores64(x, score)
    for t in range(32):
        bias = (1.0 - s[t]).float()
        check(x[t:t + 1], k, bias, score=score)
        bias[::3] -= 0.25
        check(x[t:t + 1], k, bias, score=score, groups=4, top_groups=2, group_top=2)
        check(x[t:t + 1], k, bias, score=score, groups=4, top_groups=3, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_a_rounding_apart(score):
    x = torch.full((64, 256), 3.0, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (x.view(torch.int32) + torch.randint(0, 40, x.shape, generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
    check(x, 8, score=score)
    check(x, 8, score=score, groups=8, top_groups=3, group_top=1)
    check(x - 5.0, 32, score=score)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts,k", [(64, 8), (256, 8), (1000, 32)])
def test_equal_logits_go_to_the_lowest_index(experts, k, with_bias, dtype):
    bias = torch.zeros(experts, device="cuda") if with_bias else None
    x = torch.zeros(5, experts, device="cuda", dtype=dtype)
    x[1] = 2.0
    x[2, ::2] = 1.0
    x[3] = randn(experts, seed=1).round().to(dtype)
    x[4, :] = -0.0
    x[4, 7:20] = 0.0  # equal to -0
    for score in ("softmax", "sigmoid"):
        check(x, k, bias, score=score)
        check(x, k, bias, score=score, groups=4, top_groups=2, group_top=1)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_one_lane_holds_all_that_is_chosen(with_bias, dtype):
    # neighbours: the best of a row are 30 experts in a row
    x = randn(40, 1024, seed=2).to(dtype)
    for t in range(40):
        x[t, 25 * t:25 * t + 30] = (8 + randn(30, seed=t)).to(dtype)
    bias = randn(1024, seed=3, scale=0.01) if with_bias else None
    for k in (1, 8, 9, 30, 32):
        check(x, k, bias, score="sigmoid")
        check(x[:, :512], k, bias[:512].contiguous() if with_bias else None, score="softmax")


def test_experts_that_are_not_available():
    for dtype in R.DTYPES:
        x = randn(6, 64, seed=5).to(dtype)
        x[0] = -INF
        x[1, 3:] = -INF
        x[2, :60] = -INF
        x[3, ::2] = -INF
        x[4, 7] = -INF
        for score in ("softmax", "sigmoid"):
            for bias in (None, randn(64, seed=1, scale=0.1)):
                check(x, 8, bias, score=score)
                check(x, 8, bias, score=score, renormalize=False)
                check(x, 8, bias, score=score, groups=8, top_groups=2, group_top=2)
    bias = torch.zeros(64, device="cuda")
    bias[5:] = -INF
    check(randn(9, 64, seed=6), 8, bias, score="sigmoid")
    bias[9] = INF  # always taken, and its score has to be exact all the same
    check(randn(9, 64, seed=6), 4, bias, score="sigmoid")


def test_not_a_number_is_not_chosen():
    x = randn(4, 64, seed=7)
    x[1, 5], x[2] = float("nan"), float("nan")
    w, ids, _ = nrm.route_fwd(x, 6, score="sigmoid")
    assert (ids[1] != 5).all() and (ids[2] == -1).all() and not w[2].any() and (ids[[0, 1, 3]] >= 0).all()
    bias = torch.zeros(64, device="cuda")
    bias[9] = float("nan")
    assert (nrm.route_fwd(x, 6, bias, score="sigmoid")[1] != 9).all()


def test_far_logits_and_large_biases():
    x = randn(50, 128, seed=8, scale=30.0)
    bias = randn(128, seed=9, scale=50.0)
    for score in ("softmax", "sigmoid"):
        check(x, 8, None, score=score)
        check(x, 8, bias, score=score)
        check(x, 8, bias, score=score, groups=4, top_groups=2, group_top=2)
        check(x * 1e5, 8, bias, score=score)
        check(x, 20, bias, score=score, renormalize=False)
    # sigmoids that all round to 0: the weights are 0, not NaN
    w, ids, _ = nrm.route_fwd(x * 0 - 1000.0, 4, bias, score="sigmoid")
    assert not w.any() and (ids >= 0).all()


@pytest.mark.parametrize("experts,k", [(64, 6), (64, 12), (700, 9)])
def test_biases_whose_range_is_beyond_binary32(experts, k):
    x = randn(21, experts, seed=8)
    bias = randn(experts, seed=9, scale=0.1)
    bias[3], bias[5], bias[6] = 3e38, -3e38, 2.9e38
    for score in ("softmax", "sigmoid"):
        check(x, k, bias, score=score)
        check(x, k, bias, score=score, groups=4, top_groups=2, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_saturated_scores(score):
    # sigmoids that binary32 rounds to 1, softmaxes of one expert alone
    x = 20.0 + randn(30, 128, seed=12, scale=3.0)
    x[1::2] += 200.0 * (torch.arange(128, device="cuda") == 77)
    bias = randn(128, seed=13, scale=1e-6)
    check(x, 8, None, score=score)
    check(x, 8, bias, score=score)
    check(x, 20, bias, score=score)
    check(x, 8, bias, score=score, groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("dtype", R.DTYPES)
def test_strides_and_outputs(dtype):
    full = randn(77, 300, seed=10).to(dtype)
    for off, n in ((0, 256), (1, 256), (8, 256), (3, 161)):
        x = full[:, off:off + n]
        w, ids = torch.full((78, 8), 7.0, device="cuda"), torch.full((78, 8), 7, device="cuda")
        out = nrm.route_fwd(x, 8, weights=w[:77], ids=ids[:77])
        want = R.route(x, 8)
        assert out[0].data_ptr() == w.data_ptr() and torch.equal(ids[:77].cpu(), want[1])
        R.check(w[:77].cpu(), want[0], 2 * R.SCORE * want[0], "weights")
        assert (w[77] == 7).all() and (ids[77] == 7).all()
    x = randn(3, 4, 5, 64, seed=1).to(dtype)
    w, ids, sc = nrm.route_fwd(x, 2, want_scores=True)
    assert w.shape == (3, 4, 5, 2) and sc.shape == x.shape
    assert torch.equal(ids.view(60, 2).cpu(), R.route(x.view(60, 64), 2)[1])
    assert nrm.route_fwd(x[:0], 2)[0].shape == (0, 4, 5, 2)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("balance", [False, True])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (5, 7, 3), (203, 64, 6), (99, 160, 6), (64, 256, 8), (9, 1000, 32), (4, 500, 10)])
def test_backward(tokens, experts, k, balance, renorm, score, dtype):
    x = randn(tokens, experts, seed=k, scale=1.5).to(dtype)
    ids = R.route(x, k, score=score)[1].cuda()
    dw = randn(tokens, k, seed=1)
    ds = randn(tokens, experts, seed=2, scale=0.1) if balance else None
    how = dict(score=score, renormalize=renorm, scale=1.7, dscores=ds)
    ref, slack = R.route_grad(dw, x, ids, **how)
    dx = nrm.route_bwd(dw, x, ids, **how)
    R.check(dx, ref, R.out_bound(dtype, ref, slack), "dx")
    assert torch.equal(nrm.route_bwd(dw, x, ids, **how), dx)
    x2 = x.clone()
    assert nrm.route_bwd(dw, x2, ids, out=x2, **how) is x2 and torch.equal(x2, dx)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_of_listed_twice_missing_and_unavailable(score):
    x = randn(6, 64, seed=1)
    x[2, 10:] = -INF
    x[3] = -INF
    ids = R.route(x, 6, score=score)[1].cuda()
    ids[0, 3] = ids[0, 1]
    ids[1] = 9
    ids[4] = torch.tensor([64, -1, -5, 1 << 40, 0, 63])
    dw, ds = randn(6, 6, seed=2), randn(6, 64, seed=3)
    for renorm in (False, True):
        for dscores in (None, ds):
            how = dict(score=score, renormalize=renorm, dscores=dscores)
            ref, slack = R.route_grad(dw, x, ids, **how)
            dx = nrm.route_bwd(dw, x, ids, **how)
            R.check(dx, ref, R.out_bound(torch.float32, ref, slack), "dx")


@pytest.mark.parametrize("dtype", R.DTYPES)
def test_backward_strides(dtype):
    full, out = randn(33, 300, seed=1).to(dtype), torch.full((33, 301), 7.0, device="cuda", dtype=dtype)
    x, o = full[:, 3:164], out[:, 5:166]
    ids, dw = R.route(x, 4)[1].cuda(), randn(33, 4, seed=2)
    ref, slack = R.route_grad(dw, x, ids)
    assert nrm.route_bwd(dw, x, ids, out=o) is o
    R.check(o, ref, R.out_bound(dtype, ref, slack), "dx")
    assert (out[:, :5] == 7).all() and (out[:, 166:] == 7).all()


def test_streams_and_graphs():
    x, bias = randn(500, 256, seed=1).bfloat16(), randn(256, seed=2, scale=0.05)
    how = dict(score="sigmoid", scale=2.5)
    w, ids, _ = nrm.route_fwd(x, 8, bias, groups=8, top_groups=4, group_top=2, **how)
    dx = nrm.route_bwd(w, x, ids, **how)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = nrm.route_fwd(x, 8, bias, groups=8, top_groups=4, group_top=2, stream=side, **how)
    b = nrm.route_bwd(a[0], x, a[1], stream=side, **how)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a[0], w) and torch.equal(a[1], ids) and torch.equal(b, dx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = nrm.route_fwd(x, 8, bias, groups=8, top_groups=4, group_top=2, **how)
        b = nrm.route_bwd(a[0], x, a[1], **how)
    b.fill_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0], w) and torch.equal(a[1], ids) and torch.equal(b, dx)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[1], ids.flip(0)) and torch.equal(b, dx.flip(0))


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("experts,k,groups,top_groups,group_top", [(64, 6, 1, 1, 1), (160, 6, 8, 3, 2), (256, 8, 8, 4, 2), (255, 8, 1, 1, 1),
                                                                   (7, 3, 1, 1, 1), (128, 8, 4, 2, 1)])
def test_the_plans_agree(experts, k, groups, top_groups, group_top, dtype):
    # a warp a token, by force, where eight lanes a token are the rule
    x, bias = randn(500, experts, seed=14).to(dtype), randn(experts, seed=15, scale=0.05)
    for b in (bias, None):
        for score in ("sigmoid", "softmax"):
            how = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top)
            w, ids, _ = nrm.route_fwd(x, k, b, **how)
            assert nrm.last_plan()[4] == 32  # tokens a CTA
            nrm.force_plan(nrm.PLAN_GENERIC)
            try:
                w2, ids2, _ = nrm.route_fwd(x, k, b, **how)
                assert nrm.last_plan()[4] == 8
                check(x, k, b, **how)
            finally:
                nrm.force_plan(nrm.PLAN_AUTO)
            assert torch.equal(ids, ids2) and (w - w2).abs().max() <= 2 * R.SCORE


@pytest.mark.parametrize("k", [8, 20])
def test_weights_to_the_last_bits(k):
    # u = 2^-24.  expf is good to 2 steps (4 u), __fdividef as well, a sum or product to
    # u: a sigmoid to 10 u, renormalised with 5 levels of additions to 10 + 10 + 5 + 4 =
    # 29 u; a renormalised softmax of logits at most 16 below the chosen ones' largest,
    # whose differences are exact here, to 4 + 4 + 5 + 4 = 17 u
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.rand(4000, 64, generator=g, device="cuda") * 160 - 80
    w, ids, _ = nrm.route_fwd(x, k, score="sigmoid", renormalize=False)
    s = torch.sigmoid(x.double()).gather(1, ids)
    assert ((w.double() - s).abs() <= 10 * R.U * s).all()
    x = x.abs().neg()  # scores of all sizes among the chosen
    w, ids, _ = nrm.route_fwd(x, k, score="sigmoid")
    s = torch.sigmoid(x.double()).gather(1, ids)
    s /= s.sum(1, keepdim=True)
    assert ((w.double() - s).abs() <= 29 * R.U * s).all()
    x = torch.randint(0, 16 * 64, (4000, 64), generator=g, device="cuda") / 64.0
    w, ids, _ = nrm.route_fwd(x, k)
    s = torch.softmax(x.double().gather(1, ids), -1)
    assert ((w.double() - s).abs() <= 17 * R.U * s).all()
