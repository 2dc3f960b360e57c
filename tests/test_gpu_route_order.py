"""Which experts routing takes where the choice is delicate, on the GPU against
the 64-bit definition of block_ref.py, by both plans (eight lanes a token, and
by force a warp a token)."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

INF = float("inf")


@pytest.fixture(autouse=True, scope="module")
def _built():
    nrm.build()


@pytest.fixture(params=["auto", "a warp a token"], autouse=True)
def plan(request):
    nrm.force_plan(nrm.PLAN_AUTO if request.param == "auto" else nrm.PLAN_GENERIC)
    yield
    nrm.force_plan(nrm.PLAN_AUTO)


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return scale * torch.randn(*shape, generator=g, device="cuda")


def rand(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(*shape, generator=g, device="cuda")


def check(x, k, bias=None, **how):
    """ids equal; weights of scores within 2^-17 each (block_ref.py: SCORE), which
    their sum is as well."""
    want, ids = R.route(x, k, bias, **how)
    w, got, _ = nrm.route_fwd(x, k, bias, **how)
    wrong = (got.cpu() != ids).any(1).nonzero()[:, 0]
    assert not len(wrong), (len(wrong), int(wrong[0]), got[wrong[0]].tolist(), ids[wrong[0]].tolist())
    R.check(w.cpu(), want, 2 * R.SCORE * want.abs() + 2.0 ** -126, "weights")


# experts, k, groups, top_groups
GROUPED = [(64, 12, 4, 1), (64, 8, 4, 2), (160, 6, 8, 3), (256, 8, 8, 4), (256, 8, 8, 2), (512, 10, 4, 2), (1024, 32, 32, 7),
           (96, 3, 12, 5), (32, 4, 32, 6), (756, 20, 12, 2), (768, 8, 3, 1), (255, 8, 3, 2), (24, 6, 8, 4)]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("experts,k,groups,top_groups", GROUPED)
@pytest.mark.parametrize("score,with_bias,group_top", [("softmax", False, 1), ("sigmoid", False, 1), ("softmax", False, 2),
                                                       ("sigmoid", False, 2), ("softmax", True, 1), ("sigmoid", True, 1)])
def test_kept_groups_with_fewer_experts_than_places(experts, k, groups, top_groups, score, with_bias, group_top, dtype):
    # from no available expert a token to a third of them: what the kept groups
    # have not is nobody's place
    x = randn(300, experts, seed=experts + k, scale=1.5).to(dtype)
    x[rand(300, experts, seed=1) > torch.arange(300, device="cuda")[:, None] / 900] = -INF
    bias = None
    if with_bias:
        bias = randn(experts, seed=3, scale=0.05)
        bias[rand(experts, seed=4) < 0.2] = -INF
    check(x, k, bias, score=score, groups=groups, top_groups=top_groups, group_top=group_top)


def test_kept_groups_with_fewer_experts_than_places_by_hand():
    # four groups of 128, two kept, eight available in them, ten places
    x = torch.full((1, 512), -INF, device="cuda")
    for e, v in ((0, 8.0), (1, 8.5), (2, 9.0), (3, 9.5), (128, 8.25), (129, 8.75), (130, 9.25), (131, 9.75), (256, 1.0), (257, 1.5),
                 (358, 2.0), (359, 1.75)):
        x[0, e] = v
    for dtype in R.DTYPES:
        ids = nrm.route_fwd(x.to(dtype), 10, groups=4, top_groups=2)[1]
        assert ids[0].tolist() == [131, 3, 130, 2, 129, 1, 128, 0, -1, -1]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("experts,k,groups,top_groups", GROUPED)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("least", [-0.5, -40.0, 0.75, 1000.0])
def test_groups_of_one_available_expert(experts, k, groups, top_groups, score, least, dtype):
    # the sum of a group's two best counts the one it has, whatever the biases' range
    x = randn(300, experts, seed=experts + k, scale=1.5).to(dtype)
    x[rand(300, experts, seed=1) > 0.2 + 1.5 * groups / experts] = -INF
    bias = (least + rand(experts, seed=5) * (1.5 if abs(least) < 1 else 0.3)).double().float()
    check(x, k, bias, score=score, groups=groups, top_groups=top_groups, group_top=2)
    bias[rand(experts, seed=4) < 0.3] = -INF
    check(x, k, bias, score=score, groups=groups, top_groups=top_groups, group_top=2)


def test_groups_of_one_available_expert_by_hand():
    # a sigmoid of 0 is 1/2: one expert of 1.25 against two of 0.5 each, biases from -0.5 on
    x = torch.zeros(1, 64, device="cuda")
    x[0, 1:4] = x[0, 6:] = -INF
    bias = torch.full((64,), -0.5, device="cuda")
    bias[0], bias[4], bias[5] = 0.75, 0.0, 0.0
    assert nrm.route_fwd(x, 2, bias, score="sigmoid", groups=16, top_groups=1, group_top=2)[1].tolist() == [[0, -1]]
    # biases of 1 and more: two of 1.75 each are more than one of 3
    bias = torch.ones(64, device="cuda")
    bias[0], bias[4], bias[5] = 2.5, 1.25, 1.25
    assert nrm.route_fwd(x, 2, bias, score="sigmoid", groups=16, top_groups=1, group_top=2)[1].tolist() == [[4, 5]]


def step_up(x, steps):
    return (x.view(torch.int32) + steps).view(torch.float32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts,k", [(64, 2), (64, 6), (256, 8), (512, 10), (128, 20)])
def test_equal_ones_left_out_beside_a_smaller_one_taken(experts, k, with_bias, score):
    # some logits a step apart, most of them equal to another, the rest far below:
    # which of them come first is a matter of their last bits
    tokens = 400
    x = randn(tokens, experts, seed=1, scale=0.1) - 4.0
    x = torch.where(rand(tokens, experts, seed=2) < 1.6 * k / experts,
                    step_up(torch.ones(tokens, experts, device="cuda"), (rand(tokens, experts, seed=3) * 3).int()), x)
    bias = torch.zeros(experts, device="cuda") if with_bias else None
    check(x, k, bias, score=score)
    check(x, k, bias, score=score, groups=4, top_groups=2, group_top=1)


@pytest.mark.parametrize("dtype", R.DTYPES)
def test_equal_ones_left_out_by_hand(dtype):
    x = torch.zeros(2, 64, device="cuda", dtype=dtype)
    x[0, 0], x[0, 1], x[0, 2] = 16.0, 16.125, 16.125  # one step of the fixed point for all three
    x[1, 7], x[1, 3], x[1, 60] = 16.125, 16.0, 16.125
    bias = torch.zeros(64, device="cuda")
    assert nrm.route_fwd(x, 2, bias, score="sigmoid")[1].tolist() == [[1, 2], [7, 60]]
    if dtype is torch.float32:
        x = torch.full((1, 64), -3.0, device="cuda")
        x[0, 3], x[0, 7], x[0, 20] = 1.0, 1.0 + 2.0 ** -23, 1.0 + 2.0 ** -23
        for score in ("softmax", "sigmoid"):
            for b in (None, bias):
                assert nrm.route_fwd(x, 2, b, score=score)[1].tolist() == [[7, 20]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_whose_sum_is_beyond_binary32(score):
    x = randn(20, 64, seed=6)
    bias = 1.8e38 + 1.2e38 * rand(64, seed=7)
    check(x, 6, bias, score=score, groups=8, top_groups=3, group_top=2)
    check(x, 6, -bias, score=score, groups=8, top_groups=3, group_top=2)
    x[:, ::3] = -INF
    bias[5] = -3e38
    check(x, 6, bias, score=score, groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("experts,k,groups,top_groups,group_top", [(64, 6, 1, 1, 1), (64, 6, 8, 2, 1), (64, 6, 8, 2, 2), (256, 8, 1, 1, 1),
                                                                   (500, 20, 1, 1, 1), (7, 2, 1, 1, 1)])
def test_softmax_without_a_value(experts, k, groups, top_groups, group_top, dtype):
    # a NaN or an infinity among a token's logits leaves no softmax, so no expert is
    # available; the tokens beside it have theirs
    x = randn(40, experts, seed=8).to(dtype)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[1::3] = True
    x[1::6, experts // 2] = float("nan")
    x[4::12, experts - 1] = INF
    x[10::12, 0] = -float("nan")
    x[7, :] = float("nan")
    how = dict(groups=groups, top_groups=top_groups, group_top=group_top)
    want, ids = R.route(torch.where(bad[:, None], -INF, x), k, **how)
    for bias in (None, torch.zeros(experts, device="cuda")):
        for renorm in (True, False):
            w, got, _ = nrm.route_fwd(x, k, bias, renormalize=renorm, **how)
            assert torch.equal(got.cpu(), ids) and (got[bad] == -1).all() and not w[bad].any()
            assert torch.isfinite(w).all()
    # a sigmoid is each expert's own: a NaN is not available, an infinity is 1
    got = nrm.route_fwd(x, k, score="sigmoid", **how)[1].cpu()
    assert torch.equal(got, R.route(x, k, score="sigmoid", **how)[1])
