"""Head norms with the position rotation, forward and backward, on the GPU
against the 64-bit definition of block_ref.py."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

MOST = 4096  # positions of the table


@pytest.fixture(autouse=True, scope="module")
def _built():
    nrm.build()


def randn(*shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def make(tokens, hq, hk, d, rot, dtype, seed, pad=0.2, most=MOST):
    """q and k as slices of one projection, weights, table, positions (some outside the table)."""
    qkv = randn(tokens, hq + 2 * hk, d, seed=seed, dtype=dtype, scale=2.0)
    wq, wk = ((1 + randn(d, seed=seed + i, scale=0.2)).to(dtype) for i in (1, 2))
    g = torch.Generator(device="cuda").manual_seed(seed)
    pos = torch.randint(0, most, (tokens,), generator=g, device="cuda")
    out = torch.rand(tokens, generator=g, device="cuda") < pad
    pos[out] = torch.where(torch.arange(tokens, device="cuda") % 2 == 0, -1, most)[out]
    return qkv[:, :hq], qkv[:, hq:hq + hk], wq, wk, R.angle_table(most, rot, device="cuda"), pos


def check_fwd(got, x, w, table, pos, near, eps=1e-6):
    ref, slack = R.head_norm(x, w, table, pos, eps, near)
    R.check(got, ref, R.out_bound(got.dtype, ref, slack), "out")
    dead = ~R.live_tokens(table, pos)
    assert not got[dead].any()


def check_bwd(dx, dw, dout, x, w, table, pos, near, eps=1e-6):
    ref, slack, dw_ref, dw_slack = R.head_norm_bwd(dout, x, w, table, pos, eps, near)
    R.check(dx, ref, R.out_bound(dx.dtype, ref, slack), "dx")
    R.check(dw, dw_ref, dw_slack, "dw")
    assert not dx[~R.live_tokens(table, pos)].any()


SHAPES = [  # tokens, query heads, key heads, D, rotated: every access width and number of slots
    (1, 1, 1, 128, 128), (3, 5, 1, 64, 64), (17, 32, 8, 128, 128), (5, 12, 12, 80, 40), (9, 7, 1, 72, 72),
    (6, 4, 2, 50, 50), (6, 4, 2, 50, 24), (33, 3, 3, 96, 16), (4, 2, 1, 256, 256), (3, 2, 2, 512, 512),
    (3, 2, 2, 500, 100), (2, 3, 1, 511, 510), (7, 1, 1, 1, 0), (7, 2, 1, 2, 2), (5, 2, 1, 7, 4), (5, 2, 1, 64, 0),
    (257, 9, 3, 112, 56), (4, 1, 2, 192, 190), (3, 2, 1, 260, 4), (2, 2, 2, 130, 130),
]


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("tokens,hq,hk,d,rot", SHAPES)
def test_against_the_definition(tokens, hq, hk, d, rot, dtype, near):
    q, k, wq, wk, table, pos = make(tokens, hq, hk, d, rot, dtype, d + tokens)
    yq, yk = nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk, interleaved=near)
    check_fwd(yq, q, wq, table, pos, near)
    check_fwd(yk, k, wk, table, pos, near)
    gq, gk = randn(tokens, hq, d, seed=1, dtype=dtype), randn(tokens, hk, d, seed=2, dtype=dtype)
    dq, dk, dwq, dwk = nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, wq, wk, interleaved=near)
    check_bwd(dq, dwq, gq, q, wq, table, pos, near)
    check_bwd(dk, dwk, gk, k, wk, table, pos, near)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("tokens,hq,hk,d,rot", [(8000, 6, 2, 64, 64), (3001, 4, 4, 80, 80)])
def test_many_tokens(tokens, hq, hk, d, rot, dtype):
    q, k, wq, wk, table, pos = make(tokens, hq, hk, d, rot, dtype, 5)
    yq, yk = nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk)
    check_fwd(yq, q, wq, table, pos, False)
    check_fwd(yk, k, wk, table, pos, False)
    gq, gk = randn(tokens, hq, d, seed=1, dtype=dtype), randn(tokens, hk, d, seed=2, dtype=dtype)
    first = nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, wq, wk)
    check_bwd(first[0], first[2], gq, q, wq, table, pos, False)
    check_bwd(first[1], first[3], gk, k, wk, table, pos, False)
    for a, b in zip(first, nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, wq, wk)):
        assert torch.equal(a, b)  # the same bits every time


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("layout", ["heads first", "shifted", "padded heads", "four dimensions"])
def test_layouts(layout, dtype):
    tokens, hq, hk, d, near = 12, 6, 2, 64, False
    q, k, wq, wk, table, pos = make(tokens, hq, hk, d, d, dtype, 3)
    want = nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk)
    gq, gk = randn(tokens, hq, d, seed=1, dtype=dtype), randn(tokens, hk, d, seed=2, dtype=dtype)
    grads = nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, wq, wk)
    if layout == "four dimensions":
        view = lambda t: t.view(3, 4, *t.shape[1:])  # noqa: E731
        yq, yk = nrm.qk_norm_rope_fwd(view(q), view(k), table, pos.view(3, 4), wq, wk)
        assert torch.equal(yq, view(want[0])) and torch.equal(yk, view(want[1]))
        got = nrm.qk_norm_rope_bwd(view(gq), view(gk), view(q), view(k), table, pos.view(3, 4), wq, wk)
        assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got[:2], grads[:2]))
        return

    def lay(t):
        if layout == "heads first":
            return t.transpose(0, 1).contiguous().transpose(0, 1)
        if layout == "shifted":  # one element off every boundary
            flat = torch.full((t.numel() + 1,), 7.0, dtype=t.dtype, device="cuda")
            out = flat[1:].view(t.shape)
        else:
            out = torch.full((*t.shape[:2], d + 4), 7.0, dtype=t.dtype, device="cuda")[..., :d]
        return out.copy_(t)

    oq, ok = lay(torch.zeros_like(q)), lay(torch.zeros_like(k))
    yq, yk = nrm.qk_norm_rope_fwd(lay(q), lay(k), table, pos, wq, wk, q_out=oq, k_out=ok)
    assert yq is oq and yk is ok
    check_fwd(yq, q, wq, table, pos, near)
    check_fwd(yk, k, wk, table, pos, near)
    dq, dk, dwq, dwk = nrm.qk_norm_rope_bwd(lay(gq), lay(gk), lay(q), lay(k), table, pos, wq, wk, dq=oq, dk=ok)
    check_bwd(dq, dwq, gq, q, wq, table, pos, near)
    check_bwd(dk, dwk, gk, k, wk, table, pos, near)
    if layout == "padded heads":
        assert (oq._base[..., d:] == 7.0).all()


def test_in_place_in_one_projection():
    dtype, tokens, hq, hk, d = torch.bfloat16, 37, 8, 2, 128
    q, k, wq, wk, table, pos = make(tokens, hq, hk, d, d, dtype, 4)
    rest = q._base[:, hq + hk:].clone()
    want = nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk)
    q0, k0 = q.clone(), k.clone()
    got = nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(q._base[:, hq + hk:], rest)
    gq, gk = randn(tokens, hq, d, seed=1, dtype=dtype), randn(tokens, hk, d, seed=2, dtype=dtype)
    want = nrm.qk_norm_rope_bwd(gq, gk, q0, k0, table, pos, wq, wk)
    a, b = q0.clone(), k0.clone()
    got = nrm.qk_norm_rope_bwd(gq, gk, a, b, table, pos, wq, wk, dq=a, dk=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    got = nrm.qk_norm_rope_bwd(gq, gk, q0, k0, table, pos, wq, wk, dq=gq, dk=gk)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_without_weights_keys_or_table_rows():
    q, k, wq, wk, table, pos = make(20, 4, 2, 64, 64, torch.float32, 6)
    yq, none = nrm.qk_norm_rope_fwd(q, None, table, pos)
    assert none is None
    check_fwd(yq, q, None, table, pos, False)
    g = randn(20, 4, 64, seed=1)
    dq, dk, dwq, dwk = nrm.qk_norm_rope_bwd(g, None, q, None, table, pos)
    assert dk is None and dwq is None and dwk is None
    dq2, _, dwq, _ = nrm.qk_norm_rope_bwd(g, None, q, None, table, pos, want_dw=True)
    check_bwd(dq2, dwq, g, q, None, table, pos, False)
    assert torch.equal(dq, dq2)
    # a table of no positions: no token takes part, weights get zeros
    dq, dk, dwq, dwk = nrm.qk_norm_rope_bwd(g, g[:, :2], q, k, table[:0], pos, wq, wk)
    assert not any(t.any() for t in (dq, dk, dwq, dwk))
    # no tokens
    dq, dk, dwq, dwk = nrm.qk_norm_rope_bwd(g[:0], g[:0, :2], q[:0], k[:0], table, pos[:0], wq, wk)
    assert dq.shape == (0, 4, 64) and not dwq.any() and not dwk.any()
    assert nrm.qk_norm_rope_fwd(q[:0], k[:0], table, pos[:0], wq, wk)[1].shape == (0, 2, 64)


def test_values_of_tokens_outside_the_table_do_not_count():
    q, k, wq, wk, table, pos = make(40, 4, 2, 64, 64, torch.float16, 7, pad=0.5)
    q, k, dead = q.clone(), k.clone(), ~R.live_tokens(table, pos)
    q[dead], k[dead] = float("nan"), float("inf")
    g = randn(40, 4, 64, seed=1, dtype=torch.float16)
    g[dead] = float("nan")
    yq, yk = nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk)
    assert torch.isfinite(yq).all() and torch.isfinite(yk).all() and not yq[dead].any()
    out = nrm.qk_norm_rope_bwd(g, g[:, :2].contiguous(), q, k, table, pos, wq, wk)
    assert all(torch.isfinite(t).all() for t in out)


def test_far_positions_of_a_long_table():
    # the last row's offset passes 2^31 elements
    rot, most = 512, (1 << 22) + 5
    table = torch.zeros(most, rot, device="cuda")
    table[-1] = R.angle_table(1000, rot, device="cuda")[999]
    pos = torch.tensor([most - 1, most, 3], device="cuda")
    q = randn(3, 2, rot, seed=1)
    yq, _ = nrm.qk_norm_rope_fwd(q, None, table, pos)
    ref, slack = R.head_norm(q[:1], None, table[-1:], pos[:1] * 0, 1e-6, False)
    R.check(yq[:1], ref, R.out_bound(torch.float32, ref, slack), "far")
    assert not yq[1].any() and not yq[2].any()  # cosines and sines of 0 there


def test_streams_graphs_and_shared_workspace():
    q, k, wq, wk, table, pos = make(300, 8, 2, 128, 128, torch.bfloat16, 8)
    gq, gk = randn(300, 8, 128, seed=1, dtype=q.dtype), randn(300, 2, 128, seed=2, dtype=q.dtype)
    want = (*nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk), *nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, wq, wk))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk, stream=side),
           *nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, wq, wk, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(nrm.qk_norm_rope_bwd_workspace_size(300, 8, 2, 128), dtype=torch.uint8, device="cuda")
    outs = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs += nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk)
        outs += nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, wq, wk, workspace=ws)
        outs += nrm.qk_norm_rope_bwd(gk, gk, k, k, table, pos, wk, wk, workspace=ws)  # the same scratch again
    for t in outs:
        t.fill_(3.0)
    ws.fill_(255)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    again = nrm.qk_norm_rope_bwd(gk, gk, k, k, table, pos, wk, wk)
    assert all(torch.equal(a, b) for a, b in zip(outs[6:], again))


def test_empty_batches_of_several_dimensions():
    q, k, wq, wk, table, pos = make(6, 4, 2, 64, 64, torch.bfloat16, 6)
    for lead in ((2, 0), (0, 2), (0, 0, 3), (3, 2, 0)):
        def none(heads, inner=64):
            return torch.empty(*lead, heads, inner, dtype=torch.bfloat16, device="cuda")
        p = torch.empty(lead, dtype=torch.int64, device="cuda")
        yq, yk = nrm.qk_norm_rope_fwd(none(4), none(2), table, p, wq, wk, q_out=none(4))
        assert yq.shape == (*lead, 4, 64) and yk.shape == (*lead, 2, 64)
        sliced = none(8)
        dq, dk, dwq, dwk = nrm.qk_norm_rope_bwd(none(4), none(2), sliced[..., :4, :], sliced[..., 4:6, :], table, p, wq, wk)
        assert dq.shape == (*lead, 4, 64) and dk.shape == (*lead, 2, 64) and not dwq.any() and not dwk.any()


def test_gradient_of_the_keys_is_asked_for():
    q, k, wq, wk, table, pos = make(6, 4, 2, 64, 64, torch.float32, 6)
    with pytest.raises(ValueError, match="dk_out"):
        nrm.qk_norm_rope_bwd(q, None, q, k, table, pos, wq, wk)
    with pytest.raises(ValueError, match="dq_out"):
        nrm.qk_norm_rope_bwd(None, k, q, k, table, pos, wq, wk)
