"""Dropout and the residual path (dropout + add + RMSNorm, forward and
backward) on the GPU against the 64-bit definitions of train_ref.py."""
import numpy as np
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

SEED, OFF = 0x1234567890ABCDEF, (5 << 32) + 11


@pytest.fixture(autouse=True)
def _setup():
    nrm.build()
    nrm.force_plan(nrm.PLAN_AUTO)
    yield
    nrm.force_plan(nrm.PLAN_AUTO)


def make(rows, n, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(rows, n, generator=g)).to(dtype).cuda()


def strided(t, pad, fill=7.0):
    """A view of the same values with `pad` columns behind each row, and its buffer."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]], buf


def same_bits(a, b):
    kind = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def check_drop(y, x, mask, p):
    ref = R.drop(R.f64(x), mask, p)
    R.check(y, ref, np.where(mask, R.out_bound(x.dtype, ref, 2 * R.U * np.abs(ref)), 0.0), "dropout")
    dropped = torch.from_numpy(~mask)
    assert not (y.cpu()[dropped] != 0).any()


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 1), (1, 7), (5, 8), (4, 12), (7, 64), (2, 255), (9, 256), (3, 257),
                                    (64, 1024), (33, 1028), (1, 70001), (2, 66000), (1201, 40), (5000, 3)])
def test_dropout(rows, n, dtype):
    x = make(rows, n, dtype, n)
    mask = R.keep(rows, n, 0.3, SEED, OFF)
    y = nrm.dropout_fwd(x, 0.3, SEED, OFF)
    check_drop(y, x, mask, 0.3)
    assert same_bits(nrm.dropout_bwd(x, 0.3, SEED, OFF), y)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("p", [0.0, 2e-6, 1e-5, 0.5, 0.999, 1.0])
def test_dropout_probabilities_and_special_values(p, dtype):
    x = make(16, 512, dtype, 3)
    x[0], x[1], x[2] = float("inf"), float("nan"), float("-inf")
    mask = R.keep(16, 512, p, 42)
    y = nrm.dropout_fwd(x, p, 42).cpu().double().numpy()
    if R.bar_scale(p)[0] == 0:
        assert np.array_equal(y, R.f64(x), equal_nan=True)
    assert not (y[~mask] != 0).any()
    assert np.isposinf(y[0][mask[0]]).all() and np.isnan(y[1][mask[1]]).all() and np.isneginf(y[2][mask[2]]).all()


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("n,pad,shift", [(264, 8, 0), (264, 4, 0), (264, 1, 0), (37, 3, 1), (512, 0, 1), (512, 16, 2)])
def test_dropout_strides_alignment_in_place(n, pad, shift, dtype):
    x0 = make(21, n, dtype, 8)
    flat = torch.full((21 * (n + pad) + shift,), 7.0, dtype=dtype, device="cuda")
    x = flat[shift:].view(21, n + pad)[:, :n]
    x.copy_(x0)
    y = nrm.dropout_fwd(x, 0.25, 5, -1)  # an offset modulo 2^64
    mask = R.keep(21, n, 0.25, 5, -1)
    check_drop(y, x0, mask, 0.25)
    assert nrm.dropout_fwd(x, 0.25, 5, -1, out=x).data_ptr() == x.data_ptr()
    assert same_bits(x, y)
    rest = flat[shift:].view(21, n + pad)[:, n:]
    assert (rest == 7.0).all() and (flat[:shift] == 7.0).all()


def test_dropout_does_not_depend_on_type_or_shape_of_launch():
    masks = []
    for dtype in R.DTYPES:
        for pad in (0, 1):
            x, _ = strided(torch.ones(40, 520, dtype=dtype, device="cuda"), pad)
            masks.append((nrm.dropout_fwd(x, 0.4, 77, 3) != 0).cpu())
    assert all(torch.equal(m, masks[0]) for m in masks)


def test_dropout_counter_on_the_device_in_a_graph():
    x = make(64, 384, torch.bfloat16, 1)
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    y = torch.empty_like(x)
    nrm.dropout_fwd(x, 0.5, 9, 100, out=y, offset_dev=count)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nrm.dropout_fwd(x, 0.5, 9, 100, out=y, offset_dev=count)
        count += 1
    count.fill_(0)
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        check_drop(y, x, R.keep(64, 384, 0.5, 9, 100 + step), 0.5)
    count.fill_(-100)
    g.replay()
    torch.cuda.synchronize()
    check_drop(y, x, R.keep(64, 384, 0.5, 9, 0), 0.5)


def test_empty_calls():
    x = torch.empty(0, 96, device="cuda")
    assert nrm.dropout_fwd(x, 0.1, 1).shape == (0, 96)
    ro, y, rstd = nrm.dropout_add_rms_fwd(x, x, p=0.1)
    assert ro.shape == y.shape == (0, 96) and rstd.shape == (0,)
    dw = torch.full((96,), 5.0, device="cuda")
    dx, dr, got = nrm.dropout_add_rms_bwd(x, x, rstd, torch.ones(96, device="cuda"), 0.1, dw=dw)
    torch.cuda.synchronize()
    assert dx.shape == (0, 96) and (got == 0).all()


# sizes of every register plan and its ragged ends, and beyond them
SIZES = [(1, 1), (5, 7), (3, 40), (700, 96), (700, 257), (650, 513), (610, 1000), (40, 1024), (7, 1030), (33, 2048),
         (10, 2049), (64, 4096), (9, 5001), (5, 8192), (3, 8200), (4, 16384), (3, 16392), (2, 20001), (1300, 264)]


def inputs(rows, n, dtype):
    x, res = make(rows, n, dtype, 1), make(rows, n, dtype, 2, 2.0)
    g = torch.Generator().manual_seed(3)
    return x, res, (1 + 0.1 * torch.randn(n, generator=g)).to(dtype).cuda()


def check_fwd(x, res, w, p, eps, mask, got):
    ro, y, rstd = got
    assert same_bits(ro.cpu(), R.stream(x, res, mask, p))
    ref_y, ref_r = R.norm(R.f64(ro), 1.0 if w is None else R.f64(w), eps)
    R.check(rstd, ref_r, 40 * R.U * ref_r, "rstd")
    R.check(y, ref_y, R.out_bound(x.dtype, ref_y, 44 * R.U * np.abs(ref_y)), "y")


@pytest.mark.parametrize("plan", [nrm.PLAN_AUTO, nrm.PLAN_GENERIC])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,n", SIZES)
def test_forward(rows, n, dtype, plan):
    x, res, w = inputs(rows, n, dtype)
    mask = R.keep(rows, n, 0.2, SEED, OFF)
    nrm.force_plan(plan)
    check_fwd(x, res, w, 0.2, 1e-6, mask, nrm.dropout_add_rms_fwd(x, res, w, 0.2, SEED, OFF, 1e-6))


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("n", [96, 1001, 4096])
def test_forward_without_dropout_is_add_rms(n, dtype):
    x, res, w = inputs(50, n, dtype)
    ro, y, rstd = nrm.dropout_add_rms_fwd(x, res, w, 0.0)
    ro2, y2, rstd2 = nrm.add_rms_fwd(x, res, w, want_stats=True)
    assert same_bits(ro, ro2)
    # two binary32 evaluations of one value, each within 44 u of it, then one rounding each
    R.check(rstd, R.f64(rstd2), 80 * R.U * R.f64(rstd2), "rstd")
    R.check(y, R.f64(y2), (R.EPS[dtype] + 88 * R.U) * np.abs(R.f64(y2)) + R.TINY[dtype], "y")
    check_fwd(x, res, w, 0.0, 1e-6, np.ones((50, n), bool), (ro, y, rstd))


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("pad", [8, 3])
def test_forward_strided_in_place_no_weight(pad, dtype):
    x, res, _ = inputs(30, 520, dtype)
    mask = R.keep(30, 520, 0.6, 1)
    xs, xb = strided(x, pad)
    rs, rb = strided(res, pad)
    ys, yb = strided(torch.zeros_like(x), pad)
    got = nrm.dropout_add_rms_fwd(xs, rs, None, 0.6, 1, residual_out=rs, out=ys)
    assert got[0].data_ptr() == rs.data_ptr()
    check_fwd(x, res, None, 0.6, 1e-6, mask, got)
    for b in (xb, rb, yb):
        assert (b[:, 520:] == 7.0).all()


def check_bwd(dy, h, rstd, w, up, mask, p, got):
    dx, dres, dw = got
    one = 1.0 if w is None else R.f64(w)
    dh, slack, ref_dw, room = R.add_rms_bwd(R.f64(dy), R.f64(h), R.f64(rstd), one, 0.0 if up is None else R.f64(up))
    R.check(dres, dh, R.out_bound(dy.dtype, dh, slack), "dresidual")
    s = R.bar_scale(p)[1]
    ref = R.drop(dh, mask, p)
    R.check(dx, ref, np.where(mask, R.out_bound(dy.dtype, ref, s * slack + 2 * R.U * np.abs(ref)), 0.0), "dx")
    if dw is not None:
        R.check(dw, ref_dw, room, "dw")


@pytest.mark.parametrize("plan", [nrm.PLAN_AUTO, nrm.PLAN_GENERIC])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,n", SIZES + [(2500, 384), (1999, 130), (5, 9001), (40, 12288), (612, 16384), (611, 15999)])
def test_backward(rows, n, dtype, plan):
    _, h, w = inputs(rows, n, dtype)
    dy, up = make(rows, n, dtype, 5), make(rows, n, dtype, 6)
    rstd = 1 / torch.sqrt(h.float().square().mean(-1) + 1e-6)
    nrm.force_plan(plan)
    mask = R.keep(rows, n, 0.2, SEED, OFF)
    got = nrm.dropout_add_rms_bwd(dy, h, rstd, w, 0.2, SEED, OFF, dresidual_out=up)
    check_bwd(dy, h, rstd, w, up, mask, 0.2, got)
    again = nrm.dropout_add_rms_bwd(dy, h, rstd, w, 0.2, SEED, OFF, dresidual_out=up)
    assert all(same_bits(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [2, 610])
def test_every_number_of_256_columns(rows, dtype):
    # each is its own CTA size: whole packs and rows off the 16-byte grid
    for c in range(1, 67):
        if rows > 2 and c > 6 and c not in (32, 33, 48, 49, 64, 65):
            continue
        for n in (256 * c, 256 * c - 7):
            x, res, w = inputs(rows, n, dtype)
            mask = R.keep(rows, n, 0.2, SEED, OFF)
            got = nrm.dropout_add_rms_fwd(x, res, w, 0.2, SEED, OFF, 1e-6)
            check_fwd(x, res, w, 0.2, 1e-6, mask, got)
            check_bwd(x, got[0], got[2], w, res, mask, 0.2,
                      nrm.dropout_add_rms_bwd(x, got[0], got[2], w, 0.2, SEED, OFF, dresidual_out=res))


@pytest.mark.parametrize("plan", [nrm.PLAN_AUTO, nrm.PLAN_GENERIC])
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("n", [264, 1001, 4096])
def test_backward_optional_arguments_and_in_place(n, dtype, plan):
    rows = 37
    _, h, w = inputs(rows, n, dtype)
    dy, up = make(rows, n, dtype, 5), make(rows, n, dtype, 6)
    rstd = 1 / torch.sqrt(h.float().square().mean(-1) + 1e-6)
    nrm.force_plan(plan)
    ones = np.ones((rows, n), bool)
    # no dropout, no weight, no gradient along the stream: the plain RMSNorm backward
    dx, dres, dw = nrm.dropout_add_rms_bwd(dy, h, rstd)
    assert dx is dres and dw is None
    check_bwd(dy, h, rstd, None, None, ones, 0.0, (dx, dres, None))
    dx, dres, dw = nrm.dropout_add_rms_bwd(dy, h, rstd, want_dw=True, dx=torch.empty_like(dy))
    check_bwd(dy, h, rstd, None, None, ones, 0.0, (dx, dres, dw))
    assert nrm.dropout_add_rms_bwd(dy, h, rstd, w, want_dw=False)[2] is None
    # in place on strided buffers
    dys, dyb = strided(dy, 8)
    ups, upb = strided(up, 8)
    got = nrm.dropout_add_rms_bwd(dys, h, rstd, w, 0.35, 4, dresidual_out=ups, dx=dys, dresidual=ups)
    check_bwd(dy, h, rstd, w, up, R.keep(rows, n, 0.35, 4), 0.35, got)
    assert got[0].data_ptr() == dyb.data_ptr() and (dyb[:, n:] == 7.0).all() and (upb[:, n:] == 7.0).all()


def test_backward_workspace_is_scratch_and_graphs_can_share_it():
    rows, n = 300, 1024
    _, h, w = inputs(rows, n, torch.bfloat16)
    rstd = 1 / torch.sqrt(h.float().square().mean(-1) + 1e-6)
    ws = torch.full((nrm.dropout_add_rms_bwd_workspace_size(rows, n, torch.bfloat16),), 255, dtype=torch.uint8, device="cuda")
    dys = [make(rows, n, torch.bfloat16, 20 + i) for i in range(2)]
    want = [nrm.dropout_add_rms_bwd(d, h, rstd, w, 0.1, 7, i) for i, d in enumerate(dys)]
    got, graphs = [], []
    for i, d in enumerate(dys):
        outs = dict(dx=torch.empty_like(d), dresidual=torch.empty_like(d), dw=torch.empty(n, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(nrm.dropout_add_rms_bwd(d, h, rstd, w, 0.1, 7, i, workspace=ws, **outs))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(same_bits(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("plan", [nrm.PLAN_AUTO, nrm.PLAN_GENERIC])
@pytest.mark.parametrize("rows,n", [(1, 5001), (3, 4096), (9, 5001), (9, 1001), (700, 257), (1, 20001), (613, 40)])
def test_backward_stays_inside_its_workspace(rows, n, plan):
    nrm.force_plan(plan)
    for dtype in (torch.float16, torch.float32):
        _, h, w = inputs(rows, n, dtype)
        dy = make(rows, n, dtype, 5)
        rstd = 1 / torch.sqrt(h.float().square().mean(-1) + 1e-6)
        need = nrm.dropout_add_rms_bwd_workspace_size(rows, n, dtype)
        buf = torch.full((need + 16 * 4 * n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        got = nrm.dropout_add_rms_bwd(dy, h, rstd, w, 0.2, SEED, OFF, workspace=buf[:need])
        torch.cuda.synchronize()
        assert (buf[need:] == 0xA5).all()
        check_bwd(dy, h, rstd, w, None, R.keep(rows, n, 0.2, SEED, OFF), 0.2, got)


@pytest.mark.parametrize("rows,n", [(66001, 65536), (140000, 30727)])
def test_more_than_2_to_the_32_elements(rows, n):
    # row offsets beyond 32 bits, aligned and not; the last rows against the definition
    x = torch.ones(rows, n, dtype=torch.bfloat16, device="cuda")
    y = nrm.dropout_fwd(x, 0.25, SEED, OFF)
    del x
    last = R.keep(rows, 64, 0.25, SEED, OFF)[-3:]
    got = y[-3:, :64].float().cpu().numpy()
    assert np.array_equal(got != 0, last) and (got[last] == np.float32(1.3359375)).all()
    first = R.keep(2, n, 0.25, SEED, OFF)
    assert np.array_equal(y[:2].float().cpu().numpy() != 0, first)


def test_side_stream():
    x, res, w = inputs(64, 1024, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        got = nrm.dropout_add_rms_fwd(x, res, w, 0.2, SEED, OFF, stream=handle)
        bwd = nrm.dropout_add_rms_bwd(x, got[0], got[2], w, 0.2, SEED, OFF, stream=handle)
        side.synchronize()
        mask = R.keep(64, 1024, 0.2, SEED, OFF)
        check_fwd(x, res, w, 0.2, 1e-6, mask, got)
        check_bwd(x, got[0], got[2], w, None, mask, 0.2, bwd)


def test_refused_tensors():
    x, res, w = inputs(8, 64, torch.float16)
    f = torch.zeros(8, device="cuda")
    for call in (lambda: nrm.dropout_fwd(x.t(), 0.1, 0), lambda: nrm.dropout_fwd(x, 0.1, 0, out=x.float()),
                 lambda: nrm.dropout_fwd(x, 0.1, 0, offset_dev=f), lambda: nrm.dropout_add_rms_fwd(x, res[:4], w),
                 lambda: nrm.dropout_add_rms_fwd(x, res, w.float()), lambda: nrm.dropout_add_rms_fwd(x, res, w, rstd=f[:4]),
                 lambda: nrm.dropout_add_rms_bwd(x, res, f[:4]), lambda: nrm.dropout_add_rms_bwd(x, res, f, dw=f),
                 lambda: nrm.dropout_add_rms_bwd(x, res, f.half())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nrm.dropout_fwd(x.double(), 0.1, 0)
    for call, status in ((lambda: nrm.dropout_fwd(x, 1.5, 0), 5), (lambda: nrm.dropout_add_rms_fwd(x, res, w, out=x), 4),
                         (lambda: nrm.dropout_add_rms_bwd(x, res, f, dresidual=x), 4),
                         (lambda: nrm.dropout_add_rms_bwd(x, res, f, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), 7)):
        with pytest.raises(nrm.NrmError) as e:
            call()
        assert e.value.status == status
