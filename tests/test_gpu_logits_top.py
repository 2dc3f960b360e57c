"""Log-probabilities with entropy and top alternatives, forward and backward, on
the GPU against the 64-bit definitions of block_ref.py.  The alternatives have
to be equal, ties included."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

INF = float("inf")


@pytest.fixture(autouse=True, scope="module")
def _built():
    nrm.build()


def make(rows, v, dtype, seed=0, scale=3.0, out=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = scale * torch.randn(rows, v, generator=g, device="cuda")
    t = torch.randint(0, v, (rows,), generator=g, device="cuda")
    z[torch.arange(rows), t] += 6 * torch.rand(rows, generator=g, device="cuda")
    t[torch.rand(rows, generator=g, device="cuda") < out] = -100
    return z.to(dtype), t


def check_fwd(z, t, k, s=1.0, got=None):
    got = nrm.logprob_top_fwd(z, t, k, s) if got is None else got
    ref, bound = R.logprob_top(z, t, k, s)
    got = dict(zip(("logp", "entropy", "ids", "top", "stats"), got))
    wrong = (got["ids"] != ref["ids"]).nonzero()
    assert not len(wrong), (wrong[:5].tolist(), got["ids"][wrong[0, 0]].tolist(), ref["ids"][wrong[0, 0]].tolist())
    for name in ("logp", "entropy", "top", "stats"):
        fin = torch.isfinite(ref[name])
        assert torch.equal(got[name].double()[~fin], ref[name][~fin]), name
        R.check(got[name][fin], ref[name][fin], (bound[name] + R.U * ref[name].abs() + 1e-45)[fin], name)
    return got


def check_bwd(z, t, f, g, h, a, s=1.0, ids=None, in_place=True):
    ids = f["ids"] if ids is None else ids
    args = (t, f["stats"], f["entropy"], ids, s)
    ref, slack = R.logprob_top_grad(z, t, f["stats"], f["entropy"], ids, g, h, a, s)
    dz = nrm.logprob_top_bwd(g, h, a, z, *args)
    R.check(dz, ref, R.out_bound(z.dtype, ref, slack), "dlogits")
    if in_place:
        z2 = z.clone()
        assert nrm.logprob_top_bwd(g, h, a, z2, *args, out=z2) is z2
        assert torch.equal(z2, dz)
    return dz


def randn(*shape, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


# one column, one pack, ragged ends; a warp a row, a CTA, clusters of 2 to 8, many rows
SIZES = [(1, 1), (3, 2), (5, 7), (4, 8), (2, 65), (700, 33), (9, 1000), (400, 1001), (3, 4096), (500, 4096), (310, 2049),
         (2, 8191), (700, 8193), (310, 16384), (1, 40000), (17, 50001), (2, 131072), (40, 70001), (170, 20000)]


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", SIZES)
def test_against_the_definition(rows, v, dtype):
    for k, s in ((5, 1.0), (0, 0.7), (32, 1.0), (1, 1.3)):
        z, t = make(rows, v, dtype, seed=v + k)
        f = check_fwd(z, t, k, s)
        g, h, a = randn(rows), randn(rows, seed=2), randn(rows, k, seed=3)
        check_bwd(z, t, f, g, h, a, s)


@pytest.mark.parametrize("dtype", R.DTYPES)
def test_long_rows(dtype):
    # groups of several segments, and a row past 2^21 packs of a thread's first
    for rows, v in ((2, 600001), (300, 300007), (1, 5000003)):
        z, t = make(rows, v, dtype, seed=rows)
        f = check_fwd(z, t, 20)
        check_bwd(z, t, f, randn(rows), randn(rows, seed=2), randn(rows, 20, seed=3), in_place=False)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", [(3, 900), (400, 2000), (400, 4000), (2, 30000), (330, 9000), (310, 40001), (1, 300000)])
@pytest.mark.parametrize("k", [1, 8, 32])
def test_ties(rows, v, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.zeros(rows, v, device="cuda")
    z[1::8] = torch.finfo(dtype).min  # every logit the same
    z[2::8] = torch.randint(0, 2, (v,), generator=g, device="cuda").float()
    z[3::8] = torch.randint(0, 40, (v,), generator=g, device="cuda").float()
    z[4::8] = -1e4  # masked by one value but for three
    z[4::8, v // 2:v // 2 + 3] = torch.tensor([1.0, 3.0, 2.0], device="cuda")
    z[5::8, ::2] = -0.0  # equal to 0
    z[6::8] = -(torch.arange(v, device="cuda") % 7).float()
    z[7::8, v - 1] = 1.0
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    check_fwd(z.to(dtype), t, k)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", [(2, 3000), (400, 3000), (3, 65536), (320, 65536), (320, 12345), (1, 400000)])
def test_orders_and_periods(rows, v, dtype):
    # rising and falling rows, the largest all in one thread's or one pack's places
    i = torch.arange(v, device="cuda", dtype=torch.float64)
    z = torch.empty(rows, v, device="cuda", dtype=torch.float64)
    for r in range(rows):
        z[r] = (i / v * 20, -i / v * 20, (i % 2048 == 5) * (10 + i / v), (i % 64 < 8) * 5 + (i * 7919 % 1009) / 1009,
                (i // 8 == v // 16) * (9 + i % 8), (i % 1024 < 4) * (3 + (i * 31 % 977) / 97))[r % 6]
    t = torch.full((rows,), v - 1, device="cuda")
    for k in (4, 32):
        check_fwd(z.to(dtype), t, k)


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", [(4, 40), (4, 700), (400, 1200), (6, 20011), (320, 20011), (2, 200000)])
def test_masked_logits(rows, v, dtype):
    z, t = make(rows, v, dtype, seed=3, out=0.0)
    keep = torch.rand(v, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) < 0.05
    masked = torch.where(keep, z, -INF)
    masked[0] = -INF
    masked[1] = -INF
    masked[1, v // 2] = 1.5  # fewer than k are left
    t[1] = v // 2
    masked[torch.arange(2, rows), t[2:]] = z[torch.arange(2, rows), t[2:]]
    f = check_fwd(masked, t, 20)
    assert (f["ids"][0] == -1).all() and f["entropy"][0] == 0 and f["ids"][1, 1:].max() == -1
    dz = check_bwd(masked, t, f, randn(rows), randn(rows, seed=2), randn(rows, 20, seed=3))
    assert not dz[0].any() and not dz[masked == -INF].any()
    low = torch.where(masked == -INF, torch.finfo(dtype).min, masked)  # by the type's lowest value instead
    f = check_fwd(low, t, 20)
    check_bwd(low, t, f, randn(rows), randn(rows, seed=2), randn(rows, 20, seed=3))


@pytest.mark.parametrize("offset", [0.0, 1e4, -1e4])
@pytest.mark.parametrize("rows,v", [(300, 1500), (40, 30000)])
def test_common_offsets(rows, v, offset):
    z, t = make(rows, v, torch.float32, seed=4)
    z = (z * 64).round() / 64 + offset  # exact with the offset
    f = check_fwd(z, t, 8)
    check_bwd(z, t, f, randn(rows), randn(rows, seed=2), randn(rows, 8, seed=3))


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", [(3, 700), (320, 700), (3, 30000), (320, 30000)])
def test_not_a_number_and_infinity(rows, v, dtype):
    z, t = make(rows, v, dtype, seed=5, out=0.0)
    want = R.logprob_top(z, t, 6)[0]["ids"]
    bad = z.clone()
    at = (want[:, 0] + 1) % v  # not one of a row's alternatives, or else the next one is
    bad[torch.arange(rows), at] = float("nan")
    logp, ent, ids, top, _ = nrm.logprob_top_fwd(bad, t, 6)
    assert torch.isnan(logp).all() and torch.isnan(ent).all()
    assert torch.equal(ids, R.logprob_top(torch.where(torch.isnan(bad), -INF, bad), t, 6)[0]["ids"])
    bad = z.clone()
    bad[:, v // 3] = INF
    logp, ent, ids, _, _ = nrm.logprob_top_fwd(bad, t, 6)
    assert (ids[:, 0] == v // 3).all() and torch.isnan(ent).all()
    assert torch.equal(ids, R.logprob_top(bad, t, 6)[0]["ids"])


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v,pad,shift", [(7, 1000, 8, 0), (7, 1000, 3, 1), (400, 1000, 1, 0), (5, 30001, 2, 3), (330, 9000, 5, 1),
                                              (3, 65536, 16, 2)])
def test_strides_and_alignment(rows, v, pad, shift, dtype):
    z0, t = make(rows, v, dtype, seed=6)

    def place(z):
        flat = torch.full((rows * (v + pad) + shift,), 50.0, dtype=dtype, device="cuda")  # larger than any logit
        view = flat[shift:].view(rows, v + pad)[:, :v]
        view.copy_(z)
        return view, flat

    z, _ = place(z0)
    f = check_fwd(z, t, 9)
    want = nrm.logprob_top_fwd(z0, t, 9)
    assert torch.equal(f["ids"], want[2]) and torch.equal(f["stats"][:, 0], want[4][:, 0])
    g, h, a = randn(rows), randn(rows, seed=2), randn(rows, 9, seed=3)
    out, flat = place(z0)
    dz = nrm.logprob_top_bwd(g, h, a, z, t, f["stats"], f["entropy"], f["ids"], out=out)
    ref, slack = R.logprob_top_grad(z0, t, f["stats"], f["entropy"], f["ids"], g, h, a)
    R.check(dz, ref, R.out_bound(dtype, ref, slack), "dlogits")
    assert (flat[:shift] == 50).all() and (flat[shift:].view(rows, v + pad)[:, v:] == 50).all()


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v", [(40, 500), (40, 30003)])
def test_backward_of_any_ids(rows, v, dtype):
    z, t = make(rows, v, dtype, seed=7)
    f = check_fwd(z, t, 8)
    ids = f["ids"].clone()
    ids[:, 3] = ids[:, 0]  # named twice
    ids[::2, 4] = t[::2]   # the target
    ids[1::2, 5] = v
    ids[::3, 6] = -7
    ids[::4, 7] = 0        # the row's ends
    ids[1::4, 7] = v - 1
    ids[5] = v // 2        # one entry eight times
    g, h, a = randn(rows), randn(rows, seed=2), randn(rows, 8, seed=3)
    check_bwd(z, t, f, g, h, a, ids=ids)
    check_bwd(z, t, f, None, None, a, ids=ids)
    # gradients that are missing or 0
    for gg, hh, aa in ((g, None, None), (None, h, None), (g, h, None), (g, None, a), (g * 0, h * 0, a * 0)):
        dz = check_bwd(z, t, f, gg, hh, aa)
    assert not dz.any()
    # the same gradient as the log-probability alone
    one = nrm.logprob_bwd(g, z, t, None, stats=f["stats"])
    two = nrm.logprob_top_bwd(g, None, None, z, t, f["stats"])
    assert (one.float() - two.float()).abs().max() <= 2.0 ** -18 + R.EPS[dtype] * one.float().abs().max()


@pytest.mark.parametrize("k", [32, 20])
def test_ids_of_another_model_with_all_lanes(k):
    # a teacher's ids: 33 names a row
    z, t = make(64, 3001, torch.bfloat16, seed=8, out=0.0)
    f = check_fwd(z, t, 4)
    ids = torch.randint(0, 3001, (64, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    check_bwd(z, t, f, randn(64), randn(64, seed=2), randn(64, k, seed=3), ids=ids)


def test_gradient_against_differences():
    # the chain forward and backward, in binary32: central differences of the forward itself
    z, t = make(4, 50, torch.float32, seed=9, scale=1.0, out=0.0)
    f = nrm.logprob_top_fwd(z, t, 3)
    g, h, a = randn(4), randn(4, seed=2), randn(4, 3, seed=3)
    dz = nrm.logprob_top_bwd(g, h, a, z, t, f[4], f[1], f[2])
    step = 2.0 ** -6
    for j in (0, 7, int(f[2][0, 0]), int(t[0]), 49):
        hi, lo = z.clone(), z.clone()
        hi[:, j] += step
        lo[:, j] -= step

        def loss(x):
            lp = R.logprob_top(x, t, 3)[0]
            top = torch.log_softmax(x.double(), -1).gather(1, f[2])
            return lp["logp"] * g + lp["entropy"] * h + (top * a).sum(1)

        d = (loss(hi) - loss(lo)) / (2 * step)
        # third derivatives of log-softmax and entropy are below 8 in all: h^2 / 6 times the gradients' sum
        assert ((d - dz[:, j]).abs() <= 8 * step ** 2 / 6 * (g.abs() + h.abs() + a.abs().sum(1)) + 1e-6).all()


def test_shapes_outputs_and_empty():
    z, t = make(12, 777, torch.bfloat16, seed=10)
    want = nrm.logprob_top_fwd(z, t, 4)
    got = nrm.logprob_top_fwd(z.view(3, 4, 777), t.view(3, 4), 4)
    assert [tuple(x.shape) for x in got] == [(3, 4), (3, 4), (3, 4, 4), (3, 4, 4), (3, 4, 2)]
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got, want))
    bufs = [torch.empty_like(x) for x in want]
    got = nrm.logprob_top_fwd(z, t, 4, logp=bufs[0], entropy=bufs[1], top_ids=bufs[2], top_logp=bufs[3], stats=bufs[4])
    assert all(a is b and torch.equal(a, c) for a, b, c in zip(got, bufs, want))
    assert nrm.logprob_top_fwd(z[:0], t[:0], 4)[2].shape == (0, 4)
    assert nrm.logprob_top_bwd(want[0][:0], None, None, z[:0], t[:0], want[4][:0]).shape == (0, 777)


def test_streams_and_graphs():
    for rows, v in ((500, 3000), (20, 50000), (400, 20000)):
        z, t = make(rows, v, torch.bfloat16, seed=11)
        g, h, a = randn(rows), randn(rows, seed=2), randn(rows, 5, seed=3)

        def step(**kw):
            f = nrm.logprob_top_fwd(z, t, 5, **kw)
            return (*f, nrm.logprob_top_bwd(g, h, a, z, t, f[4], f[1], f[2], **kw))

        want = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for x in got:
            x.fill_(1)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert nrm.device_fault() == 0


@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,v,shift", [(310, 16385, 0), (310, 16389, 3), (310, 16387, 5), (700, 8193, 0), (3, 65537, 0), (620, 300007, 0)])
@pytest.mark.parametrize("k", [1, 2, 5, 32])
def test_ties_with_the_last_columns(rows, v, shift, k, dtype):
    # most logits are equal, some larger ones as well, and the k-th largest among
    # the columns behind the last whole pack: lower columns of its value come first
    flat = torch.zeros(rows * v + shift, device="cuda", dtype=dtype)
    z = flat[shift:].view(rows, v)
    for r in range(min(rows, 9)):
        z[r, v - 1 - r % 3] = 1.0
        z[r, :k - 1] = 1.0  # k with the one at the end
        z[r, v // 4 + 3::4096] = 1.0
    z[min(rows, 9) - 1, :] = 1.0
    if rows > 9:
        z[9:, 0], z[9:, min(4096, v // 2)], z[9:, v - 1] = 1.0, 1.0, 1.0
    check_fwd(z, torch.zeros(rows, dtype=torch.int64, device="cuda"), k)
