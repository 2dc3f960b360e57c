"""The training operators without a GPU: the tests' own definitions (the
generator against its published vectors, the gradients against differences),
and the refusals of the library (no call here reaches a launch on a machine
without a device; the pointers are never dereferenced)."""
import numpy as np
import pytest

import train_ref as R

OK, NULL, SHAPE, DTYPE, ALIAS, VALUE, UNSUP, WS, DEVICE = range(9)
A = 0x100000


@pytest.fixture(scope="module")
def lib():
    import os

    import row_wise_normalization_reduce_gb300 as nrm
    if not os.path.exists(nrm.LIB_PATH):
        nrm.build()
    return nrm.lib()


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_published_vectors(ctr, key, want):
    assert tuple(int(v) for v in R.philox(np.array(ctr, np.uint64), key)) == want


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.1, 0.5, 0.9, 1.0])
def test_mask_rate_and_scale(p):
    k = R.keep(200, 1000, p, 12345, 3)
    t, scale = R.bar_scale(p)
    q = 1 - t / 65536
    # 200000 Bernoulli draws: six standard deviations
    assert abs(k.mean() - q) <= 6 * np.sqrt(q * (1 - q) / k.size) + 1e-12
    assert q == 0 or abs(scale * q - 1) < 1e-15
    assert (R.keep(200, 1000, p, 12345, 4) != k).any() or p in (0.0, 1e-6, 1.0)


def test_residual_backward_against_differences():
    rng = np.random.default_rng(0)
    rows, n, eps = 3, 7, 1e-3
    x, res, w = rng.normal(size=(rows, n)), rng.normal(size=(rows, n)), rng.normal(size=n)
    dy, up = rng.normal(size=(rows, n)), rng.normal(size=(rows, n))
    mask = R.keep(rows, n, 0.4, 9)

    def f(x, res, w):
        h = res + R.drop(x, mask, 0.4)
        return np.sum(R.norm(h, w, eps)[0] * dy) + np.sum(h * up)

    h = res + R.drop(x, mask, 0.4)
    dh, _, dw, _ = R.add_rms_bwd(dy, h, R.norm(h, w, eps)[1], w, up)
    step = 1e-5
    for which, grad in ((0, R.drop(dh, mask, 0.4)), (1, dh), (2, dw)):
        args = [x, res, w]
        for i in np.ndindex(args[which].shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[which][i] += step
            lo[which][i] -= step
            assert abs((f(*hi) - f(*lo)) / (2 * step) - grad[i]) < 1e-7


@pytest.mark.parametrize("s", [1.0, 0.7])
def test_policy_gradient_against_differences(s):
    rng = np.random.default_rng(1)
    rows, v = 9, 6
    z = rng.normal(size=(rows, v)) * 2
    t = rng.integers(0, v, rows)
    t[3] = -100
    logp, lse, _ = R.logprob(z, t, s)
    old = logp + np.array([-0.5, -0.1, 0.0, 0.1, 0.5, -0.5, -0.1, 0.1, 0.5])
    ref, adv = logp + rng.normal(size=rows) * 0.4, np.array([1, 1, 1, 1, 1, -1, -1, -1, -1.0])
    wt = rng.uniform(0.5, 1, rows)
    wt[6] = 0

    def loss(z):
        return R.policy(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1, s)[0]

    slope = R.policy(z, t, old, adv, wt, ref, 0.2, 0.3, 0.1, s)[2]
    dz, _ = R.grad(z, t, lse, slope, s)
    assert not dz[3].any() and not dz[6].any() and dz[0].any()
    for i in np.ndindex(z.shape):
        hi, lo = z.copy(), z.copy()
        hi[i] += 1e-5
        lo[i] -= 1e-5
        assert abs((loss(hi) - loss(lo)) / 2e-5 - dz[i]) < 1e-7


def _bad(lib, name, good, cases):
    f = getattr(lib, name)
    keys = list(good)
    for change, want in cases:
        assert set(change) <= set(keys), change
        st = f(*[dict(good, **change)[k] for k in keys])
        assert st in (want if isinstance(want, tuple) else (want,)), (name, change, st, want)


def test_dropout_refusals(lib):
    good = dict(x=A, ldx=8, y=2 * A, ldy=8, rows=4, N=8, p=0.1, seed=1, offset=0, off_dev=None, dtype=2, stream=None)
    _bad(lib, "dropout_fwd_ld", good, [
        (dict(), (OK, DEVICE)), (dict(y=A), (OK, DEVICE)), (dict(off_dev=3 * A), (OK, DEVICE)),
        (dict(x=None), NULL), (dict(y=None), NULL), (dict(rows=0, x=None, y=None), OK),
        (dict(rows=-1), SHAPE), (dict(N=0), SHAPE), (dict(ldx=7), SHAPE), (dict(ldy=7), SHAPE),
        (dict(rows=2 ** 32 + 1), SHAPE), (dict(N=2 ** 35 + 8, ldx=2 ** 36, ldy=2 ** 36), SHAPE),
        (dict(dtype=3), DTYPE), (dict(p=-0.1), VALUE), (dict(p=1.1), VALUE), (dict(p=float("nan")), VALUE),
        (dict(x=A + 1), VALUE), (dict(off_dev=A + 4), VALUE),
        (dict(y=A + 16), ALIAS), (dict(y=A, ldy=16), ALIAS), (dict(off_dev=2 * A + 8), ALIAS),
    ])


def test_dropout_add_rms_fwd_refusals(lib):
    good = dict(x=A, ldx=8, res=2 * A, ldr=8, w=3 * A, ro=4 * A, ldro=8, y=5 * A, ldy=8, rstd=6 * A, rows=4, N=8,
                p=0.1, seed=1, offset=0, off_dev=None, eps=1e-6, dtype=0, stream=None)
    _bad(lib, "dropout_add_rms_fwd_ld", good, [
        (dict(), (OK, DEVICE)), (dict(ro=2 * A), (OK, DEVICE)), (dict(w=None, rstd=None), (OK, DEVICE)),
        (dict(x=None), NULL), (dict(res=None), NULL), (dict(ro=None), NULL), (dict(y=None), NULL),
        (dict(rows=0, x=None), OK), (dict(rows=-1), SHAPE), (dict(N=0), SHAPE), (dict(ldro=7), SHAPE),
        (dict(eps=-1.0), VALUE), (dict(p=2.0), VALUE), (dict(dtype=9), DTYPE), (dict(rstd=6 * A + 2), VALUE),
        (dict(ro=A), ALIAS), (dict(y=A), ALIAS), (dict(y=2 * A), ALIAS), (dict(ro=2 * A, y=2 * A), ALIAS),
        (dict(ro=2 * A, ldro=12), ALIAS), (dict(rstd=3 * A), ALIAS), (dict(rstd=4 * A), ALIAS),
    ])


def test_dropout_add_rms_bwd_refusals(lib):
    rows, n = 4, 8
    need = lib.dropout_add_rms_bwd_workspace_size(rows, n, 0)
    assert need == rows * n * 4 + 16
    assert lib.dropout_add_rms_bwd_workspace_size(0, n, 0) == 0
    assert lib.dropout_add_rms_bwd_workspace_size(rows, n, 5) == 0
    assert lib.dropout_add_rms_bwd_workspace_size(10 ** 6, 5001, 2) == 608 * 5001 * 4 + 4 * 10 ** 6
    good = dict(dy=A, lddy=n, h=2 * A, ldh=n, rstd=3 * A, w=4 * A, up=5 * A, ldu=n, dx=6 * A, lddx=n, dr=7 * A,
                lddr=n, dw=8 * A, rows=rows, N=n, p=0.1, seed=1, offset=0, off_dev=None, dtype=0, ws=9 * A, wsb=need,
                stream=None)
    _bad(lib, "dropout_add_rms_bwd_ld", good, [
        (dict(), (OK, DEVICE)), (dict(dx=A), (OK, DEVICE)), (dict(dr=5 * A), (OK, DEVICE)),
        (dict(dx=None, dw=None, up=None, w=None, ldu=0, lddx=0), (OK, DEVICE)),
        (dict(dy=None), NULL), (dict(h=None), NULL), (dict(rstd=None), NULL), (dict(dx=None, dr=None, dw=None), NULL),
        (dict(rows=0, dy=None, dw=None, ws=None), OK), (dict(rows=-1), SHAPE), (dict(ldh=7), SHAPE),
        (dict(ldu=7), SHAPE), (dict(lddx=7), SHAPE), (dict(lddr=7), SHAPE), (dict(dtype=4), DTYPE),
        (dict(p=-1.0), VALUE), (dict(dw=8 * A + 2), VALUE), (dict(ws=None), WS), (dict(wsb=need - 1), WS),
        (dict(ws=9 * A + 8), WS), (dict(dr=A), ALIAS), (dict(dx=2 * A), ALIAS), (dict(dx=7 * A), ALIAS),
        (dict(dx=A + 32), ALIAS), (dict(dx=A, lddx=12), ALIAS), (dict(dw=3 * A), ALIAS), (dict(ws=7 * A), ALIAS),
        (dict(dx=A, dr=A), ALIAS), (dict(dr=5 * A, dx=5 * A), ALIAS),
    ])


def test_logprob_refusals(lib):
    good = dict(z=A, ldz=8, t=2 * A, logp=3 * A, lse=4 * A, rows=4, V=8, s=1.0, dtype=2, stream=None)
    _bad(lib, "logprob_fwd_ld", good, [
        (dict(), (OK, DEVICE)), (dict(lse=None), (OK, DEVICE)), (dict(z=None), NULL), (dict(t=None), NULL),
        (dict(lse=None, logp=None), NULL), (dict(rows=0, z=None), OK), (dict(V=0), SHAPE), (dict(V=2 ** 31, ldz=2 ** 31), SHAPE),
        (dict(ldz=7), SHAPE), (dict(s=0.0), VALUE), (dict(s=-1.0), VALUE), (dict(s=float("inf")), VALUE),
        (dict(t=2 * A + 4), VALUE), (dict(dtype=7), DTYPE), (dict(logp=A), ALIAS), (dict(lse=2 * A), ALIAS),
        (dict(lse=3 * A), ALIAS),
    ])
    good = dict(dlogp=A, z=2 * A, ldz=8, t=3 * A, lse=4 * A, dz=5 * A, lddz=8, rows=4, V=8, s=1.0, dtype=0, stream=None)
    _bad(lib, "logprob_bwd_ld", good, [
        (dict(), (OK, DEVICE)), (dict(dz=2 * A), (OK, DEVICE)), (dict(dlogp=None), NULL), (dict(z=None), NULL),
        (dict(t=None), NULL), (dict(lse=None), NULL), (dict(dz=None), NULL), (dict(rows=0, dz=None), OK),
        (dict(lddz=7), SHAPE), (dict(dz=2 * A, lddz=12), ALIAS), (dict(dz=2 * A + 16), ALIAS), (dict(dz=4 * A), ALIAS),
        (dict(s=float("nan")), VALUE),
    ])


def test_policy_loss_refusals(lib):
    assert lib.policy_loss_workspace_size(5) == 32 and lib.policy_loss_workspace_size(0) == 16
    good = dict(z=A, ldz=8, t=2 * A, old=3 * A, adv=4 * A, wt=5 * A, ref=6 * A, lo=0.2, hi=0.2, kl=0.1, s=1.0,
                gs=7 * A, loss=8 * A, logp=9 * A, dz=10 * A, lddz=8, rows=4, V=8, dtype=1, ws=11 * A, wsb=16, stream=None)
    _bad(lib, "policy_loss_ld", good, [
        (dict(), (OK, DEVICE)), (dict(dz=A), (OK, DEVICE)), (dict(dz=None, lddz=0), (OK, DEVICE)),
        (dict(wt=None, gs=None, logp=None, ref=None, kl=0.0), (OK, DEVICE)),
        (dict(z=None), NULL), (dict(t=None), NULL), (dict(old=None), NULL), (dict(adv=None), NULL),
        (dict(ref=None), NULL), (dict(loss=None), NULL), (dict(lo=-0.1), VALUE), (dict(lo=1.1), VALUE),
        (dict(hi=-0.1), VALUE), (dict(hi=float("inf")), VALUE), (dict(kl=-1.0), VALUE), (dict(s=0.0), VALUE),
        (dict(V=0), SHAPE), (dict(lddz=7), SHAPE), (dict(ws=None), WS), (dict(wsb=15), WS), (dict(ws=11 * A + 4), WS),
        (dict(dz=A, lddz=16), ALIAS), (dict(loss=A), ALIAS), (dict(logp=3 * A), ALIAS), (dict(loss=9 * A), ALIAS),
        (dict(ws=10 * A), ALIAS), (dict(dtype=5), DTYPE),
    ])


def test_binding_refuses_host_tensors_and_mismatches():
    import torch

    import row_wise_normalization_reduce_gb300 as nrm
    x = torch.zeros(4, 8)
    t = torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    for call in (lambda: nrm.dropout_fwd(x, 0.1, 0), lambda: nrm.dropout_bwd(x, 0.1, 0),
                 lambda: nrm.dropout_add_rms_fwd(x, x), lambda: nrm.dropout_add_rms_bwd(x, x, f),
                 lambda: nrm.logprob_fwd(x, t), lambda: nrm.logprob_bwd(f, x, t, f),
                 lambda: nrm.policy_loss(x, t, f, f), lambda: nrm.dropout_fwd(x, 0.1, 0, stream=0)):
        with pytest.raises(ValueError):
            call()
