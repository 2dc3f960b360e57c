"""The operators inside a block without a GPU: the tests' own definitions
against differences, and the refusals of the library (no call here reaches a
launch on a machine without a device; the pointers are never dereferenced)."""
import pytest
import torch

import block_ref as R

OK, NULL, SHAPE, DTYPE, ALIAS, VALUE, UNSUP, WS, DEVICE = range(9)
A = 0x1000000


@pytest.fixture(scope="module")
def lib():
    import os

    import row_wise_normalization_reduce_gb300 as nrm
    if not os.path.exists(nrm.LIB_PATH):
        nrm.build()
    return nrm.lib()


def _bad(lib, name, good, cases):
    f = getattr(lib, name)
    keys = list(good)
    for change, want in cases:
        assert set(change) <= set(keys), change
        st = f(*[dict(good, **change)[k] for k in keys])
        assert st in (want if isinstance(want, tuple) else (want,)), (name, change, st, want)


def differences(f, x, grad, tol, step=1e-5):
    """grad of the scalar f at x (64 bits) against central differences."""
    flat, g = x.reshape(-1), grad.reshape(-1)
    for i in range(flat.numel()):
        hi, lo = flat.clone(), flat.clone()
        hi[i] += step
        lo[i] -= step
        d = (f(hi.view(x.shape)) - f(lo.view(x.shape))) / (2 * step)
        assert abs(float(d) - float(g[i])) < tol, (i, float(d), float(g[i]))


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("d,rot", [(6, 6), (7, 4), (5, 0)])
def test_head_norm_gradient_against_differences(d, rot, near):
    g = torch.Generator().manual_seed(d)
    x, dout = (torch.randn(4, 2, d, generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(d, generator=g, dtype=torch.float64)
    table, pos = R.angle_table(9, rot), torch.tensor([0, 8, -1, 9])
    f = lambda x, w: (R.head_norm(x, w, table, pos, 1e-3, near)[0] * dout).sum()  # noqa: E731
    dx, _, dw, _ = R.head_norm_bwd(dout, x, w, table, pos, 1e-3, near)
    differences(lambda t: f(t, w), x, dx, 1e-8)
    differences(lambda t: f(x, t), w, dw, 1e-8)
    assert not dx[2:].any()


def test_head_norm_refusals(lib):
    t, hq, hk, d = 4, 6, 2, 64
    row = (hq + 2 * hk) * d
    good = dict(q=A, qt=row, qh=d, k=A + hq * d * 2, kt=row, kh=d, tab=2 * A, pos=3 * A, wq=4 * A, wk=5 * A, qo=6 * A,
                qot=hq * d, qoh=d, ko=7 * A, kot=hk * d, koh=d, t=t, hq=hq, hk=hk, d=d, rot=d, most=100, eps=1e-6, near=0,
                dtype=2, stream=None)
    _bad(lib, "qk_norm_rope_fwd", good, [
        (dict(), (OK, DEVICE)), (dict(wq=None, wk=None), (OK, DEVICE)), (dict(near=1), (OK, DEVICE)),
        (dict(hk=0, k=None, ko=None, wk=None), (OK, DEVICE)), (dict(rot=0, tab=None), (OK, DEVICE)),
        (dict(most=0, tab=None), (OK, DEVICE)), (dict(t=0, q=None, pos=None), OK),
        (dict(qo=A, qot=row, qoh=d, ko=A + hq * d * 2, kot=row, koh=d), (OK, DEVICE)),  # in place in the projection
        (dict(qt=d, qh=t * d, kt=d, kh=t * d, k=8 * A), (OK, DEVICE)),  # tokens within heads
        (dict(t=1, qt=0, kt=0, qot=0, kot=0), (OK, DEVICE)), (dict(hk=1, kh=0, koh=0), (OK, DEVICE)),
        (dict(q=None), NULL), (dict(k=None), NULL), (dict(tab=None), NULL), (dict(pos=None), NULL), (dict(qo=None), NULL),
        (dict(ko=None), NULL), (dict(t=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hk=-1), SHAPE), (dict(d=0), SHAPE),
        (dict(d=513, rot=64, qt=row * 9, qh=513, kt=row * 9, kh=513), UNSUP), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE),
        (dict(rot=-2), SHAPE), (dict(most=-1), SHAPE), (dict(most=2 ** 60), SHAPE), (dict(t=2 ** 41), SHAPE),
        (dict(qh=d - 1), SHAPE), (dict(qt=0), SHAPE), (dict(qoh=0), SHAPE), (dict(qot=d, qoh=d), SHAPE),
        (dict(qt=2 ** 60), SHAPE), (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(dtype=3), DTYPE),
        (dict(q=A + 1), VALUE), (dict(wk=5 * A + 1), VALUE), (dict(tab=2 * A + 2), VALUE), (dict(pos=3 * A + 4), VALUE),
        (dict(qo=A), ALIAS), (dict(qo=A + 2, qot=row), ALIAS), (dict(qo=4 * A), ALIAS), (dict(ko=6 * A), ALIAS),
        (dict(ko=3 * A), ALIAS), (dict(qo=2 * A), ALIAS), (dict(qo=A + hq * d * 2, qot=row, qoh=d), ALIAS),
    ])


def test_head_norm_bwd_refusals(lib):
    t, hq, hk, d = 4, 6, 2, 64
    need = lib.qk_norm_rope_bwd_workspace_size(t, hq, hk, d)
    assert need == 608 * 2 * d * 4
    assert lib.qk_norm_rope_bwd_workspace_size(t, hq, hk, 513) == 0 == lib.qk_norm_rope_bwd_workspace_size(t, 0, hk, d)
    good = dict(gq=A, gqt=hq * d, gqh=d, gk=2 * A, gkt=hk * d, gkh=d, q=3 * A, qt=hq * d, qh=d, k=4 * A, kt=hk * d, kh=d,
                tab=5 * A, pos=6 * A, wq=7 * A, wk=8 * A, dq=9 * A, dqt=hq * d, dqh=d, dk=10 * A, dkt=hk * d, dkh=d,
                dwq=11 * A, dwk=12 * A, t=t, hq=hq, hk=hk, d=d, rot=d, most=100, eps=1e-6, near=0, dtype=0, ws=13 * A,
                wsb=need, stream=None)
    _bad(lib, "qk_norm_rope_bwd", good, [
        (dict(), (OK, DEVICE)), (dict(dwq=None, dwk=None, ws=None, wsb=0), (OK, DEVICE)), (dict(dwk=None), (OK, DEVICE)),
        (dict(dq=A, dk=2 * A), (OK, DEVICE)), (dict(dq=3 * A, dk=4 * A), (OK, DEVICE)),
        (dict(t=0, dwq=None, dwk=None, q=None), OK), (dict(gq=None), NULL), (dict(gk=None), NULL), (dict(dq=None), NULL),
        (dict(dk=None), NULL), (dict(ws=None), WS), (dict(wsb=need - 1), WS), (dict(ws=13 * A + 8), WS),
        (dict(dwq=11 * A + 2), VALUE), (dict(gq=A + 2), VALUE), (dict(hk=0), SHAPE), (dict(gqh=d - 1), SHAPE),
        (dict(dq=A, dqt=2 * hq * d), ALIAS), (dict(dq=2 * A), ALIAS), (dict(dk=9 * A), ALIAS), (dict(dwq=9 * A), ALIAS),
        (dict(dwk=11 * A), ALIAS), (dict(ws=9 * A), ALIAS), (dict(ws=3 * A), ALIAS), (dict(dwq=6 * A), ALIAS),
        (dict(dwk=13 * A), ALIAS), (dict(dwq=7 * A), ALIAS), (dict(d=600, rot=0), UNSUP), (dict(dtype=9), DTYPE),
    ])


def test_binding_refuses_mismatches():
    import row_wise_normalization_reduce_gb300 as nrm
    x, pos, table = torch.zeros(4, 2, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(10, 8)
    for call in (lambda: nrm.qk_norm_rope_fwd(x, x, table, pos), lambda: nrm.qk_norm_rope_bwd(x, x, x, x, table, pos),
                 lambda: nrm.qk_norm_rope_fwd(x, None, table, pos, stream=0)):
        with pytest.raises(ValueError):
            call()
