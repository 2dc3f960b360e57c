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
                 lambda: nrm.qk_norm_rope_fwd(x, None, table, pos, stream=0), lambda: nrm.route_fwd(x, 2),
                 lambda: nrm.route_bwd(x[..., :2], x, pos[:, None]), lambda: nrm.route_fwd(x, 2, score="none"),
                 lambda: nrm.logprob_top_fwd(x, torch.zeros(4, 2, dtype=torch.int64), 2),
                 lambda: nrm.logprob_top_bwd(None, None, None, x, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2, 2))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(1)
    x, dw, ds = (torch.randn(3, n, generator=g, dtype=torch.float64) for n in (7, 2, 7))
    ids = R.route(x, 2, score=score)[1]
    ids[2, 1] = -1

    def f(x):
        s = R.scores64(x, score)
        w = torch.where(ids >= 0, s.gather(1, ids.clamp(0)), 0.0)
        return 1.5 * ((w / w.sum(-1, keepdim=True) if renorm else w) * dw).sum() + (s * ds).sum()

    dx, _ = R.route_grad(dw, x, ids, score=score, renormalize=renorm, scale=1.5, dscores=ds)
    differences(f, x, dx, 1e-8)


def test_route_definition_by_hand():
    x = torch.tensor([[0.0, 2.0, 1.0, 1.0, -float("inf"), 5.0]])
    w, ids = R.route(x, 3, renormalize=True)
    e = torch.tensor([5.0, 2.0, 1.0], dtype=torch.float64).exp()
    assert ids.tolist() == [[5, 1, 2]] and torch.allclose(w, (e / e.sum())[None], rtol=1e-14)
    # groups (0, 1), (2, 3), (4, 5): sums of two 2, 2, 5 and of one 2, 1, 5
    assert R.route(x, 2, groups=3, top_groups=1)[1].tolist() == [[5, -1]]
    assert R.route(x, 3, groups=3, top_groups=2)[1].tolist() == [[5, 1, 0]]
    b = torch.tensor([0.0, -1.0, 0.5, 0.0, 9.0, 0.0])
    assert R.route(x, 2, b, score="sigmoid")[1].tolist() == [[2, 5]]


def test_route_refusals(lib):
    good = dict(x=A, ldx=64, bias=2 * A, w=3 * A, ids=4 * A, sc=5 * A, t=4, e=64, k=6, score=0, groups=8, top=3, gt=2, renorm=1,
                scale=1.0, dtype=2, stream=None)
    _bad(lib, "route_fwd", good, [
        (dict(), (OK, DEVICE)), (dict(bias=None, sc=None), (OK, DEVICE)), (dict(t=0, x=None, w=None), OK), (dict(score=1), (OK, DEVICE)),
        (dict(x=None), NULL), (dict(w=None), NULL), (dict(ids=None), NULL), (dict(t=-1), SHAPE), (dict(e=0, k=0), SHAPE),
        (dict(k=0), SHAPE), (dict(k=65, top=8), SHAPE), (dict(k=25), SHAPE), (dict(ldx=63), SHAPE), (dict(groups=7), SHAPE),
        (dict(groups=0), SHAPE), (dict(top=0), SHAPE), (dict(top=9), SHAPE), (dict(gt=0), SHAPE), (dict(t=2 ** 60), SHAPE),
        (dict(gt=3), UNSUP), (dict(gt=3, top=8), (OK, DEVICE)), (dict(e=1025, ldx=1025, groups=1, top=1), UNSUP),
        (dict(e=64, k=33, groups=1, top=1), UNSUP), (dict(groups=64, k=1, top=2), UNSUP), (dict(e=1020, ldx=1020, groups=17), UNSUP),
        (dict(score=2), VALUE), (dict(scale=float("inf")), VALUE), (dict(x=A + 1), VALUE), (dict(bias=2 * A + 2), VALUE),
        (dict(ids=4 * A + 4), VALUE), (dict(sc=5 * A + 1), VALUE), (dict(dtype=3), DTYPE), (dict(w=A), ALIAS), (dict(ids=2 * A), ALIAS),
        (dict(sc=3 * A), ALIAS), (dict(sc=A), ALIAS),
    ])
    good = dict(dw=A, x=2 * A, ldx=64, ids=3 * A, ds=4 * A, dx=5 * A, lddx=64, t=4, e=64, k=6, score=0, renorm=1, scale=1.0, dtype=0,
                stream=None)
    _bad(lib, "route_bwd", good, [
        (dict(), (OK, DEVICE)), (dict(ds=None), (OK, DEVICE)), (dict(dx=2 * A), (OK, DEVICE)), (dict(t=0, dw=None), OK),
        (dict(dw=None), NULL), (dict(x=None), NULL), (dict(ids=None), NULL), (dict(dx=None), NULL), (dict(lddx=63), SHAPE),
        (dict(k=65), SHAPE), (dict(k=33), UNSUP), (dict(score=-1), VALUE), (dict(dw=A + 2), VALUE), (dict(dx=2 * A, lddx=65), ALIAS),
        (dict(dx=4 * A), ALIAS), (dict(dx=A), ALIAS), (dict(dx=3 * A), ALIAS), (dict(dtype=-1), DTYPE),
    ])


def test_logprob_top_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    rows, v, k, s = 3, 6, 2, 0.7
    z, dh, da = (torch.randn(*n, generator=g, dtype=torch.float64) for n in ((rows, v), (rows,), (rows, k)))
    dl, t = torch.randn(rows, generator=g, dtype=torch.float64), torch.tensor([0, 5, -100])
    f, _ = R.logprob_top(z, t, k, s)
    ids = f["ids"].clone()
    ids[1] = torch.tensor([5, -1])

    def loss(z):
        lp = torch.log_softmax(s * z, -1)
        h = -(lp.exp() * lp).sum(-1)
        top = torch.where(ids >= 0, lp.gather(1, ids.clamp(0)), 0.0)
        return ((lp.gather(1, t.clamp(0)[:, None])[:, 0] * dl + h * dh + (top * da).sum(1)) * (t >= 0)).sum()

    dz, _ = R.logprob_top_grad(z, t, f["stats"], f["entropy"], ids, dl, dh, da, s)
    differences(loss, z, dz, 1e-8)
    assert not dz[2].any()


def test_logprob_top_definition_by_hand():
    z = torch.tensor([[1.0, 3.0, -float("inf"), 3.0, 0.0], [0.0] * 5, [-float("inf")] * 5])
    f, _ = R.logprob_top(z, torch.tensor([3, 9, 0]), 5)
    assert f["ids"].tolist() == [[1, 3, 0, 4, -1], [-1] * 5, [-1] * 5]
    d = 2 + torch.tensor(-2.0, dtype=torch.float64).exp() + torch.tensor(-3.0, dtype=torch.float64).exp()
    assert abs(float(f["logp"][0] + d.log())) < 1e-14 and f["logp"][1] == 0 and f["logp"][2] == -float("inf")
    assert f["top"][0, 4] == -float("inf") and not f["top"][1].any()


def test_logprob_top_refusals(lib):
    good = dict(z=A, ldz=64, t=2 * A, logp=3 * A, ent=4 * A, ids=5 * A, top=6 * A, st=7 * A, rows=4, V=64, k=5, s=1.0, dtype=2,
                stream=None)
    _bad(lib, "logprob_top_fwd_ld", good, [
        (dict(), (OK, DEVICE)), (dict(logp=None, ent=None, st=None), (OK, DEVICE)), (dict(k=0, ids=None, top=None), (OK, DEVICE)),
        (dict(k=32), (OK, DEVICE)), (dict(V=3, ldz=3), (OK, DEVICE)), (dict(rows=0, z=None), OK), (dict(z=None), NULL),
        (dict(t=None), NULL), (dict(ids=None), NULL), (dict(top=None), NULL), (dict(k=0, logp=None, ent=None, st=None), NULL),
        (dict(k=33), UNSUP), (dict(k=-1), SHAPE), (dict(V=0), SHAPE), (dict(rows=2 ** 58, V=1, ldz=1), SHAPE), (dict(V=2 ** 31, ldz=2 ** 31), SHAPE), (dict(ldz=63), SHAPE),
        (dict(s=0.0), VALUE), (dict(s=float("nan")), VALUE), (dict(s=3e38), VALUE), (dict(ids=5 * A + 4), VALUE),
        (dict(st=7 * A + 2), VALUE), (dict(z=A + 1), VALUE), (dict(dtype=4), DTYPE), (dict(ids=A), ALIAS), (dict(top=5 * A), ALIAS),
        (dict(ent=2 * A), ALIAS), (dict(st=3 * A), ALIAS),
    ])
    good = dict(g=A, h=2 * A, a=3 * A, z=4 * A, ldz=64, t=5 * A, st=6 * A, ent=7 * A, ids=8 * A, dz=9 * A, lddz=64, rows=4, V=64,
                k=5, s=1.0, dtype=0, stream=None)
    _bad(lib, "logprob_top_bwd_ld", good, [
        (dict(), (OK, DEVICE)), (dict(dz=4 * A), (OK, DEVICE)), (dict(g=None, h=None, ent=None), (OK, DEVICE)),
        (dict(a=None, ids=None), (OK, DEVICE)), (dict(k=0, a=None, ids=None), (OK, DEVICE)), (dict(rows=0, dz=None), OK),
        (dict(g=None, h=None, a=None), NULL), (dict(ent=None), NULL), (dict(ids=None), NULL), (dict(st=None), NULL),
        (dict(z=None), NULL), (dict(t=None), NULL), (dict(dz=None), NULL), (dict(k=0, g=None, h=None), NULL), (dict(k=33), UNSUP),
        (dict(k=-1), SHAPE), (dict(lddz=63), SHAPE), (dict(dz=4 * A, lddz=65), ALIAS), (dict(dz=8 * A), ALIAS), (dict(dz=7 * A), ALIAS),
        (dict(dz=3 * A), ALIAS), (dict(st=6 * A + 2), VALUE), (dict(ids=8 * A + 4), VALUE), (dict(s=-1.0), VALUE), (dict(dtype=3), DTYPE),
    ])


def test_pointers_that_are_not_used_are_not_looked_at(lib):
    # refused by nothing: off their alignment, or where an output lies
    good = dict(q=A, qt=64, qh=64, k=None, kt=0, kh=0, tab=2 * A, pos=3 * A, wq=None, wk=None, qo=6 * A, qot=64, qoh=64,
                         ko=None, kot=0, koh=0, t=4, hq=1, hk=0, d=64, rot=64, most=100, eps=1e-6, near=0, dtype=0, stream=None)
    _bad(lib, "qk_norm_rope_fwd", good, [
        (dict(), (OK, DEVICE)), (dict(k=A + 1, wk=A + 1, ko=A + 1), (OK, DEVICE)), (dict(wk=6 * A), (OK, DEVICE)),
        (dict(rot=0, tab=2 * A + 1), (OK, DEVICE)), (dict(rot=0, tab=6 * A), (OK, DEVICE))])
    back = dict(gq=A, gqt=64, gqh=64, gk=None, gkt=0, gkh=0, q=2 * A, qt=64, qh=64, k=None, kt=0, kh=0, tab=3 * A, pos=4 * A, wq=None,
                wk=None, dq=5 * A, dqt=64, dqh=64, dk=None, dkt=0, dkh=0, dwq=6 * A, dwk=None, t=4, hq=1, hk=0, d=64, rot=64, most=100,
                eps=1e-6, near=0, dtype=0, ws=7 * A, wsb=608 * 2 * 64 * 4, stream=None)
    _bad(lib, "qk_norm_rope_bwd", back, [
        (dict(), (OK, DEVICE)), (dict(gk=A + 1, k=A + 1, wk=A + 1, dk=A + 1), (OK, DEVICE)), (dict(wk=6 * A), (OK, DEVICE)),
        (dict(rot=0, tab=3 * A + 1), (OK, DEVICE)), (dict(rot=0, tab=7 * A), (OK, DEVICE))])
    top = dict(g=A, h=None, a=None, z=2 * A, ldz=64, t=3 * A, st=4 * A, ent=None, ids=None, dz=5 * A, lddz=64, rows=4, V=64, k=5, s=1.0,
               dtype=0, stream=None)
    _bad(lib, "logprob_top_bwd_ld", top, [
        (dict(), (OK, DEVICE)), (dict(ent=6 * A + 1), (OK, DEVICE)), (dict(ent=5 * A), (OK, DEVICE)), (dict(ids=5 * A), (OK, DEVICE))])
