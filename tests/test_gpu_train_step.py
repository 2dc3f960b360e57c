"""The training operators together, as a fine-tuning step uses them: two
residual blocks with dropout and RMSNorm, a matrix product between them, logits,
reference log-probabilities and the policy loss; then the backward through all of
it.  Against the same step in 64 bits by torch's own differentiation on the CPU
with the masks of train_ref.py, and captured into a graph whose dropout counter
advances on the device."""
import numpy as np
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

T, D, V, P, EPS = 48, 96, 1000, 0.2, 1e-5
CLIP, KL, SEED = (0.2, 0.3), 0.05, 99


@pytest.fixture(autouse=True)
def _setup():
    nrm.build()
    nrm.force_plan(nrm.PLAN_AUTO)
    yield


def parameters():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"x": r(T, D), "res": r(T, D), "w1": 1 + 0.1 * r(D), "w2": 1 + 0.1 * r(D), "m": r(D, D) / D ** 0.5, "v": r(D, V) / D ** 0.5 * 2}
    t = torch.randint(0, V, (T,), generator=g)
    t[5], t[20] = -100, V
    wt = torch.rand(T, generator=g) / T
    wt[7] = 0
    adv = torch.where(torch.rand(T, generator=g) < 0.5, 1.0, -1.0) * (0.5 + torch.rand(T, generator=g))
    return p, t, wt, adv


def step(p, t, old, ref, adv, wt, offset, offset_dev=None):
    """One training step: the loss and the gradients of everything in p."""
    drop = dict(p=P, seed=SEED, offset_dev=offset_dev)
    h1, y1, r1 = nrm.dropout_add_rms_fwd(p["x"], p["res"], p["w1"], offset=offset, eps=EPS, **drop)
    u = y1 @ p["m"]
    h2, y2, r2 = nrm.dropout_add_rms_fwd(u, h1, p["w2"], offset=offset + 1, eps=EPS, **drop)
    z = nrm.dropout_fwd(y2, P, SEED, offset + 2, offset_dev=offset_dev)
    logits = z @ p["v"]
    loss, logp, dlogits = nrm.policy_loss(logits, t, old, adv, wt, ref, *CLIP, KL)
    g = {"v": z.t() @ dlogits}
    dy2 = nrm.dropout_bwd(dlogits @ p["v"].t(), P, SEED, offset + 2, offset_dev=offset_dev)
    du, dh1, g["w2"] = nrm.dropout_add_rms_bwd(dy2, h2, r2, p["w2"], offset=offset + 1, **drop)
    g["m"] = y1.t() @ du
    g["x"], g["res"], g["w1"] = nrm.dropout_add_rms_bwd(du @ p["m"].t(), h1, r1, p["w1"], offset=offset, dresidual_out=dh1, **drop)
    return loss, logp, g


def exact_logits(p, offset):
    m = [torch.from_numpy(R.keep(T, D, P, SEED, offset + i)) for i in range(3)]
    s = R.bar_scale(P)[1]
    norm = lambda h, w: h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w  # noqa: E731
    h1 = p["res"] + m[0] * p["x"] * s
    h2 = h1 + m[1] * (norm(h1, p["w1"]) @ p["m"]) * s
    return (m[2] * norm(h2, p["w2"]) * s) @ p["v"]


def exact(p, t, old, ref, adv, wt, offset):
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    ok = (t >= 0) & (t < V) & (wt != 0)
    lp = torch.log_softmax(exact_logits(q, offset), -1)[torch.arange(T), t.clamp(0, V - 1)]
    lp = torch.where(ok, lp, 0.0)
    old, ref, adv, wt = (a.double() for a in (old, ref, adv, wt))
    ratio = torch.exp(lp - old)
    k = ref - lp
    term = torch.maximum(-adv * ratio, -adv * ratio.clamp(1 - CLIP[0], 1 + CLIP[1])) + KL * (torch.exp(k) - k - 1)
    loss = torch.where(ok, wt * term, 0.0).sum()
    loss.backward()
    return loss.detach(), lp.detach(), {k: v.grad for k, v in q.items()}


def rows_of(p, t, offset):
    """Old and reference log-probabilities away from the clip bounds."""
    with torch.no_grad():
        lp = torch.log_softmax(exact_logits({k: v.double() for k, v in p.items()}, offset), -1)[torch.arange(T), t.clamp(0, V - 1)]
    g = torch.Generator().manual_seed(4)
    away = torch.tensor([-0.5, -0.1, 0.05, 0.5])[torch.randint(0, 4, (T,), generator=g)]
    return (lp - away).float(), (lp + 0.2 * torch.randn(T, generator=g)).float()


def near(got, want, what):
    # five binary32 stages, each within 64 roundings of its operands' norms
    # (sums of 96 to 1000 terms): 5 * 64 * 2^-24 < 2e-5 of the norm
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    assert float((got - want).norm()) <= 2e-5 * float(want.norm()), (what, float((got - want).norm() / want.norm()))


def test_step_against_differentiation():
    p, t, wt, adv = parameters()
    old, ref = rows_of(p, t, 3)
    want = exact(p, t, old, ref, adv, wt, 3)
    got = step({k: v.cuda() for k, v in p.items()}, t.cuda(), old.cuda(), ref.cuda(), adv.cuda(), wt.cuda(), 3)
    near(got[0], want[0], "loss")
    near(got[1], want[1], "logp")
    assert set(got[2]) == set(want[2])
    for k in got[2]:
        near(got[2][k], want[2][k], k)


def test_step_in_a_graph_with_a_counter_on_the_device():
    p, t, wt, adv = parameters()
    old, ref = rows_of(p, t, 0)
    q = {k: v.cuda() for k, v in p.items()}
    rest = [a.cuda() for a in (t, old, ref, adv, wt)]
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q, *rest, 0, count)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(q, *rest, 0, count)
        count += 3
    seen = []
    for i in range(3):
        want = step(q, *rest, 3 * i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([*got[:2], *got[2].values()], [*want[:2], *want[2].values()]):
            # the same kernels on the same masks; the products between them may
            # take another algorithm under capture
            near(a, b.cpu(), i)
        seen.append(float(got[0]))
    assert len(set(seen)) == 3
