"""The operators of a transformer block together, as a training step uses them:
RMSNorm, head norms with the position rotation on slices of one projection, the
residual add, routing to experts with a balance term on all scores, and the
log-probabilities with entropy and alternatives, each with its gradient through
the library, against the same step in 64 bits by autograd."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

import row_wise_normalization_reduce_gb300 as nrm  # noqa: E402

SEQS, LEN, D, HQ, HK, HD, E, K, V, TOP = 2, 13, 48, 4, 2, 16, 12, 3, 101, 4
EPS = 1e-5


@pytest.fixture(autouse=True, scope="module")
def _built():
    nrm.build()


class Norm(torch.autograd.Function):
    """residual + x and its RMSNorm."""
    @staticmethod
    def forward(ctx, x, residual, w):
        h, y, rstd = nrm.add_rms_fwd(x, residual, w, EPS, want_stats=True)
        ctx.save_for_backward(h, rstd, w)
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        h, rstd, w = ctx.saved_tensors
        dx, dr, dw = nrm.dropout_add_rms_bwd(dy.contiguous(), h, rstd, w, dresidual_out=dh.contiguous())
        return dx, dr, dw


class Heads(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qkv, wq, wk, table, pos):
        q, k = qkv[:, :HQ], qkv[:, HQ:HQ + HK]
        ctx.save_for_backward(qkv, wq, wk, table, pos)
        return nrm.qk_norm_rope_fwd(q, k, table, pos, wq, wk, EPS)

    @staticmethod
    def backward(ctx, dq, dk):
        qkv, wq, wk, table, pos = ctx.saved_tensors
        out = torch.zeros_like(qkv)  # the values' part has no gradient from here
        _, _, dwq, dwk = nrm.qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), qkv[:, :HQ], qkv[:, HQ:HQ + HK], table, pos,
                                              wq, wk, EPS, dq=out[:, :HQ], dk=out[:, HQ:HQ + HK])
        return out, dwq, dwk, None, None


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias):
        w, ids, scores = nrm.route_fwd(logits, K, bias, score="sigmoid", groups=4, top_groups=2, group_top=2, scale=1.5,
                                       want_scores=True)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return w, ids, scores

    @staticmethod
    def backward(ctx, dw, _, dscores):
        logits, ids = ctx.saved_tensors
        return nrm.route_bwd(dw.contiguous(), logits, ids, score="sigmoid", scale=1.5, dscores=dscores.contiguous()), None


class Loss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets):
        logp, ent, ids, top, stats = nrm.logprob_top_fwd(logits, targets, TOP)
        ctx.save_for_backward(logits, targets, ent, ids, stats)
        ctx.mark_non_differentiable(ids)
        return logp, ent, ids, top

    @staticmethod
    def backward(ctx, dlogp, dent, _, dtop):
        logits, targets, ent, ids, stats = ctx.saved_tensors
        return nrm.logprob_top_bwd(dlogp.contiguous(), dent.contiguous(), dtop.contiguous(), logits, targets, stats, ent, ids), None


def plain(ids=None, top_ids=None):
    """The same four by formulas, for autograd."""
    def norm(x, residual, w):
        h = x + residual
        return h, h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * w

    def heads(qkv, wq, wk, table, pos):
        live = R.live_tokens(table, pos)[:, None, None]
        out = []
        for x, w in ((qkv[:, :HQ], wq), (qkv[:, HQ:HQ + HK], wk)):
            y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
            t = table.double()[pos.clamp(0, table.shape[0] - 1)][:, None]
            c, s, (a, b) = t[..., :HD // 2], t[..., HD // 2:], y.chunk(2, -1)
            out.append(torch.where(live, torch.cat([a * c - b * s, b * c + a * s], -1), 0.0))
        return out

    def route(logits, bias):
        s = torch.sigmoid(logits)
        w = s.gather(1, ids)
        return 1.5 * w / w.sum(-1, keepdim=True), ids, s

    def loss(logits, targets):
        lp = torch.log_softmax(logits, -1)
        live = targets >= 0
        z = torch.zeros((), dtype=lp.dtype, device=lp.device)
        top = torch.where(live[:, None], lp.gather(1, top_ids.clamp(0)), z)
        return (torch.where(live, lp.gather(1, targets.clamp(0)[:, None])[:, 0], z),
                torch.where(live, -(lp.exp() * lp).sum(-1), z), top_ids, top)

    return norm, heads, route, loss


def step(p, x, table, pos, targets, bias, ops):
    norm, heads, route, loss = ops
    h, y = norm(x, torch.zeros_like(x), p["w0"])
    qkv = (y @ p["qkv"]).view(-1, HQ + 2 * HK, HD)
    q, k = heads(qkv, p["wq"], p["wk"], table, pos)
    q, k, v = (t.reshape(SEQS, LEN, -1, HD).transpose(1, 2) for t in (q, k, qkv[:, HQ + HK:]))
    k, v = (t.repeat_interleave(HQ // HK, 1) for t in (k, v))
    att = (q @ k.transpose(-1, -2) / HD ** 0.5).masked_fill(torch.ones(LEN, LEN, dtype=torch.bool, device=x.device).triu(1), -1e9)
    att = (torch.softmax(att, -1) @ v).transpose(1, 2).reshape(SEQS * LEN, HQ * HD)
    h, y = norm(att @ p["o"], h, p["w1"])
    w, ids, scores = route(y @ p["router"], bias)
    out = torch.einsum("tk,tkd->td", w, torch.tanh(torch.einsum("td,tkde->tke", y, p["experts"][ids])))
    h, y = norm(out, h, p["w2"])
    logp, ent, top_ids, top = loss(y @ p["head"], targets)
    share = torch.arange(1, TOP + 1, device=x.device, dtype=x.dtype) / TOP
    total = -logp.sum() - 0.1 * ent.sum() + 0.05 * (top * share).sum() + 0.3 * (scores.mean(0).square()).sum()
    return total, ids, top_ids


def test_a_step_of_all_operators():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = {"w0": 1 + 0.2 * r(D), "w1": 1 + 0.2 * r(D), "w2": 1 + 0.2 * r(D), "wq": 1 + 0.2 * r(HD), "wk": 1 + 0.2 * r(HD),
         "qkv": r(D, (HQ + 2 * HK) * HD) / D ** 0.5, "o": r(HQ * HD, D) / 8, "router": r(D, E) / 5, "experts": r(E, D, D) / 7,
         "head": r(D, V) / 4}
    x, bias, table = r(SEQS * LEN, D), 0.1 * r(E), R.angle_table(LEN, HD)
    pos, targets = torch.arange(LEN).repeat(SEQS), torch.randint(0, V, (SEQS * LEN,), generator=g)
    pos[-2:], targets[-2:], targets[:3] = -1, -100, -100  # padding; a prompt
    p, x, bias, table, pos, targets = ({n: t.cuda() for n, t in p.items()}, *(t.cuda() for t in (x, bias, table, pos, targets)))

    def grads(dtype, ops):
        q = {n: t.detach().clone().to(dtype).requires_grad_() for n, t in p.items()}
        xx = x.detach().clone().to(dtype).requires_grad_()
        total, ids, top_ids = step(q, xx, table, pos, targets, bias, ops)
        total.backward()
        return total.detach(), ids, top_ids, {**{n: t.grad for n, t in q.items()}, "x": xx.grad}

    ours = (Norm.apply, Heads.apply, Route.apply, Loss.apply)
    total, ids, top_ids, got = grads(torch.float32, ours)
    want_total, _, _, want = grads(torch.float64, plain(ids, top_ids))
    # every operator is good to 2^-16 of the sums it makes of absolute values and the
    # products over at most 64 entries to 2^-18; a path passes some twenty of them, a
    # gradient's terms cancel to a tenth of their sum at worst: 2^-9 of its norm
    assert abs(float(total - want_total)) <= 2.0 ** -12 * abs(float(want_total))
    for name, t in got.items():
        err = float((t.double() - want[name]).norm() / want[name].norm())
        assert err <= 2.0 ** -9, (name, err)
    again = grads(torch.float32, ours)[3]
    assert all(torch.equal(again[n], t) for n, t in got.items() if n in ("wq", "wk", "w0", "w2"))


def test_the_forward_captured_with_an_eager_graph_alive():
    # a decoding step in a CUDA graph: head norms in place in the projection's
    # output, routing and the alternatives of the last logits
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(7, HQ + 2 * HK, HD, device="cuda", generator=g).bfloat16()
    wq, wk = (torch.ones(HD, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table, pos = R.angle_table(64, HD, device="cuda"), torch.arange(7, device="cuda") * 9
    router, logits = (torch.randn(7, n, device="cuda", generator=g).bfloat16() for n in (E, 1000))
    targets = torch.zeros(7, dtype=torch.int64, device="cuda")
    work = qkv.clone()

    def run():
        work.copy_(qkv)
        q, k = nrm.qk_norm_rope_fwd(work[:, :HQ], work[:, HQ:HQ + HK], table, pos, wq, wk, q_out=work[:, :HQ], k_out=work[:, HQ:HQ + HK])
        return (q, k, *nrm.route_fwd(router, K)[:2], *nrm.logprob_top_fwd(logits, targets, TOP))

    want = [t.clone() for t in run()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for t in got[2:]:
            t.fill_(0)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pos += 1  # the next step's positions and logits, the same graph
    logits.copy_(logits.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got]
    assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_two_streams_at_once():
    # the same operators on two streams, each call with scratch and outputs of its own
    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        return r(900, 8, 128), r(900, 2, 128), r(900, 8, 128), r(900, 2, 128), r(900, 256), r(300, 30000)

    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    table, pos = R.angle_table(900, 128, device="cuda"), torch.arange(900, device="cuda")
    targets = torch.arange(300, device="cuda")

    def run(i):
        q, k, gq, gk, router, logits = i
        f = nrm.logprob_top_fwd(logits, targets, 9)
        w_, ids, _ = nrm.route_fwd(router, 8, score="sigmoid")
        return (*nrm.qk_norm_rope_bwd(gq, gk, q, k, table, pos, w, w), *f, w_, ids, nrm.route_bwd(w_, router, ids, score="sigmoid"),
                nrm.logprob_top_bwd(f[0], f[1], f[3], logits, targets, f[4], f[1], f[2]))

    both = [inputs(1), inputs(2)]
    want = [run(i) for i in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for i, s in zip(both, streams):
            with torch.cuda.stream(s):
                got.append(run(i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
