"""The stats forms of the log-probability without a GPU: what the library
refuses (no call here reaches a launch; the pointers are never dereferenced),
and why the forms are there, in the arithmetic of the two contracts."""
import numpy as np
import pytest

from test_train_ops_cpu import ALIAS, DEVICE, DTYPE, NULL, OK, SHAPE, VALUE, A, _bad, lib  # noqa: F401


def test_refusals(lib):  # noqa: F811
    good = dict(z=A, ldz=8, t=2 * A, logp=3 * A, lse=4 * A, stats=5 * A, rows=4, V=8, s=1.0, dtype=2, stream=None)
    _bad(lib, "logprob_fwd_stats_ld", good, [
        (dict(), (OK, DEVICE)), (dict(lse=None, logp=None), (OK, DEVICE)), (dict(stats=None), (OK, DEVICE)),
        (dict(z=None), NULL), (dict(t=None), NULL), (dict(lse=None, logp=None, stats=None), NULL),
        (dict(rows=0, z=None), OK), (dict(V=0), SHAPE), (dict(ldz=7), SHAPE), (dict(s=0.0), VALUE),
        (dict(stats=5 * A + 2), VALUE), (dict(dtype=7), DTYPE), (dict(stats=A), ALIAS), (dict(stats=2 * A), ALIAS),
        (dict(stats=3 * A), ALIAS), (dict(stats=4 * A - 16), ALIAS),
    ])
    good = dict(dlogp=A, z=2 * A, ldz=8, t=3 * A, stats=4 * A, dz=5 * A, lddz=8, rows=4, V=8, s=1.0, dtype=0, stream=None)
    _bad(lib, "logprob_bwd_stats_ld", good, [
        (dict(), (OK, DEVICE)), (dict(dz=2 * A), (OK, DEVICE)), (dict(dlogp=None), NULL), (dict(z=None), NULL),
        (dict(t=None), NULL), (dict(stats=None), NULL), (dict(dz=None), NULL), (dict(rows=0, dz=None), OK),
        (dict(lddz=7), SHAPE), (dict(dz=2 * A, lddz=12), ALIAS), (dict(dz=4 * A), ALIAS), (dict(dz=4 * A + 16), ALIAS),
        (dict(stats=4 * A + 1), VALUE), (dict(s=float("nan")), VALUE),
    ])


@pytest.mark.parametrize("offset", [0.0, 1e3, 1e4, float(np.finfo(np.float32).min)])
def test_what_one_number_loses(offset):
    # a uniform row of v logits: 1 / v from the maximum and log v; from their sum
    # in binary32 within |lse| 2^-24, and nothing of it at the lowest value
    v = 1003
    m, logd = np.float32(offset), np.float32(np.log(v))
    lse = np.float32(m + logd)
    one = np.exp(float(m) - float(lse))
    two = np.exp((float(m) - float(m)) - float(logd))
    assert abs(two * v - 1) < 2.0 ** -21
    if abs(offset) < 2.0 ** 24:
        assert abs(one * v - 1) <= abs(float(lse)) * 2.0 ** -24 + 2.0 ** -21
    else:
        assert one == 1.0


@pytest.mark.parametrize("s,want", [(2.3e38, (OK, DEVICE)), (2.5e38, VALUE), (3.4e38, VALUE), (1e-45, (OK, DEVICE))])
def test_the_largest_inverse_temperatures(lib, s, want):  # noqa: F811
    # s log2(e), the kernels' factor, has to be finite: infinite, it makes 0 times infinity of the row's maximum
    want = want if isinstance(want, tuple) else (want,)
    assert lib.logprob_fwd(A, 2 * A, 3 * A, 4 * A, 4, 8, s, 0, None) in want
    assert lib.logprob_bwd(A, 2 * A, 3 * A, 4 * A, 5 * A, 4, 8, s, 0, None) in want
    assert lib.policy_loss(A, 2 * A, 3 * A, 4 * A, None, None, 0.2, 0.2, 0.0, s, None, 5 * A, 6 * A, 7 * A, 4, 8, 0, 8 * A, 16, None) in want
