"""Prompt attention where values are not finite: what a query does not see changes neither results nor, by much, the
time; what it sees decides its columns."""
import numpy as np
import pytest
import torch

import mixer_refs as R
import test_gpu_attn as TA
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu
BAD = [float("nan"), float("inf"), float("-inf")]


def _time(f, n=5):
    f()
    torch.cuda.synchronize()
    best = float("inf")
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@gpu
@pytest.mark.parametrize("t", TA.TYPES)
@pytest.mark.parametrize("D,Hq,Hk", [(256, 16, 2), (128, 4, 4), (128, 6, 2)])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([37, 5], [37, 70]), ([130, 1, 64], [130, 129, 64]), ([65], [191]),
                                   ([20], [3])])
def test_values_behind_a_sequence(P, t, D, Hq, Hk, lq, lk):
    """Every sequence has rows behind it in its buffer that hold NaN and infinities: the bits of a buffer of zeros."""
    rng = np.random.default_rng(D + sum(lk))
    gap = 140
    q, _, _ = TA._inputs(rng, t, sum(lq), 1, Hq, Hk, D)
    outs = []
    for bad in (False, True):
        out = torch.full_like(q, 9.0)
        a = 0
        for nq, nk in zip(lq, lk):
            r2 = np.random.default_rng(nk)
            _, k, v = TA._inputs(r2, t, 1, nk + gap, Hq, Hk, D)
            k[nk:], v[nk:] = 0, 0
            if bad:
                for i in range(gap):
                    v[nk + i], k[nk + i] = BAD[i % 3], BAD[i % 3]
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            assert P.redlite_attn_prefill(q[a:a + nq], k, v, R.cu([nq]), R.cu([nk]), out[a:a + nq], 0.1,
                                          status) == P.REDLITE_OK
            assert int(status) == 0
            ref, lim = TA._reference(TA._host(q[a:a + nq]), TA._host(k)[:nk], TA._host(v)[:nk], [nq], [nk], 0.1, t)
            TA._check(out[a:a + nq], ref, lim)
            a += nq
        outs.append(out)
    assert torch.equal(*outs)


@gpu
@pytest.mark.parametrize("t", TA.TYPES)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("val", BAD)
def test_one_bad_value_decides_its_column_alone(P, t, D, val):
    """A value that some queries see and others do not, in one column of one head."""
    rng = np.random.default_rng(D)
    n, at = 300, 141
    q, k, v = TA._inputs(rng, t, n, n, 4, 2, D)
    clean = torch.empty_like(q)
    assert P.redlite_attn_prefill(q, k, v, R.cu([n]), R.cu([n]), clean, 0.1) == P.REDLITE_OK
    v[at, 1, 77] = val
    out = torch.empty_like(q)
    assert P.redlite_attn_prefill(q, k, v, R.cu([n]), R.cu([n]), out, 0.1) == P.REDLITE_OK
    got, base = out.float(), clean.float()
    assert bool((~torch.isfinite(got[at:, 2:, 77])).all())
    if val != val:
        assert bool(torch.isnan(got[at:, 2:, 77]).all())
    got[at:, 2:, 77] = base[at:, 2:, 77]
    # rows that do not see it: as if it were not there, up to the rounding of p in the one column
    ref, lim = TA._reference(TA._host(q)[at - 20:at], TA._host(k)[:at], TA._host(v)[:at], [20], [at], 0.1, t)
    TA._check(out[at - 20:at], ref, lim)
    got[:at, 2:, 77] = base[:at, 2:, 77]
    assert torch.equal(got, base)


@gpu
@pytest.mark.parametrize("t", TA.TYPES)
@pytest.mark.parametrize("D", [128, 256])
def test_a_score_of_minus_infinity_has_no_weight(P, t, D):
    """An infinite key element against a negative query element: as if the key were not there; zeros where all are."""
    rng = np.random.default_rng(D)
    q, k, v = TA._inputs(rng, t, 3, 150, 4, 2, D)
    q[:, :, 0] = -1
    keep = np.ones(150, bool)
    keep[[0, 70, 149]] = False
    k[torch.tensor(~keep).cuda(), :, 0] = float("inf")
    out = torch.empty_like(q)
    assert P.redlite_attn_prefill(q[2:], k, v, R.cu([1]), R.cu([150]), out[2:], 0.1) == P.REDLITE_OK
    ref, lim = TA._reference(TA._host(q)[2:], TA._host(k)[keep], TA._host(v)[keep], [1], [147], 0.1, t)
    TA._check(out[2:], ref, lim)
    k[:, :, 0] = float("inf")
    assert P.redlite_attn_prefill(q, k, v, R.cu([3]), R.cu([150]), out, 0.1) == P.REDLITE_OK
    assert bool((out == 0).all())


@gpu
@pytest.mark.parametrize("where", ["behind", "key", "first value", "all values"])
def test_time_with_values_that_are_not_finite(P, where):
    """A prompt over a long context: not an order of magnitude slower for a NaN behind it, in a key or in its values."""
    nq, nk, D = 512, 8192, 256
    q = torch.randn(nq, 16, D, device="cuda").bfloat16()
    k, v = (torch.randn(nk + 100, 2, D, device="cuda").bfloat16() for _ in range(2))
    cq, ck = R.cu([nq]), R.cu([nk - 3])
    out = torch.empty_like(q)

    def call():
        assert P.redlite_attn_prefill(q, k, v, cq, ck, out, 0.1) == P.REDLITE_OK

    base = _time(call)
    if where == "behind":
        k[nk - 3:], v[nk - 3:] = float("nan"), float("nan")
    elif where == "key":
        k[5, 0, 3] = float("nan")
    elif where == "first value":
        v[0, :, 3] = float("nan")
    else:
        v[:, 1] = float("nan")
    slow = _time(call)
    assert slow <= 8 * base, (base, slow)
