"""Causal attention over packed prompts against a 64-bit reference."""
import ctypes

import numpy as np
import pytest
import torch

import mixer_refs as R

gpu = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def P():
    from routed_expert_ffn_iq2_b200 import build

    build.build()
    import routed_expert_ffn_iq2_b200 as P

    return P


def test_refusals_before_device_work(P):
    L, p = P.lib(), ctypes.c_void_p(0x10000)

    def call(dtype=1, q=p, qs=4096, k=p, ks=512, vs=512, cu=p, n=1, nq=4, nk=4, Hq=16, Hk=2, D=256, scale=1.0, out=p,
             os=4096):
        return L.redlite_attn_prefill(dtype, q, qs, k, ks, p, vs, cu, p, n, nq, nk, Hq, Hk, D, scale, out, os, None, None)

    assert call(n=0) == P.REDLITE_OK and call(nq=0) == P.REDLITE_OK
    for kw in (dict(dtype=3), dict(dtype=-1), dict(n=-1), dict(nq=-1), dict(nk=-1), dict(Hq=15), dict(Hk=0), dict(Hq=0),
               dict(q=None), dict(k=None), dict(cu=None), dict(out=None), dict(qs=4095), dict(qs=4092), dict(ks=256),
               dict(vs=516), dict(os=8), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(q=ctypes.c_void_p(0x10008)), dict(out=ctypes.c_void_p(0x10002))):
        assert call(**kw) == P.REDLITE_EINVAL, kw
    for kw in (dict(dtype=0), dict(D=64), dict(D=192), dict(D=512)):
        assert call(**kw) == P.REDLITE_EUNSUPPORTED, kw


def test_binding_refuses_what_does_not_fit_together(P):
    q, k = torch.zeros(4, 4, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    # tensors in host memory
    assert P.redlite_attn_prefill(q, k, k, cu, cu, q, 1.0) == P.REDLITE_EINVAL


def _reference(q, k, v, lq, lk, scale, t):
    """(out, bound) in 64 bits.  Bound, with p the probabilities, W = sum p |v| and V = max |v| of the row:
      - p is rounded to the type: at most half a step each, u W (fp16 below 2^-14: 2^-25 of a largest p of at
        least 1, for each of n keys: n 2^-25 V);
      - scores: products of 16-bit numbers are exact in fp32, their sum of D terms is off by at most D / 16
        steps of 2^-22 of A = scale sum |q| |k| (a tensor-core step adds 16 products), then two fp32 roundings
        of log2 e s and the exponential's 2^-22: a change e of all exponents moves the output by 2 e V;
      - the sums over n keys: n / 16 steps of 2^-22 of W, the same for the sum of p and one division;
      - half a step of the output type."""
    u = R.HALF_ULP[t]
    Hq, D = q.shape[1:]
    r = Hq // k.shape[1]
    out, lim = np.zeros(q.shape), np.zeros(q.shape)
    a = b = 0
    for nq, nk in zip(lq, lk):
        for h in range(Hq):
            kk, vv = k[b:b + nk, h // r], v[b:b + nk, h // r]
            for i in range(nq):
                n = min(nk, max(0, i + nk - nq + 1))
                if n == 0:
                    continue
                z = scale * (kk[:n] @ q[a + i, h])
                p = R.softmax(z)
                o = p @ vv[:n]
                W, V = p @ np.abs(vv[:n]), np.abs(vv[:n]).max()
                A = scale * (np.abs(kk[:n]) @ np.abs(q[a + i, h])).max()
                e = 2.0 ** -22 * (A * (D / 16 + 4) + 2)
                s = u * W + n * 2.0 ** -25 * V + 2 * e * V + 2.0 ** -22 * (n / 8 + 4) * W
                out[a + i, h], lim[a + i, h] = o, s + (np.abs(o) + s) * u
        a, b = a + nq, b + nk
    return out, lim


def _inputs(rng, t, nq, nk, Hq, Hk, D, joint=False):
    q, k, v = (torch.tensor(rng.standard_normal(s)).to(t).cuda() for s in ((nq, Hq, D), (nk, Hk, D), (nk, Hk, D)))
    if joint:
        x = torch.cat([q, k, v], 1)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    return q, k, v


def _host(x):
    return x.double().cpu().numpy()


def _check(out, ref, lim):
    got = _host(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= lim).all(), float((np.abs(got - ref) / np.maximum(lim, 1e-300)).max())


@gpu
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("D,Hq,Hk,lq,lk", [
    (128, 1, 1, [1], [1]),
    (256, 2, 2, [1], [1]),
    (128, 8, 2, [5], [5]),
    (256, 16, 2, [37, 5, 1], [37, 5, 1]),
    (128, 4, 4, [127, 0, 128, 129], [127, 0, 128, 129]),
    (256, 4, 2, [130, 1], [130, 1]),
    (128, 6, 2, [70, 3], [200, 131]),          # three query heads each: no group; keys from an earlier part
    (256, 12, 1, [20, 0, 33], [148, 50, 33]),  # groups of four
    (128, 16, 1, [9, 4, 6, 5], [3, 0, 7, 4]),  # fewer keys than queries, and none
    (256, 3, 3, [2, 300], [1, 280]),
    (128, 32, 1, [260], [420]),
    (128, 64, 1, [3], [130]),                  # groups of 64: two tokens per tile
])
def test_matches_reference(P, t, D, Hq, Hk, lq, lk):
    rng = np.random.default_rng(D + Hq + sum(lk))
    q, k, v = _inputs(rng, t, sum(lq), sum(lk), Hq, Hk, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    assert P.redlite_attn_prefill(q, k, v, R.cu(lq), R.cu(lk), out, 2 * D ** -0.5, status) == P.REDLITE_OK
    _check(out, *_reference(_host(q), _host(k), _host(v), lq, lk, 2 * D ** -0.5, t))
    assert int(status) == 0


@gpu
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("order", [1, -1])
def test_growing_and_falling_scores(P, t, D, order):
    """Keys whose scores climb (or fall) by hundreds along the sequence: the running reference moves at every step."""
    rng = np.random.default_rng(D)
    n, Hq = 400, 2
    q, k, v = _inputs(rng, t, n, n, Hq, 1, D)
    ramp = torch.linspace(0, 40, n, device="cuda")[:, None]
    q[:, :, 0] = 4.0
    k[:, :, 0] = (ramp if order > 0 else ramp.flip(0)).to(t)
    out = torch.empty_like(q)
    assert P.redlite_attn_prefill(q, k, v, R.cu([n]), R.cu([n]), out, 1.0) == P.REDLITE_OK
    _check(out, *_reference(_host(q), _host(k), _host(v), [n], [n], 1.0, t))


@gpu
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("D", [128, 256])
def test_masked_places_have_no_effect(P, t, D):
    """NaN, infinities and the type's lowest value in keys and values that a query does not see, in the same tile,
    in the next sequence and behind the last one."""
    rng = np.random.default_rng(1)
    lq, lk, Hq, Hk = [40, 25], [40, 60], 4, 2
    q, k, v = _inputs(rng, t, 70, 110, Hq, Hk, D)
    cq, ck = R.cu(lq), R.cu(lk)
    clean = torch.full_like(q, 9.0)
    assert P.redlite_attn_prefill(q, k, v, cq, ck, clean, 0.1) == P.REDLITE_OK
    ref, lim = _reference(_host(q)[:65], _host(k)[:100], _host(v)[:100], lq, lk, 0.1, t)
    _check(clean[:65], ref, lim)
    low = torch.finfo(t).min
    bad = [float("nan"), float("inf"), float("-inf"), low]
    for x, y in ((k, v), (v, k)):
        for i, val in enumerate(bad):
            x[30 + i, i % Hk, i] = val          # seen by queries 30 + i .. of the first sequence
            x[100 + i] = val                    # behind the last sequence
            q[65 + i] = val
    out = torch.full_like(q, 9.0)
    assert P.redlite_attn_prefill(q, k, v, cq, ck, out, 0.1) == P.REDLITE_OK
    _check(out[:30], ref[:30], lim[:30])
    _check(out[40:65], ref[40:], lim[40:])
    assert bool((out[65:] == 9.0).all())
    # who sees the NaN gives NaN, in the heads of its key/value head
    assert bool(torch.isnan(out[30:40, :Hq // Hk]).all())
    _check(out[30, Hq // Hk:], ref[30, Hq // Hk:], lim[30, Hq // Hk:])


@gpu
def test_bad_offsets_are_reported(P):
    rng = np.random.default_rng(2)
    q, k, v = _inputs(rng, torch.bfloat16, 60, 60, 4, 2, 128)
    base = torch.zeros_like(q)
    assert P.redlite_attn_prefill(q, k, v, R.cu([20, 20, 20]), R.cu([20, 20, 20]), base, 0.1) == P.REDLITE_OK
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = [0, 20, 40, 60]
    for cq, ck, broken in (([0, 20, 40, 61], good, [2]), ([-1, 20, 40, 60], good, [0]), (good, [0, 20, 40, 61], [2]),
                           (good, [0, 20, 10, 60], [1, 2]), ([0, 20, 2147483647, 60], good, [1, 2]),
                           (good, [-2147483648, 20, 40, 60], [0])):
        status.zero_()
        out = torch.full_like(q, 9.0)
        c0, c1 = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cq, ck))
        assert P.redlite_attn_prefill(q, k, v, c0, c1, out, 0.1, status) == P.REDLITE_OK
        assert int(status) == P.REDLITE_STATUS_BAD_LENGTH
        for s in range(3):
            if s not in broken:
                assert torch.equal(out[20 * s:20 * s + 20], base[20 * s:20 * s + 20]), (cq, ck, s)


@gpu
def test_streams_graphs_strides(P):
    rng = np.random.default_rng(3)
    lens = [300, 1, 0, 77]
    q, k, v = _inputs(rng, torch.bfloat16, 378, 378, 16, 2, 256)
    cu = R.cu(lens)
    base = torch.zeros_like(q)
    assert P.redlite_attn_prefill(q, k, v, cu, cu, base, 0.07) == P.REDLITE_OK
    x = torch.cat([q, k, v], 1)
    wide = torch.full((378, 20, 256), 4.0, dtype=q.dtype, device="cuda")
    assert P.redlite_attn_prefill(x[:, :16], x[:, 16:18], x[:, 18:], cu, cu, wide[:, 2:18], 0.07) == P.REDLITE_OK
    assert torch.equal(wide[:, 2:18], base)
    assert bool((wide[:, :2] == 4).all()) and bool((wide[:, 18:] == 4).all())
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        assert P.redlite_attn_prefill(q, k, v, cu, cu, out, 0.07) == P.REDLITE_OK
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    assert torch.equal(out, base)
    cu.copy_(torch.tensor([0, 2, 130, 200, 370], dtype=torch.int32))
    out.fill_(5.0)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    n = [2, 128, 70, 170]
    _check(out[:370], *_reference(_host(q)[:370], _host(k), _host(v), n, n, 0.07, torch.bfloat16))
    assert bool((out[370:] == 5.0).all())
    # views of the wrong kind
    for a in ((q.transpose(0, 1), k, v, cu, cu, out), (q, k[:, :1], v, cu, cu, out), (q, k, v, cu, cu[:-1], out),
              (q, k, v, cu.long(), cu, out), (q, k.half(), v.half(), cu, cu, out), (q, k, v, cu, cu, out[:5])):
        assert P.redlite_attn_prefill(*a, 0.07) == P.REDLITE_EINVAL


@gpu
@pytest.mark.parametrize("t,D,Hq,Hk,lens", [(torch.float16, 128, 32, 8, [1000, 513, 0, 2047, 64, 333]),
                                            (torch.bfloat16, 128, 8, 8, [1, 200, 900]),
                                            (torch.bfloat16, 256, 16, 2, [700, 65, 1500, 128]),
                                            (torch.float16, 256, 4, 4, [300, 1, 800])])
def test_many_blocks_give_the_same_bits_every_time(P, t, D, Hq, Hk, lens):
    """Blocks that share multiprocessors, thirty times: nothing depends on how they fall, and rows of the ends of
    their tiles (the last keys are the last product's) are right."""
    rng = np.random.default_rng(D + Hq)
    n = sum(lens)
    q, k, v = _inputs(rng, t, n, n, Hq, Hk, D)
    cu = R.cu(lens)
    first = torch.empty_like(q)
    assert P.redlite_attn_prefill(q, k, v, cu, cu, first, 2 * D ** -0.5) == P.REDLITE_OK
    hq, hk, hv = _host(q), _host(k), _host(v)
    at = 0
    for m in lens:
        for i in sorted({0, m // 2, m - 17, m - 1} & set(range(m))):
            # the last query of a sequence cut off behind i sees what query i sees
            ref, lim = _reference(hq[at + i:at + i + 1], hk[at:at + i + 1], hv[at:at + i + 1], [1], [i + 1],
                                  2 * D ** -0.5, t)
            _check(first[at + i:at + i + 1], ref, lim)
        at += m
    out = torch.empty_like(q)
    for _ in range(30):
        out.fill_(9.0)
        assert P.redlite_attn_prefill(q, k, v, cu, cu, out, 2 * D ** -0.5) == P.REDLITE_OK
        assert torch.equal(out, first)


@gpu
def test_strided_rows_past_32_bits(P):
    """Rows of a joint tensor so wide that element offsets pass 2^31."""
    T, W = 40, 1 << 26
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(4)
    q, k, v = _inputs(rng, torch.bfloat16, T, T, 4, 1, 128)
    x[:, :512], x[:, W - 256:W - 128], x[:, W - 128:] = q.view(T, -1), k.view(T, -1), v.view(T, -1)
    out = torch.zeros_like(q)
    cu = R.cu([T])
    args = (x[:, :512].view(T, 4, 128), x[:, W - 256:W - 128].view(T, 1, 128), x[:, W - 128:].view(T, 1, 128))
    assert P.redlite_attn_prefill(*args, cu, cu, out, 0.1) == P.REDLITE_OK
    base = torch.zeros_like(q)
    assert P.redlite_attn_prefill(q, k, v, cu, cu, base, 0.1) == P.REDLITE_OK
    assert torch.equal(out, base)
