"""Calls of the token mixers at the edges of what they take: many heads, many
sequences, magnitudes far apart, two calls at once."""
import numpy as np
import pytest
import torch

import mixer_refs as R
import test_gpu_attn as TA
import test_gpu_delta as TD
import test_gpu_kv4 as TK
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]


# --------------------------------------------------------------- append, load


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
@pytest.mark.parametrize("D,H", [(256, 20), (256, 8), (256, 9), (128, 33), (128, 16), (128, 15)])
def test_append_then_load_many_heads(P, t, D, H):
    """More heads than a block has rows, as many, and numbers that do not divide them."""
    rng = np.random.default_rng(D + H)
    lens, start, page = [3, 18], [14, 0], 16
    k, v, tab, cache = TK._fill(P, rng, t, D, H, page, lens, start, joint=H % 2 == 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, st = R.cu(lens), torch.tensor(start, dtype=torch.int32, device="cuda")
    assert P.redlite_kv4_append(k, v, cu, st, tab, cache, page, status) == P.REDLITE_OK
    ko, vo = (torch.zeros(21, H, D, device="cuda") for _ in range(2))
    assert P.redlite_kv4_load(cache, page, tab, cu, st, ko, vo, status) == P.REDLITE_OK
    for x, y in ((k, ko), (v, vo)):
        assert np.array_equal(y.cpu().numpy(), R.dequantise(*R.quantise(x.double().cpu().numpy())).astype(np.float32))
    # into 16 bits: the same values, rounded once
    kh, vh = (torch.zeros(21, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert P.redlite_kv4_load(cache, page, tab, cu, st, kh, vh, status) == P.REDLITE_OK
    assert torch.equal(kh, ko.bfloat16()) and torch.equal(vh, vo.bfloat16())
    assert int(status) == 0


@gpu
def test_append_rows_of_many_sequences(P):
    """One token each for 700 sequences, a few with two or none, in pages of their own."""
    rng = np.random.default_rng(1)
    lens = rng.choice([0, 1, 1, 1, 2], 700).tolist()
    start = rng.integers(0, 60, 700).tolist()
    k, v, tab, cache = TK._fill(P, rng, torch.float32, 128, 1, 16, lens, start)
    cu, st = R.cu(lens), torch.tensor(start, dtype=torch.int32, device="cuda")
    assert P.redlite_kv4_append(k, v, cu, st, tab, cache, 16) == P.REDLITE_OK
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    assert P.redlite_kv4_load(cache, 16, tab, cu, st, ko, vo) == P.REDLITE_OK
    for x, y in ((k, ko), (v, vo)):
        assert np.array_equal(y.cpu().numpy(), R.dequantise(*R.quantise(x.double().cpu().numpy())).astype(np.float32))


# --------------------------------------------------------------------- decode


def _reference16(C, tab, q, lens, scale, t):
    """(out, bound) of the decode for 16-bit activations, in 64 bits.  Besides the scores' bound of the fp32 form
    (2 max|v| 2^-20 (A + 1); a query's elements below 2^-30 of its largest count as that in A):
      - p and p d are rounded to fp16: 2^-10 of |p d (code - 8)|, code - 8 at most 8 in size; where they fall below
        fp16's normal range, 2^-25 of each token instead, times 8 (and times |d| where it is p).  p is relative to a
        reference that the largest score passes by 2^(room - 8) at least, room = 15 - log2 of the largest |d|
        (rounded up, 1 at least, 16 at most), so a normalised term is off by 2^-25 2^(8 - room);
      - p m is a product of two fp16 parts of p: the same 2^-25, times |m| + 8 |d|;
      - sums in fp32: 2^-20 of their terms;
      - half a step of the output (2^-25 below fp16's normal range)."""
    B, Hq, D = q.shape
    qn = q.double().cpu().numpy()
    out, lim = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b, n in enumerate(lens):
        for h in range(Hq if n else 0):
            kh = h // (Hq // C.heads)
            pages = tab[b, :-(-n // C.page)]
            k, v = C.values(0, pages, n, kh), C.values(1, pages, n, kh)
            p = R.softmax(scale * (k @ qn[b, h]))
            out[b, h] = p @ v
            qa = np.maximum(np.abs(qn[b, h]), 2.0 ** -30 * np.abs(qn[b, h]).max()).reshape(-1, 32).sum(-1)
            d, m = C.steps(0, pages, n, kh)
            A = scale * (qa * (32 * np.abs(d) + np.abs(m - 16 * d))).sum(-1).max()
            d, m = C.steps(1, pages, n, kh)
            d, big = np.abs(d), np.abs(d).max()
            room = 15 - min(16, max(1, int(np.floor(np.log2(max(big, 1e-30)))) + 1))
            small = n * 2.0 ** -25 * 2.0 ** (8 - room)
            g = 8 * 2.0 ** -10 * 1.001 * (p @ d) + small * (8 * (1 + big) + np.abs(m).max() + 8 * big)
            g = g + 2.0 ** -20 * (p @ (8 * d + np.abs(m + 8 * d) + np.abs(m)))
            lim[b, h] = np.repeat(g, 32) + 2 * np.abs(v).max() * 2.0 ** -20 * (A + 1)
    u = R.HALF_ULP[t]
    return out, lim + (np.abs(out) + lim) * u + 2.0 ** -25


def _check(out, ref, lim):
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= lim).all(), float((np.abs(got - ref) / lim).max())


@gpu
@pytest.mark.parametrize("t", HALVES)
@pytest.mark.parametrize("D,Hq,Hk", [(256, 16, 2), (128, 6, 2)])
@pytest.mark.parametrize("what", ["tiny", "two", "large", "growing", "falling", "mixed", "negative", "groups"])
def test_decode_steps_of_any_size(P, t, D, Hq, Hk, what):
    """Steps from 1e-4 to the thousands, alike, along the sequence or from token to token: p d stays in fp16."""
    rng = np.random.default_rng(D + len(what))
    lens, page = [700, 33, 130], 32
    C, tab, q = TK._decode_case(P, rng, t, D, Hq, Hk, page, lens, qmag=2.0)
    d = C.d[1].astype(np.float64) / 0.4                     # 0.125 .. 1
    m = C.m[1].astype(np.float64)
    place = np.zeros((C.n_pages, page))                     # 0 .. 1 along a sequence
    for b, n in enumerate(lens):
        for i in range(n):
            place[tab[b, i // page], i % page] = i / n
    place = place.reshape(C.n_pages, 1, -1, 16, 1)
    f = {"tiny": 1e-4, "two": 2.0, "large": 3500.0, "growing": 10.0 ** (6 * place - 2.5),
         "falling": 10.0 ** (3.5 - 6 * place), "mixed": 10.0 ** rng.uniform(-2, 3.5, d.shape[:4] + (1,)),
         "negative": -10.0 ** rng.uniform(-2, 3, d.shape), "groups": 10.0 ** rng.uniform(-1, 3, (D // 32,))}[what]
    C.d[1], C.m[1] = (d * f).astype(np.float16), np.clip(m * np.abs(f), -9000, 9000).astype(np.float16)
    if what == "negative":
        C.d[0] = np.where(rng.random(C.d[0].shape) < 0.5, -C.d[0], C.d[0])
    C.pack()
    scale = D ** -0.5
    _check(TK._call(P, C, tab, q, lens, scale), *_reference16(C, tab, q, lens, scale, t))


@gpu
@pytest.mark.parametrize("qmag,scale", [(1e30, 2e-31), (1e-30, 1e29), (1e-38, 1e37), (3e4, 1e-5)])
def test_decode_queries_of_any_size(P, qmag, scale):
    rng = np.random.default_rng(2)
    lens = [300, 0, 65]
    C, tab, q = TK._decode_case(P, rng, torch.bfloat16, 256, 4, 2, 64, lens, qmag=qmag)
    q[0, 1] = 0                      # a head without any
    q[0, 2, 17] = 0
    _check(TK._call(P, C, tab, q, lens, scale), *_reference16(C, tab, q, lens, scale, torch.bfloat16))


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
def test_decode_scores_far_apart(P, t):
    """Scores that climb or fall by hundreds along the sequence, so that the running reference moves at every tile."""
    rng = np.random.default_rng(3)
    lens, page = [500, 500], 64
    C, tab, q = TK._decode_case(P, rng, t, 128, 4, 1, page, lens)
    for b in range(2):
        for i in range(500):
            C.m[0][tab[b, i // page], 0, i % page // 16, i % 16, 0] = (i if b else 500 - i) / 32
    C.pack()
    q[:, :, :32] = 0.5
    if t == torch.float32:
        ref, tol = TK._reference(C, tab, q, lens, 1.0)
        lim = tol + np.abs(ref) * R.HALF_ULP[t] * 1.001
    else:
        ref, lim = _reference16(C, tab, q, lens, 1.0, t)
    _check(TK._call(P, C, tab, q, lens, 1.0), ref, lim)


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
@pytest.mark.parametrize("B,top", [(300, 40), (1200, 3), (257, 200)])
def test_decode_many_sequences(P, t, B, top):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, top, B).tolist()
    lens[-1] = lens[255] = 0
    C, tab, q = TK._decode_case(P, rng, t, 128, 2, 1, 16, lens)
    out = TK._call(P, C, tab, q, lens, 0.1)
    if t == torch.float32:
        ref, tol = TK._reference(C, tab, q, lens, 0.1)
        _check(out, ref, tol + np.abs(ref) * R.HALF_ULP[t] * 1.001)
    else:
        _check(out, *_reference16(C, tab, q, lens, 0.1, t))


# ------------------------------------------------------------------ attention


@gpu
@pytest.mark.parametrize("t", HALVES)
@pytest.mark.parametrize("D,n", [(128, 33), (256, 100), (128, 1100)])
def test_attention_over_many_sequences(P, t, D, n):
    rng = np.random.default_rng(n)
    lq = rng.choice([0, 0, 1, 2, 5], n)
    lk = lq + rng.choice([0, 0, 3, 40], n)
    lq[0] = lq[-1] = 0
    if n == 33:
        lq[31], lk[31], lq[32], lk[32] = 130, 130, 1, 7
    q, k, v = TA._inputs(rng, t, int(lq.sum()), int(lk.sum()), 2, 1, D)
    out = torch.full_like(q, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert P.redlite_attn_prefill(q, k, v, R.cu(lq), R.cu(lk), out, 0.1, status) == P.REDLITE_OK
    TA._check(out, *TA._reference(TA._host(q), TA._host(k), TA._host(v), lq, lk, 0.1, t))
    assert int(status) == 0


@gpu
@pytest.mark.parametrize("t,top", [(torch.bfloat16, 3e38), (torch.float16, 6e4)])
@pytest.mark.parametrize("D", [128, 256])
def test_attention_values_near_the_end_of_the_range(P, t, top, D):
    """Values whose unnormalised sums leave fp32 (bf16): their mean does not."""
    rng = np.random.default_rng(D)
    q, k, v = TA._inputs(rng, t, 150, 150, 4, 2, D)
    v[:, 0] = top                                             # all alike
    v[:, 1] = (top * torch.sign(v[:, 1].float())).to(t)       # of either sign
    out = torch.empty_like(q)
    assert P.redlite_attn_prefill(q, k, v, R.cu([150]), R.cu([150]), out, 0.05) == P.REDLITE_OK
    TA._check(out, *TA._reference(TA._host(q), TA._host(k), TA._host(v), [150], [150], 0.05, t))


@gpu
def test_attention_without_any_key(P):
    """Every sequence without keys, and no key rows at all: zeros."""
    q = torch.randn(7, 4, 128, device="cuda").bfloat16()
    k = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 9.0)
    assert P.redlite_attn_prefill(q, k, k, R.cu([3, 4]), R.cu([0, 0]), out, 1.0) == P.REDLITE_OK
    assert bool((out == 0).all())


# ----------------------------------------------------------------- delta rule


@gpu
@pytest.mark.parametrize("t", TD.TYPES)
def test_delta_many_sequences(P, t):
    """More sequences than a block has threads, of every number of chunks, a slot for each in any order."""
    rng = np.random.default_rng(4)
    n, hk, hv = 300, 1, 2
    lens = rng.choice([0, 1, 3, 17, 64, 65], n, p=[.2, .3, .2, .2, .05, .05])
    lens[[5, 99]] = 200, 130
    T = int(lens.sum())
    dev = TD._inputs(rng, t, T, hk, hv, 64, 64, True)
    pool = torch.tensor(rng.standard_normal((n, hv, 64, 64)), dtype=torch.float32).cuda()
    slots = torch.tensor(rng.permutation(n).astype(np.int32)).cuda()
    state = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = TD._prefill(P, dev, R.cu(lens), state, state, slots, 0.125, 1e-6, status)
    ref, S, big = R.delta(*[TD._host(x) for x in dev], lens, TD._host(pool[slots.long()]), 0.125, 1e-6)
    lim, slim = TD._limits(ref, big, lens, 0.125, 64, np.abs(TD._host(dev[2])).max(), t)
    assert (np.abs(TD._host(out) - ref) <= lim).all() and int(status) == 0
    assert (np.abs(TD._host(state[slots.long()]) - S) <= slim).all()


@gpu
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
def test_delta_rows_of_any_size(P, t, dk, dv):
    """Keys as given from 1e-6 to length 1, queries from 1e-8 to 1e8, values from 1e-4 to 1e4, updates switched off."""
    rng = np.random.default_rng(dk)
    lens, hk, hv = [150, 70], 2, 4
    T = sum(lens)
    q, k, v, g, beta = TD._inputs(rng, t, T, hk, hv, dk, dv, False)
    qs = 10.0 ** rng.uniform(-8, 8, (T, hk, 1))
    q = (q.double() * torch.tensor(qs).cuda()).to(t)
    k = (k.double() * torch.tensor(0.99 * 10.0 ** rng.uniform(-6, 0, (T, hk, 1))).cuda()).to(t)
    v = (v.double() * torch.tensor(10.0 ** rng.uniform(-4, 4, (T, hv, 1))).cuda()).to(t)
    k[3], q[4], v[5] = 0, 0, 0
    beta[20:90, 1] = 0
    beta[100, :] = 1
    dev = [q, k, v, g, beta]
    st = torch.tensor(rng.standard_normal((2, hv, dk, dv)), dtype=torch.float32).cuda()
    s = torch.zeros_like(st)
    out = TD._prefill(P, dev, R.cu(lens), st, s, None, 0.3, -1.0)
    ref, S, big = R.delta(*[TD._host(x) for x in dev], lens, TD._host(st), 0.3, -1.0)
    # the bound of a unit query, for the length each query has
    lim, slim = TD._limits(ref, big, lens, 0.3, dk, np.abs(TD._host(v)).max(), t)
    length = np.sqrt((TD._host(q) ** 2).sum(-1))
    tol = np.abs(ref) * R.HALF_ULP[t] * 1.001
    lim = (lim - tol) * np.repeat(length, hv // hk, 1)[..., None] + tol
    assert (np.abs(TD._host(out) - ref) <= lim).all()
    assert (np.abs(TD._host(s) - S) <= slim).all()
    # and the step, token by token from the first state
    a = st[:1].clone()
    for i in range(30):
        o = torch.zeros(1, hv, dv, dtype=t, device="cuda")
        assert P.redlite_delta_step(*[x[i:i + 1].contiguous() for x in dev], a, a, None, o, 0.3, -1.0) == P.REDLITE_OK
        assert (np.abs(TD._host(o)[0] - ref[i]) <= lim[i]).all()


# ----------------------------------------------------------- two calls at once


@gpu
def test_calls_on_two_streams_at_once(P):
    """Prompts on one stream, single tokens on the other, each with its own workspace: the bits of calls alone."""
    rng = np.random.default_rng(6)
    lens = [900, 64, 333]
    T = sum(lens)
    q, k, v = TA._inputs(rng, torch.bfloat16, T, T, 16, 2, 256)
    dev = TD._inputs(rng, torch.bfloat16, T, 2, 4, 128, 128, True)
    cu = R.cu(lens)
    cl = [3000, 1, 700, 2000]
    C, tab, q1 = TK._decode_case(P, rng, torch.bfloat16, 256, 16, 2, 64, cl)
    cache, tb = torch.tensor(C.bytes).cuda(), torch.tensor(tab).cuda()
    ln = torch.tensor(cl, dtype=torch.int32, device="cuda")
    one = [x[:4].contiguous() for x in dev]
    wd = torch.empty(P.redlite_delta_workspace_bytes(T, 3, 2, 4, 128, 128), dtype=torch.uint8, device="cuda")
    wk = torch.empty(P.redlite_kv4_decode_workspace_bytes(4, 16, 2, 256), dtype=torch.uint8, device="cuda")

    def outputs():
        return [torch.zeros_like(q), torch.zeros_like(dev[2]), torch.zeros(3, 4, 128, 128, device="cuda"),
                torch.zeros_like(q1), torch.zeros_like(one[2]), torch.zeros(4, 4, 128, 128, device="cuda")]

    def prompts(o, s):
        assert P.redlite_attn_prefill(q, k, v, cu, cu, o[0], 0.1, None, s) == P.REDLITE_OK
        assert P.redlite_delta_prefill(*dev, cu, None, o[2], None, o[1], wd, 0.1, 1e-6, None, s) == P.REDLITE_OK

    def tokens(o, s):
        assert P.redlite_kv4_decode(q1, cache, 64, tb, ln, o[3], wk, 0.1, None, s) == P.REDLITE_OK
        assert P.redlite_delta_step(*one, o[5], o[5], None, o[4], 0.1, 1e-6, None, s) == P.REDLITE_OK

    base = outputs()
    cur = torch.cuda.current_stream()
    prompts(base, cur)
    tokens(base, cur)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        got = outputs()
        torch.cuda.synchronize()
        prompts(got, a)
        tokens(got, b)
        torch.cuda.synchronize()
        for x, y in zip(base, got):
            assert torch.equal(x, y)
