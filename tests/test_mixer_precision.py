"""The precision that the token mixers state for 32-bit results, as relative L2 errors against 64 bits.  The bounds are
first held against emulations of the arithmetic (on the CPU): that which the kernels use passes, one with fewer bits
does not."""
import numpy as np
import pytest
import torch

import mixer_refs as R
import test_gpu_delta as TD
import test_gpu_kv4 as TK
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu

# The delta rule: operands of every product are held to 2^-22 (two fp16 parts), so a product of two is off by 2^-21 of
# its terms.  State, K S, T (...) and the update follow each other: four products, whose errors the rule (a contraction)
# passes on without growth; terms are of random sign, so norms of errors and of results grow alike.  4 x 2^-21:
DELTA = 2.0 ** -19


def _l2(x, ref):
    return float(np.sqrt(((x - ref) ** 2).sum() / (ref ** 2).sum()))


def _bits(x, n):
    """x rounded to n significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, n)), e - n)


def _chunked(q, k, v, g, beta, state, scale, bits):
    """The chunked form of one head in 64 bits, operands of its products rounded to `bits` bits."""
    C = 64

    def mul(a, b):
        return _bits(a, bits) @ _bits(b, bits)

    S, out = state.copy(), np.zeros_like(v)
    for a in range(0, len(q), C):
        Q, K, V, b = q[a:a + C], k[a:a + C], v[a:a + C], beta[a:a + C, None]
        c = np.cumsum(g[a:a + C])[:, None]
        low = np.tril(np.ones((len(Q), len(Q))))
        decay = np.exp(np.where(low > 0, c - c.T, 0)) * low
        T = np.linalg.inv(np.eye(len(Q)) + np.tril(b * decay * mul(K, K.T), -1))
        D = mul(T, b * V - b * np.exp(c) * mul(K, S))
        out[a:a + C] = scale * (np.exp(c) * mul(Q, S) + mul(decay * mul(Q, K.T), D))
        S = np.exp(c[-1]) * S + mul(K.T, np.exp(c[-1] - c) * D)
    return out, S


def _delta_inputs(seed, t=torch.float32, lens=(700, 64, 130), hk=2, hv=4, dk=128, dv=128):
    rng = np.random.default_rng(seed)
    T = sum(lens)
    q, k, v = (torch.tensor(rng.standard_normal(s)).to(t) for s in ((T, hk, dk), (T, hk, dk), (T, hv, dv)))
    g = torch.tensor(-rng.exponential(1.0, (T, hv)) * 10 ** rng.uniform(-3, -1, (1, hv)), dtype=torch.float32)
    beta = torch.tensor(1 / (1 + np.exp(-rng.standard_normal((T, hv)))), dtype=torch.float32)
    state = torch.tensor(rng.standard_normal((len(lens), hv, dk, dv)), dtype=torch.float32)
    return list(lens), [q, k, v, g, beta], state


def test_the_delta_bound_tells_arithmetics_apart():
    lens, dev, state = _delta_inputs(1, lens=(700,), hk=1, hv=2)
    q, k, v, g, beta = [x.double().numpy() for x in dev]
    ref, S, _ = R.delta(q, k, v, g, beta, lens, state.double().numpy(), 0.1, 1e-6)
    qn, kn = (x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) for x in (q, k))
    for bits, good in ((24, True), (22, True), (17, False), (16, False), (11, False)):  # 16: two bf16 parts, 11: one fp16
        for h in range(2):
            o, s = _chunked(qn[:, 0], kn[:, 0], v[:, h], g[:, h], beta[:, h], state[0, h].double().numpy(), 0.1, bits)
            assert (_l2(o, ref[:, h]) <= DELTA) == good and (_l2(s, S[0, h]) <= DELTA) == good, bits


@gpu
@pytest.mark.parametrize("t", TD.TYPES)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("lens", [(700, 64, 130), (4000,), (1, 63, 0, 65)])
def test_delta_prefill_precision(P, t, dk, dv, lens):
    """States in 32 bits for every type of the activations, outputs for fp32 ones."""
    lens, dev, state = _delta_inputs(len(lens), t, lens, dk=dk, dv=dv)
    dev = [x.cuda() for x in dev]
    out_state = torch.zeros_like(state).cuda()
    out = TD._prefill(P, dev, R.cu(lens), state.cuda(), out_state, None, 0.1, 1e-6)
    ref, S, _ = R.delta(*[TD._host(x) for x in dev], lens, state.double().numpy(), 0.1, 1e-6)
    for s, n in enumerate(lens):
        for h in range(4):
            assert _l2(TD._host(out_state)[s, h], S[s, h]) <= DELTA
    if t == torch.float32:
        assert _l2(TD._host(out), ref) <= DELTA


# One query over the 4-bit cache, fp32: its products hold 24 bits and its sums are fp32, as those of the plain form in 32
# bits are, which rounds its values besides.  So its error is the plain form's; twice that for the order of the sums.
DECODE = 2.0


def _plain32(C, tab, q, lens, scale):
    out = np.zeros(q.shape)
    for b, n in enumerate(lens):
        for h in range(q.shape[1] if n else 0):
            kh = h // (q.shape[1] // C.heads)
            pages = tab[b, :-(-n // C.page)]
            k, v = (C.values(w, pages, n, kh).astype(np.float32) for w in range(2))
            z = (k * q[b, h].astype(np.float32)).sum(-1, dtype=np.float32) * np.float32(scale)
            p = np.exp(z - z.max())
            out[b, h] = (p[:, None] * v).sum(0, dtype=np.float32) / p.sum(dtype=np.float32)
    return out


def _exact(C, tab, q, lens, scale):
    return TK._reference(C, tab, torch.tensor(q), lens, scale)[0]


def _parts(x, n):
    """x in n bf16 parts, with what they leave out lost."""
    x = torch.tensor(x)
    y = torch.zeros_like(x)
    for _ in range(n):
        y += (x - y).bfloat16().double()
    return y.numpy()


def test_the_decode_bound_tells_arithmetics_apart():
    rng = np.random.default_rng(3)
    lens, page, D, Hk = [700], 64, 256, 1
    n, tab = R.table(rng, lens, page)
    C = R.Cache(rng, n, Hk, D, page)
    q = rng.standard_normal((1, 8, D)).astype(np.float32).astype(np.float64)
    exact = _exact(C, tab, q, lens, 0.1)
    plain = _l2(_plain32(C, tab, q, lens, 0.1), exact)
    pages = tab[0, :-(-700 // page)]
    d, m = C.steps(1, pages, 700, 0)
    v, k = C.values(1, pages, 700, 0), C.values(0, pages, 700, 0)
    code = (v.reshape(700, -1, 32) - m[..., None]) / d[..., None]
    for parts, good in ((3, True), (2, False), (1, False)):
        out = np.zeros_like(exact)
        for h in range(8):
            z = 0.1 * (k @ _parts(q[0, h], parts))
            p = np.exp(z - z.max())
            o = np.einsum("tg,tge->ge", _parts(16 * p[:, None] * d, parts), (code - 8) / 16)
            o = o + np.einsum("t,tg->g", _parts(p, parts), m + 8 * d)[:, None]
            out[0, h] = o.reshape(-1) / p.sum()
        assert (_l2(out, exact) <= DECODE * plain) == good, (parts, _l2(out, exact), plain)


@gpu
@pytest.mark.parametrize("D,Hq,Hk,lens", [(256, 16, 2, [700]), (128, 8, 1, [333, 17, 1000]), (128, 24, 2, [2500]),
                                          (256, 4, 4, [100, 5])])
def test_decode_precision(P, D, Hq, Hk, lens):
    rng = np.random.default_rng(D + Hq)
    scale = 1.5 * D ** -0.5
    C, tab, q = TK._decode_case(P, rng, torch.float32, D, Hq, Hk, 64, lens)
    out = TK._call(P, C, tab, q, lens, scale).double().cpu().numpy()
    qn = q.double().cpu().numpy()
    exact = _exact(C, tab, qn, lens, scale)
    assert _l2(out, exact) <= DECODE * _l2(_plain32(C, tab, qn, lens, scale), exact)
