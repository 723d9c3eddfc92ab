"""One-query attention over the 4-bit cache for 16-bit activations whose value steps are small: the products of a
probability with a step are held relative to the largest ones, not to fp16's smallest number."""
import numpy as np
import pytest
import torch

import mixer_refs as R
import test_gpu_kv4 as TK
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu


def _reference(C, tab, q, lens, scale):
    """(out, bound) in 64 bits.  Per token: p and p d are rounded to fp16, 2^-10 of p d in all, or 2^-22 of the largest
    p times the head's largest |d| where that is more; both times |code - 8| <= 8.  Their signs are random (codes
    are), so a sum of independent terms c_t passes 6 sqrt(sum c_t^2) once in 10^7.  Besides: p m in two fp16 parts of p
    (2^-22 of it, or 2^-25 of a largest p of at least 2^6), scores and sums in fp32 as in the fp32 form."""
    B, Hq, D = q.shape
    qn = q.double().cpu().numpy()
    out, lim = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b, n in enumerate(lens):
        for h in range(Hq):
            kh = h // (Hq // C.heads)
            pages = tab[b, :-(-n // C.page)]
            k, v = C.values(0, pages, n, kh), C.values(1, pages, n, kh)
            p = R.softmax(scale * (k @ qn[b, h]))
            out[b, h] = p @ v
            qa = np.abs(qn[b, h]).reshape(-1, 32).sum(-1)
            d, m = C.steps(0, pages, n, kh)
            A = scale * (qa * (32 * np.abs(d) + np.abs(m - 16 * d))).sum(-1).max()
            d, m = C.steps(1, pages, n, kh)
            c = 8 * (2.0 ** -10 * p[:, None] * d + 2.0 ** -22 * p.max() * d.max())
            g = 6 * np.sqrt((c * c).sum(0)) + 2.0 ** -20 * (p @ (8 * d + np.abs(m + 8 * d) + np.abs(m)))
            g = g + n * 2.0 ** -31 * p.max() * np.abs(m + 8 * d).max()
            lim[b, h] = np.repeat(g, 32) + 2 * np.abs(v).max() * 2.0 ** -20 * (A + 1)
    return out, lim + (np.abs(out) + lim) * R.HALF_ULP[q.dtype] * 1.001


@gpu
@pytest.mark.parametrize("D,Hq,Hk", [(256, 8, 1), (128, 8, 2)])
@pytest.mark.parametrize("size,end", [(2.0 ** -5, 1), (2.0 ** -12, 1), (2.0 ** -15, 1), (2.0 ** -18, 1), (2.0 ** -21, 1),
                                      (2.0 ** -20, 2.0 ** 22), (1.0, 2.0 ** -20)])
def test_decode_with_small_steps(P, D, Hq, Hk, size, end):
    """30,000 tokens, scores of deviation 2; steps of one size, or growing or falling along the sequence."""
    rng = np.random.default_rng(D)
    lens, page, t = [30000, 77, 16], 64, torch.bfloat16
    C, tab, q = TK._decode_case(P, rng, t, D, Hq, Hk, page, lens, qmag=1.0)
    place = np.zeros((C.n_pages, page))
    for b, n in enumerate(lens):
        for i in range(n):
            place[tab[b, i // page], i % page] = i / n
    f = size * end ** place.reshape(C.n_pages, 1, -1, 16, 1)
    d = C.d[1].astype(np.float64) / 0.4
    C.d[1] = (d * f).astype(np.float16)
    C.m[1] = np.clip(-7.5 * d * f + 0.3 * f * rng.standard_normal(d.shape), -6e4, 6e4).astype(np.float16)
    C.pack()
    # scores: unit keys have entries of deviation about 1.2
    scale = 2.0 / (1.2 * np.sqrt(D))
    out = TK._call(P, C, tab, q, lens, scale).double().cpu().numpy()
    ref, lim = _reference(C, tab, q, lens, scale)
    assert np.isfinite(out).all()
    assert (np.abs(out - ref) <= lim).all(), float((np.abs(out - ref) / lim).max())
