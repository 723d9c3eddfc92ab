"""One-query attention over the longest contexts that a block table can name: 2^31 - 1 tokens, on two pages."""
import numpy as np
import pytest
import torch

import mixer_refs as R
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 128, 2 ** 31 - 15])
def test_decode_of_the_longest_lengths(P, t, n):
    """All pages but the last are page 0.  The last token decides head 0 by its key alone; the others weigh every token
    alike up to their scores.  Bound: a warp adds some 57,000 tiles of 16 tokens one after another, in three products
    each at most (2^-23 of the sum a time), and four probabilities a tile and thread (2^-24 each): 57,000 x 5 x 2^-23 =
    3.4e-2 of sum p |v|; where one token holds the whole sum, 2^-10 of d code (p d in fp16) and half a step."""
    rng = np.random.default_rng(n % 1000)
    D, Hq, page, scale = 128, 4, 4096, 0.1
    C = R.Cache(rng, 2, 1, D, page)
    C.m[1] = (C.m[1].astype(np.float32) + 4.0).astype(np.float16)
    last = (n - 1) % page
    C.d[0][1, 0, last // 16, last % 16, 0], C.m[0][1, 0, last // 16, last % 16, 0] = 0, 100
    C.pack()
    q = torch.tensor(rng.standard_normal((2, Hq, D))).to(t)
    q[0, :, :32] = 0
    q[0, 0, :32] = 1
    pages = (n - 1) // page + 1
    tab = torch.zeros(2, 2 ** 31 // page, dtype=torch.int32)
    tab[0, pages - 1] = 1
    lens = [n, 130]
    cache, status = torch.tensor(C.bytes).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0).cuda()
    ws = torch.empty(P.redlite_kv4_decode_workspace_bytes(2, Hq, 1, D), dtype=torch.uint8, device="cuda")
    assert P.redlite_kv4_decode(q.cuda(), cache, page, tab.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), out, ws,
                                scale, status) == P.REDLITE_OK
    assert int(status) == 0
    got, qn = out.double().cpu().numpy(), q.double().numpy()
    k, v = (np.concatenate([C.values(w, [0], page, 0), C.values(w, [1], last + 1, 0)]) for w in range(2))
    often = np.concatenate([np.full(page, np.log(pages - 1.0)), np.zeros(last + 1)])
    for h in range(Hq):
        p = R.softmax(scale * (k @ qn[0, h]) + often)
        ref, W = p @ v, p @ np.abs(v)
        lim = 3.4e-2 * W if h else 2.0 ** -10 * 8 * 0.4 + 2.0 ** -8 * W
        assert (np.abs(got[0, h] - ref) <= lim).all(), (h, float((np.abs(got[0, h] - ref) / lim).max()))
        p = R.softmax(scale * (C.values(0, [0], 130, 0) @ qn[1, h]))
        v1 = C.values(1, [0], 130, 0)
        assert (np.abs(got[1, h] - p @ v1) <= 2.0 ** -7 * (p @ np.abs(v1))).all()
