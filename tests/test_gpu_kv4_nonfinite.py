"""One-query attention over the 4-bit cache where something that counts is a NaN: softmax of a NaN is NaN, whichever
warp or block met it, and nothing else changes."""
import numpy as np
import pytest
import torch

import mixer_refs as R
import test_gpu_kv4 as TK
import test_gpu_mixer_edges as TE
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu
NAN = float("nan")


def _expect(out, nan, C, tab, q, lens, scale):
    """`nan` [B, Hq, D] where the definition gives NaN; the rest against the reference of the finite inputs."""
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), nan)
    if q.dtype == torch.float32:
        ref, tol = TK._reference(C, tab, q, lens, scale)
        lim = tol + np.abs(ref) * R.HALF_ULP[q.dtype] * 1.001
    else:
        ref, lim = TE._reference16(C, tab, q, lens, scale, q.dtype)
    assert (np.abs(got - ref)[~nan] <= np.broadcast_to(lim, ref.shape)[~nan]).all()


def _spoil(C, tab, which, b, token, head, group):
    """What append stores for a group that holds a NaN."""
    at = (tab[b, token // C.page], head, token % C.page // 16, token % 16, group)
    C.d[which][at] = C.m[which][at] = np.nan


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
@pytest.mark.parametrize("D,Hq,Hk,page,lens", [
    (256, 16, 2, 64, [1]),
    (128, 8, 2, 16, [16, 17, 0, 1]),
    (256, 24, 2, 32, [700, 40, 129]),  # 12 query heads per key/value head
    (128, 4, 1, 64, [5000]),           # cut over many blocks
])
def test_a_nan_in_a_query(P, t, D, Hq, Hk, page, lens):
    rng = np.random.default_rng(D + sum(lens))
    C, tab, q = TK._decode_case(P, rng, t, D, Hq, Hk, page, lens)
    bad = q.clone()
    nan = np.zeros(q.shape, bool)
    for b, n in enumerate(lens):
        h = (3 * b + 1) % Hq
        bad[b, h, 37 * (b + 1) % D] = NAN
        nan[b, h] = n > 0
    _expect(TK._call(P, C, tab, bad, lens, 0.1), nan, C, tab, q, lens, 0.1)
    # every element of every head
    out = TK._call(P, C, tab, torch.full_like(q, NAN), lens, 0.1)
    for b, n in enumerate(lens):
        assert bool(torch.isnan(out[b]).all()) if n else bool((out[b] == 0).all())


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
@pytest.mark.parametrize("D,lens,tokens", [
    (128, [1, 17, 17], [0, 16, 3]),         # alone; alone in its tile; beside finite ones
    (256, [40, 16, 130], [32, 0, 129]),
    (128, [6000, 33], [5999, 16]),          # the newest token of a sequence that is cut over blocks
    (256, [3000], [1500]),
])
def test_a_nan_in_a_key(P, t, D, lens, tokens):
    rng = np.random.default_rng(D + sum(lens))
    Hq, Hk, page = 8, 2, 32
    C, tab, q = TK._decode_case(P, rng, t, D, Hq, Hk, page, lens)
    clean = TK._call(P, C, tab, q, lens, 0.1)
    ref = R.Cache.__new__(R.Cache)
    ref.__dict__.update(C.__dict__, d=[x.copy() for x in C.d], m=[x.copy() for x in C.m])
    nan = np.zeros(q.shape, bool)
    for b, i in enumerate(tokens):
        _spoil(C, tab, 0, b, i, b % Hk, b % (D // 32))
        nan[b, 4 * (b % Hk):4 * (b % Hk) + 4] = True
    C.pack()
    out = TK._call(P, C, tab, q, lens, 0.1)
    _expect(out, nan, ref, tab, q, lens, 0.1)
    # heads of the other key/value head keep their bits
    assert torch.equal(out[~torch.tensor(nan).cuda()], clean[~torch.tensor(nan).cuda()])


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
@pytest.mark.parametrize("D,lens", [(128, [4000, 50]), (256, [16, 2500])])
def test_keys_that_are_all_nan(P, t, D, lens):
    rng = np.random.default_rng(D)
    C, tab, q = TK._decode_case(P, rng, t, D, 4, 1, 64, lens)
    nan = np.zeros(q.shape, bool)
    nan[0] = True
    ref = R.Cache.__new__(R.Cache)
    ref.__dict__.update(C.__dict__, d=[x.copy() for x in C.d], m=[x.copy() for x in C.m])
    for i in range(lens[0]):
        _spoil(C, tab, 0, 0, i, 0, i % (D // 32))
    C.pack()
    _expect(TK._call(P, C, tab, q, lens, 0.1), nan, ref, tab, q, lens, 0.1)


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
@pytest.mark.parametrize("D,n", [(128, 17), (256, 2000)])
def test_a_nan_in_a_value_stays_in_its_group(P, t, D, n):
    rng = np.random.default_rng(D + n)
    C, tab, q = TK._decode_case(P, rng, t, D, 8, 2, 16, [n, 30])
    ref = R.Cache.__new__(R.Cache)
    ref.__dict__.update(C.__dict__, d=[x.copy() for x in C.d], m=[x.copy() for x in C.m])
    _spoil(C, tab, 1, 0, n - 1, 1, 2)
    C.pack()
    nan = np.zeros(q.shape, bool)
    nan[0, 4:, 64:96] = True
    _expect(TK._call(P, C, tab, q, [n, 30], 0.1), nan, ref, tab, q, [n, 30], 0.1)


@gpu
@pytest.mark.parametrize("t", TK.TYPES)
def test_a_nan_token_that_was_appended(P, t):
    """Seventeen tokens, the newest key a NaN: as from append, alone in its tile."""
    rng = np.random.default_rng(3)
    k, v = (torch.tensor(rng.standard_normal((17, 2, 128))).to(t).cuda() for _ in range(2))
    k[16, 1, 5] = NAN
    q = torch.tensor(rng.standard_normal((1, 4, 128))).to(t).cuda()
    cache = torch.zeros(2, 2, 1, 2560, dtype=torch.uint8, device="cuda")
    tab = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert P.redlite_kv4_append(k, v, R.cu([17]), z, tab, cache, 16) == P.REDLITE_OK
    ws = torch.empty(P.redlite_kv4_decode_workspace_bytes(1, 4, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    for n in (16, 17):
        assert P.redlite_kv4_decode(q, cache, 16, tab, z + n, out, ws, 0.1) == P.REDLITE_OK
        assert bool(torch.isfinite(out[:, :2]).all())
        assert bool((torch.isnan(out[:, 2:]) if n == 17 else torch.isfinite(out[:, 2:])).all())
