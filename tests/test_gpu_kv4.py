"""The 4-bit key/value cache: append and load against the stored form's
definition (exact), one-query attention against a 64-bit reference."""
import ctypes

import numpy as np
import pytest
import torch

import mixer_refs as R

gpu = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def P():
    from routed_expert_ffn_iq2_b200 import build

    build.build()
    import routed_expert_ffn_iq2_b200 as P

    return P


# ------------------------------------------------------------- refusals (host)


def test_refusals_before_device_work(P):
    L, p = P.lib(), ctypes.c_void_p(0x10000)

    def append(dtype=0, k=p, ks=512, cu=p, n=1, T=1, H=2, D=256, page=64, width=4, pages=8, cache=p):
        return L.redlite_kv4_append(dtype, k, p, ks, 512, cu, p, n, T, H, D, page, p, width, pages, cache, None, None)

    assert append(T=0) == P.REDLITE_OK and append(n=0) == P.REDLITE_OK
    for kw in (dict(dtype=3), dict(T=-1), dict(n=-1), dict(H=0), dict(k=None), dict(cu=None), dict(cache=None),
               dict(ks=511), dict(ks=256), dict(width=0), dict(pages=0), dict(cache=ctypes.c_void_p(0x10008)),
               dict(k=ctypes.c_void_p(0x10004))):
        assert append(**kw) == P.REDLITE_EINVAL, kw
    for kw in (dict(D=64), dict(D=192), dict(page=8), dict(page=24), dict(page=8192)):
        assert append(**kw) == P.REDLITE_EUNSUPPORTED, kw
    assert append(dtype=1, ks=516) == P.REDLITE_EINVAL  # 1032 bytes: rows off their 16-byte boundaries

    def decode(dtype=1, q=p, qs=4096, n=1, Hq=16, Hk=2, D=256, page=64, width=4, pages=8, scale=1.0, ws=1 << 30,
               out=p):
        return L.redlite_kv4_decode(dtype, q, qs, n, Hq, Hk, D, p, page, p, width, pages, p, scale, out, 4096, p, ws,
                                    None, None)

    assert decode(n=0) == P.REDLITE_OK
    for kw in (dict(dtype=-1), dict(n=-1), dict(Hq=15), dict(Hk=0), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(out=None), dict(qs=4095),
               dict(width=0), dict(pages=0)):
        assert decode(**kw) == P.REDLITE_EINVAL, kw
    assert decode(D=512) == P.REDLITE_EUNSUPPORTED
    assert decode(ws=64) == P.REDLITE_ENOMEM
    assert P.redlite_kv4_page_bytes(2, 256, 64) == 2 * 4 * 5120
    assert P.redlite_kv4_page_bytes(2, 256, 40) == 0 and P.redlite_kv4_page_bytes(0, 256, 64) == 0
    assert P.redlite_kv4_decode_workspace_bytes(4, 16, 3, 256) == 0


# --------------------------------------------------------------- append, load


def _fill(P, rng, t, D, H, page, lens, start, joint=False, special=False):
    T = sum(lens)
    k = rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((1, H, D))) + rng.standard_normal((1, H, D))
    v = rng.standard_normal((T, H, D)) * 10.0 ** rng.uniform(-6, 3, (T, H, 1))
    if special:
        k[0, :, :32] = 0.25          # a constant group: step 0
        k[0, :, 32:64] = 0.0
        v[0, :, :32] = 1e-9          # below fp16: everything rounds to 0
        v[0, :, 32:64] = np.linspace(-1e5, 1e5, 32)  # clamped
        # quotients that end on .5: ties to even
        k[-1, :, :32] = np.concatenate([[0.0, 15.0], np.arange(15) + 0.5, np.arange(15)])
    kt, vt = torch.tensor(k).to(t).cuda(), torch.tensor(v).to(t).cuda()
    if joint:
        both = torch.cat([kt, vt], 1)
        kt, vt = both[:, :H], both[:, H:]
    n, tab = R.table(rng, [a + b for a, b in zip(start, lens)], page, spare=2)
    cache = torch.randint(0, 256, (n, H, page // 16, 20 * D), dtype=torch.uint8, device="cuda")
    return kt, vt, torch.tensor(tab).cuda(), cache


@gpu
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("D,H,page,lens,start,joint", [
    (256, 2, 64, [1], [0], False),
    (256, 2, 64, [1] * 5, [0, 63, 64, 127, 500], False),
    (128, 1, 16, [33, 0, 7, 1], [0, 5, 15, 16], True),
    (128, 8, 128, [130, 2], [127, 300], True),
    (256, 3, 32, [0, 47, 0, 65], [9, 31, 1, 0], False),
])
def test_append_then_load_is_exact(P, t, D, H, page, lens, start, joint):
    rng = np.random.default_rng(D + sum(lens))
    k, v, tab, cache = _fill(P, rng, t, D, H, page, lens, start, joint, special=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, st = R.cu(lens), torch.tensor(start, dtype=torch.int32, device="cuda")
    before = cache.clone()
    assert P.redlite_kv4_append(k, v, cu, st, tab, cache, page, status) == P.REDLITE_OK
    ko = torch.full((k.shape[0] + 2, H, D), 7.0, device="cuda")
    vo = ko.clone()
    assert P.redlite_kv4_load(cache, page, tab, cu, st, ko, vo, status) == P.REDLITE_OK
    for x, y in ((k, ko), (v, vo)):
        ref = R.dequantise(*R.quantise(x.double().cpu().numpy())).astype(np.float32)
        assert np.array_equal(y[:-2].cpu().numpy(), ref, equal_nan=True)
        assert bool((y[-2:] == 7.0).all())  # rows behind the last sequence
    # a second append of the same rows changes nothing; other tokens' bytes were left alone
    again = cache.clone()
    assert P.redlite_kv4_append(k, v, cu, st, tab, cache, page, status) == P.REDLITE_OK
    assert torch.equal(cache, again)
    mine = R.Cache.zeros(cache.shape[0], H, D, page)  # all ones where a written token lies
    tb = tab.cpu().numpy()
    for s, (n, a) in enumerate(zip(lens, start)):
        for pos in range(a, a + n):
            at = (tb[s, pos // page], slice(None), pos % page // 16, pos % 16)
            for w in range(2):
                mine.codes[w][at] = 15
                mine.d[w].view(np.uint16)[at] = 0xffff
                mine.m[w].view(np.uint16)[at] = 0xffff
    mine.pack()
    assert np.isin(mine.bytes, (0, 255)).all()
    keep = torch.tensor(mine.bytes == 0).cuda()
    assert torch.equal(cache[keep], before[keep])
    assert int(status) == 0


@gpu
def test_append_non_finite_groups_read_back_as_nan(P):
    k = torch.zeros(3, 1, 128, device="cuda")
    k[0, 0, 5], k[1, 0, 40], k[2, 0, 127] = float("nan"), float("inf"), float("-inf")
    v = torch.ones_like(k)
    cache = torch.zeros(1, 1, 1, 2560, dtype=torch.uint8, device="cuda")
    tab = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert P.redlite_kv4_append(k, v, R.cu([3]), z, tab, cache, 16) == P.REDLITE_OK
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    assert P.redlite_kv4_load(cache, 16, tab, R.cu([3]), z, ko, vo) == P.REDLITE_OK
    bad = torch.isnan(ko).view(3, 4, 32).all(-1).cpu()
    assert bad.tolist() == [[True, False, False, False], [False, True, False, False], [False, False, False, True]]
    assert bool((vo == 1).all()) and int(torch.isnan(ko).sum()) == 96


@gpu
def test_bad_pages_and_starts_are_reported_and_skipped(P):
    rng = np.random.default_rng(3)
    lens, start, page = [20, 20, 20], [0, 0, 10], 16
    k, v, tab, cache = _fill(P, rng, torch.float32, 128, 2, page, lens, start)
    tab[0, 1] = cache.shape[0]   # one past the last page
    tab[1, 0] = -5
    before = cache.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    assert P.redlite_kv4_append(k, v, R.cu(lens), st, tab, cache, page, status) == P.REDLITE_OK
    assert int(status) == P.REDLITE_STATUS_BAD_PAGE
    ko, vo = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    assert P.redlite_kv4_load(cache, page, tab, R.cu(lens), st, ko, vo, status) == P.REDLITE_OK
    assert bool((ko[16:36] == 0).all()) and bool((vo[16:36] == 0).all())
    ref = R.dequantise(*R.quantise(k.double().cpu().numpy())).astype(np.float32)
    good = list(range(16)) + list(range(36, 60))
    assert np.array_equal(ko.cpu().numpy()[good], ref[good])
    # positions in front of the sequence or behind its table
    status.zero_()
    cache.copy_(before)
    st = torch.tensor([-30, 40, 0], dtype=torch.int32, device="cuda")
    tab.clamp_(0, cache.shape[0] - 1)
    assert P.redlite_kv4_append(k[:40], v[:40], R.cu([20, 20, 0]), st, tab, cache, page, status) == P.REDLITE_OK
    assert int(status) == P.REDLITE_STATUS_BAD_LENGTH
    assert torch.equal(cache, before)


# --------------------------------------------------------------------- decode


def _decode_case(P, rng, t, D, Hq, Hk, page, lens, mag=1.0, qmag=1.0, spare=3):
    n, tab = R.table(rng, lens, page, spare)
    C = R.Cache(rng, n, Hk, D, page, mag)
    q = torch.tensor(qmag * rng.standard_normal((len(lens), Hq, D))).to(t).cuda()
    return C, tab, q


def _reference(C, tab, q, lens, scale):
    """(out, bound on the error before the last rounding) in 64 bits.
    Bound, per sequence and head.  Scores: a handful of fp32 roundings of sums
    whose terms add up to A_t = scale sum_g sum|q_g| (32 d + |m - 16 d|):
    2^-20 A_t covers 8 of them, and 2^-20 the exponential's own error, its
    argument's rounding to within 2^-24 of |log2 e s_t| included in A_t.  A
    relative change e of the probabilities moves the output by at most
    2 e max|v|.  Values: the split of 16 d p and p leaves out 2^-17 of each
    term, |term| <= 8 d and |m + 8 d|, and the fp32 sums add 2^-20 of them."""
    B, Hq, D = q.shape
    Hk = C.heads
    qn = q.double().cpu().numpy()
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, 1))
    for b, n in enumerate(lens):
        for h in range(Hq if n else 0):
            kh = h // (Hq // Hk)
            pages = tab[b, :-(-n // C.page)]
            k, v = C.values(0, pages, n, kh), C.values(1, pages, n, kh)
            out[b, h] = R.softmax(scale * (k @ qn[b, h]))[None] @ v
            qa = np.abs(qn[b, h]).reshape(-1, 32).sum(-1)
            d, m = C.steps(0, pages, n, kh)
            A = scale * (qa * (32 * d + np.abs(m - 16 * d))).sum(-1).max()
            d, m = C.steps(1, pages, n, kh)
            big = (8 * d + np.abs(m + 8 * d)).max()
            tol[b, h] = 2 * np.abs(v).max() * 2.0 ** -20 * (A + 1) + big * (2.0 ** -17 + 2.0 ** -20)
    return out, tol


def _call(P, C, tab, q, lens, scale, status=None, stream=None, out=None, ws=None):
    B, Hq, D = q.shape
    cache, tb = torch.tensor(C.bytes).cuda(), torch.tensor(tab).cuda()
    out = torch.full_like(q, 9.0) if out is None else out
    if ws is None:
        # whatever a workspace holds has no effect
        ws = torch.full((P.redlite_kv4_decode_workspace_bytes(B, Hq, C.heads, D),), 255, dtype=torch.uint8, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert P.redlite_kv4_decode(q, cache, C.page, tb, ln, out, ws, scale, status, stream) == P.REDLITE_OK
    return out


def _compare(out, ref, tol):
    got = out.double().cpu().numpy()
    lim = tol + np.abs(ref) * R.HALF_ULP[out.dtype] * 1.001
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= lim).all(), float((np.abs(got - ref) / lim).max())


@gpu
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("D,Hq,Hk,page,lens", [
    (256, 16, 2, 64, [1]),
    (256, 16, 2, 64, [700]),
    (256, 2, 2, 16, [17, 0, 15, 16, 129]),
    (128, 32, 8, 32, [5, 1, 333]),
    (128, 5, 1, 128, [127, 128, 129, 2000]),
    (128, 24, 2, 16, [1, 31, 257]),       # 12 query heads per key/value head: two blocks of them
    (256, 16, 1, 48, [1000, 3]),          # 16 of them; a page of three tiles
    (128, 6, 3, 64, [0, 0, 900, 0]),
])
def test_decode_matches_reference(P, t, D, Hq, Hk, page, lens):
    rng = np.random.default_rng(D + Hq + sum(lens))
    C, tab, q = _decode_case(P, rng, t, D, Hq, Hk, page, lens, qmag=2.0)
    scale = D ** -0.5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _call(P, C, tab, q, lens, scale, status)
    _compare(out, *_reference(C, tab, q, lens, scale))
    assert int(status) == 0
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all())


@gpu
def test_decode_long_sequence_over_all_blocks(P):
    rng = np.random.default_rng(11)
    lens = [20000, 3]
    C, tab, q = _decode_case(P, rng, torch.float32, 128, 8, 1, 128, lens)
    _compare(_call(P, C, tab, q, lens, 0.3), *_reference(C, tab, q, lens, 0.3))


@gpu
@pytest.mark.parametrize("mag,qmag,scale", [(1e-3, 1.0, 1.0), (50.0, 1e-3, 1.0), (1.0, 30.0, 0.2), (1.0, 1e-20, 1e3)])
def test_decode_magnitudes(P, mag, qmag, scale):
    rng = np.random.default_rng(5)
    lens = [300, 64]
    C, tab, q = _decode_case(P, rng, torch.float32, 256, 4, 2, 32, lens, mag=mag, qmag=qmag)
    _compare(_call(P, C, tab, q, lens, scale), *_reference(C, tab, q, lens, scale))


@gpu
def test_decode_ignores_what_lies_behind_a_sequence(P):
    """NaN and infinite steps on tokens past the length, in the same tile and on other pages."""
    rng = np.random.default_rng(6)
    lens = [21, 40, 16]
    C, tab, q = _decode_case(P, rng, torch.bfloat16, 128, 8, 2, 32, lens)
    ref = _reference(C, tab, q, lens, 0.1)
    used = np.zeros((C.n_pages, C.page), bool)
    for b, n in enumerate(lens):
        for i in range(n):
            used[tab[b, i // C.page], i % C.page] = True
    bad = ~used.reshape(C.n_pages, 1, -1, 16, 1) & np.ones(C.d[0].shape, bool)
    for w in range(2):
        C.d[w][bad] = np.nan
        C.m[w][bad] = np.inf
    C.pack()
    _compare(_call(P, C, tab, q, lens, 0.1), *ref)


@gpu
def test_decode_bad_lengths_and_pages(P):
    rng = np.random.default_rng(7)
    lens = [40, 40, 40]
    C, tab, q = _decode_case(P, rng, torch.float32, 128, 4, 2, 16, lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref, tol = _reference(C, tab, q, lens, 0.1)
    out = _call(P, C, tab, q, [40, -1, 16 * tab.shape[1] + 1], 0.1, status)
    assert int(status) == P.REDLITE_STATUS_BAD_LENGTH
    _compare(out[:1], ref[:1], tol[:1])
    assert bool((out[1:] == 0).all())
    # a page that is not there: its tokens are left out
    status.zero_()
    tab[1, 2] = C.n_pages
    tab[2, 0] = -1
    out = _call(P, C, tab, q, lens, 0.1, status)
    assert int(status) == P.REDLITE_STATUS_BAD_PAGE
    ref2, tol2 = _reference(C, tab, q, [40, 32, 0], 0.1)
    keep = tab.copy()
    keep[2, :2] = tab[2, 1:3]
    ref3, tol3 = _reference(C, keep, q, [0, 0, 24], 0.1)
    _compare(out, np.stack([ref[0], ref2[1], ref3[2]]), np.stack([tol[0], tol2[1], tol3[2]]))


@gpu
def test_decode_streams_graphs_strides(P):
    """A replayed graph, another stream, rows of a joint tensor, repeated calls: the same bits."""
    rng = np.random.default_rng(8)
    lens = [500, 77, 0, 1300]
    C, tab, q = _decode_case(P, rng, torch.bfloat16, 256, 8, 2, 64, lens)
    base = _call(P, C, tab, q, lens, 0.07)
    joint = torch.zeros(4, 12, 256, dtype=q.dtype, device="cuda")
    joint[:, 2:10] = q
    wide = torch.full((4, 20, 256), 4.0, dtype=q.dtype, device="cuda")
    got = _call(P, C, tab, joint[:, 2:10], lens, 0.07, out=wide[:, 5:13])
    assert torch.equal(got, base) and bool((wide[:, :5] == 4).all()) and bool((wide[:, 13:] == 4).all())
    cache, tb = torch.tensor(C.bytes).cuda(), torch.tensor(tab).cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(P.redlite_kv4_decode_workspace_bytes(4, 8, 2, 256), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert P.redlite_kv4_decode(q, cache, 64, tb, ln, out, ws, 0.07, None, side) == P.REDLITE_OK
    side.synchronize()
    assert torch.equal(out, base)
    # two graphs that share a workspace, replayed in turn with new lengths
    other = torch.zeros_like(q)
    graphs = []
    for dst in (out, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            assert P.redlite_kv4_decode(q, cache, 64, tb, ln, dst, ws, 0.07) == P.REDLITE_OK
        graphs.append(g)
    out.zero_()
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(out, base) and torch.equal(other, base)
    ln.copy_(torch.tensor([1, 0, 640, 129], dtype=torch.int32))
    tb[2] = tb[3]  # a shared prefix
    graphs[1].replay()
    torch.cuda.synchronize()
    _compare(other, *_reference(C, tb.cpu().numpy(), q, [1, 0, 640, 129], 0.07))


@gpu
def test_append_then_decode_one_token_at_a_time(P):
    """The serving loop: append a token, attend; the same as one append of all and a decode."""
    rng = np.random.default_rng(9)
    D, Hq, Hk, page, n = 128, 8, 2, 16, 37
    k, v, tab, cache = _fill(P, rng, torch.float32, D, Hk, page, [n], [0])
    q = torch.tensor(rng.standard_normal((n, 1, Hq, D)), dtype=torch.float32).cuda()
    ws = torch.empty(P.redlite_kv4_decode_workspace_bytes(1, Hq, Hk, D), dtype=torch.uint8, device="cuda")
    C = R.Cache.zeros(cache.shape[0], Hk, D, page)
    tb = tab.cpu().numpy()
    for w, x in enumerate((k, v)):
        c, d, m = R.quantise(x.double().cpu().numpy())
        for i in range(n):
            at = (tb[0, i // page], slice(None), i % page // 16, i % 16)
            C.codes[w][at], C.d[w][at], C.m[w][at] = c[i], d[i], m[i]
    out = torch.zeros(1, Hq, D, device="cuda")
    for i in range(n):
        st = torch.tensor([i], dtype=torch.int32, device="cuda")
        assert P.redlite_kv4_append(k[i:i + 1], v[i:i + 1], R.cu([1]), st, tab, cache, page) == P.REDLITE_OK
        assert P.redlite_kv4_decode(q[i], cache, page, tab, st + 1, out, ws, 0.1) == P.REDLITE_OK
        _compare(out, *_reference(C, tb, q[i], [i + 1], 0.1))
