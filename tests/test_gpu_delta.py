"""The gated delta rule, chunked and one token at a time, against a token by
token reference in 64 bits."""
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


def test_refusals_before_device_work(P):
    L, p = P.lib(), ctypes.c_void_p(0x10000)
    odd = ctypes.c_void_p(0x10008)

    def prefill(dtype=0, q=p, qs=2048, ks=2048, vs=4096, g=p, cu=p, n=1, T=4, hk=16, hv=32, dk=128, dv=128, scale=1.0,
                si=p, so=p, slots=p, ns=4, out=p, ws=p, wb=1 << 40):
        return L.redlite_delta_prefill(dtype, q, qs, p, ks, p, vs, g, p, cu, n, T, hk, hv, dk, dv, scale, -1.0, si, so,
                                       slots, ns, out, 4096, ws, wb, None, None)

    assert prefill(n=0) == P.REDLITE_OK
    for kw in (dict(dtype=3), dict(n=-1), dict(T=-1), dict(hk=0), dict(hv=33), dict(q=None), dict(g=None), dict(cu=None),
               dict(qs=2047), dict(qs=2050), dict(vs=128), dict(so=None), dict(si=odd), dict(so=odd), dict(ns=0),
               dict(slots=None, ns=0), dict(slots=None, n=5), dict(out=None), dict(ws=None), dict(ws=odd),
               dict(scale=float("nan"))):
        assert prefill(**kw) == P.REDLITE_EINVAL, kw
    for kw in (dict(dk=96), dict(dv=256), dict(dk=32)):
        assert prefill(**kw) == P.REDLITE_EUNSUPPORTED, kw
    assert prefill(wb=1000) == P.REDLITE_ENOMEM
    assert P.redlite_delta_workspace_bytes(100, 1, 3, 4, 128, 128) == 0
    assert P.redlite_delta_workspace_bytes(100, 1, 2, 4, 128, 100) == 0

    def step(dtype=1, q=p, qs=256, n=2, hk=2, hv=4, so=p, slots=None, ns=2):
        return L.redlite_delta_step(dtype, q, qs, p, 256, p, 512, p, p, n, hk, hv, 128, 128, 1.0, -1.0, p, so, slots, ns,
                                    p, 512, None, None)

    assert step(n=0) == P.REDLITE_OK
    for kw in (dict(q=None), dict(qs=252), dict(hv=3), dict(so=None), dict(ns=1), dict(dtype=-1)):
        assert step(**kw) == P.REDLITE_EINVAL, kw


def _inputs(rng, t, T, hk, hv, dk, dv, norm, decay=1.0):
    q, k = rng.standard_normal((T, hk, dk)), rng.standard_normal((T, hk, dk))
    if not norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True)) for x in (q, k))
    v = rng.standard_normal((T, hv, dv))
    g = -decay * rng.exponential(1.0, (T, hv)) * 10 ** rng.uniform(-3, 0.5, (1, hv))
    beta = 1 / (1 + np.exp(-rng.standard_normal((T, hv))))
    dev = [torch.tensor(x).to(t).cuda() for x in (q, k, v)]
    dev += [torch.tensor(x, dtype=torch.float32).cuda() for x in (g, beta)]
    return dev


def _host(x):
    return x.double().cpu().numpy()


def _limits(ref, big, lens, scale, dk, v_max, out_type):
    """Bounds on |out - ref| and |state - ref|.  Per head let M be the largest
    state entry met and V = max|v|.  A chunk of 64 tokens makes its updates
    from products whose fp32 operands are split in two bf16 parts: each product
    of a row of S (norm at most M sqrt(dk)) with a unit key is off by at most
    2^-17 sqrt(dk) M ... in sum, with |k| = 1 and 0 <= beta <= 1 the updates of
    a chunk are off by E = 2^-17 (V + sqrt(dk) M) times the norm growth of T's
    rows; T inverts a unit lower triangle whose rows are contractions of the
    delta rule, and its error and D's splits add as much again: 8 E in all.
    The rule contracts (|I - beta k k^T| <= 1), so the errors of successive
    chunks add up at most linearly while the decay lets them live; they are of
    random sign, so their sum over n chunks is taken as sqrt(n) with a factor
    4 on top.  Output: scale |q| times the state's error per row, sqrt(dk)
    entries of random sign -> times 1 for the unit query, plus its own splits
    of the same size; plus half a step of the output type."""
    n_chunks = max(1, (max(lens) + 63) // 64)
    E = 8 * 2.0 ** -17 * (v_max + np.sqrt(dk) * big.max()) * 4 * np.sqrt(n_chunks)
    return 2 * scale * E + np.abs(ref) * R.HALF_ULP[out_type] * 1.001, E


def _prefill(P, dev, cu, state_in, state_out, slots, scale, eps, status=None, out=None, stream=None):
    q, k, v, g, beta = dev
    out = torch.full_like(v, 5.0) if out is None else out
    n = cu.numel() - 1
    ws = torch.full((P.redlite_delta_workspace_bytes(q.shape[0], n, q.shape[1], v.shape[1], q.shape[2], v.shape[2]),),
                    255, dtype=torch.uint8, device="cuda")
    assert P.redlite_delta_prefill(q, k, v, g, beta, cu, state_in, state_out, slots, out, ws, scale, eps, status,
                                   stream) == P.REDLITE_OK
    return out


@gpu
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hk,hv,dk,dv,norm,lens", [
    (1, 1, 128, 128, True, [1]),
    (2, 4, 128, 128, True, [64, 0, 65, 1, 63]),
    (1, 3, 64, 128, False, [200]),
    (2, 2, 128, 64, True, [130, 7]),
    (4, 16, 64, 64, False, [33, 128, 0, 129, 5]),
    (1, 2, 128, 128, False, [1000]),
])
def test_prefill_matches_reference(P, t, hk, hv, dk, dv, norm, lens):
    rng = np.random.default_rng(dk + hv + sum(lens))
    T, n = sum(lens), len(lens)
    dev = _inputs(rng, t, T + 3, hk, hv, dk, dv, norm)
    scale, eps = dk ** -0.5, (1e-6 if norm else -1.0)
    pool = torch.tensor(rng.standard_normal((n + 2, hv, dk, dv)), dtype=torch.float32).cuda()
    slots = torch.tensor(rng.permutation(n + 2)[:n].astype(np.int32)).cuda()
    state_out = torch.full_like(pool, 11.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _prefill(P, dev, R.cu(lens), pool, state_out, slots, scale, eps, status)
    assert int(status) == 0
    ref, S, big = R.delta(*[_host(x)[:T] for x in dev], lens, _host(pool[slots.long()]), scale, eps)
    lim, slim = _limits(ref, big, lens, scale, dk, np.abs(_host(dev[2])).max(), t)
    err = np.abs(_host(out)[:T] - ref)
    assert (err <= lim).all(), float((err / lim).max())
    serr = np.abs(_host(state_out[slots.long()]) - S)
    assert (serr <= slim).all(), float((serr / slim).max())
    assert bool((out[T:] == 5.0).all())  # rows behind the last sequence
    rest = torch.ones(n + 2, dtype=torch.bool)
    rest[slots.cpu().long()] = False
    assert bool((state_out[rest.cuda()] == 11.0).all())
    # in place, default slots, no state in front
    if n > 1:
        again = pool.clone()
        out2 = _prefill(P, dev, R.cu(lens), again, again, slots, scale, eps)
        assert torch.equal(out2, out) and torch.equal(again[slots.long()], state_out[slots.long()])
        zero = torch.zeros(n, hv, dk, dv, device="cuda")
        a, b = torch.full_like(zero, 3.0), torch.full_like(zero, 4.0)
        assert torch.equal(_prefill(P, dev, R.cu(lens), zero, a, None, scale, eps),
                           _prefill(P, dev, R.cu(lens), None, b, None, scale, eps))
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("hk,hv,dk,dv,norm,n", [(16, 32, 128, 128, True, 1), (2, 2, 64, 128, False, 3),
                                                (1, 4, 128, 64, True, 130)])
def test_step_matches_reference(P, t, hk, hv, dk, dv, norm, n):
    rng = np.random.default_rng(n)
    dev = _inputs(rng, t, n, hk, hv, dk, dv, norm)
    scale, eps = 0.7, (1e-6 if norm else -1.0)
    pool = torch.tensor(rng.standard_normal((n + 1, hv, dk, dv)), dtype=torch.float32).cuda()
    slots = torch.tensor(rng.permutation(n + 1)[:n].astype(np.int32)).cuda()
    state, out = pool.clone(), torch.zeros_like(dev[2])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert P.redlite_delta_step(*dev, state, state, slots, out, scale, eps, status) == P.REDLITE_OK
    ref, S, big = R.delta(*[_host(x) for x in dev], [1] * n, _host(pool[slots.long()]), scale, eps)
    # fp32 throughout: sums of dk products, each at most M and V in size; 2^-24 sqrt(dk) of it times a few
    e = 2.0 ** -24 * 16 * np.sqrt(dk) * (big.max() + np.abs(_host(dev[2])).max())
    err = np.abs(_host(out) - ref) - np.abs(ref) * R.HALF_ULP[t] * 1.001
    assert err.max() <= 2 * scale * e and np.abs(_host(state[slots.long()]) - S).max() <= e
    keep = torch.ones(n + 1, dtype=torch.bool)
    keep[slots.cpu().long()] = False
    assert torch.equal(state[keep.cuda()], pool[keep.cuda()]) and int(status) == 0


@gpu
def test_prefill_then_steps_continue_one_sequence(P):
    """130 tokens at once, or 100 of them and then 30 single steps on the state left behind."""
    rng = np.random.default_rng(2)
    dev = _inputs(rng, torch.float32, 130, 2, 4, 128, 128, True)
    full = torch.zeros(1, 4, 128, 128, device="cuda")
    out = _prefill(P, dev, R.cu([130]), None, full, None, 0.1, 1e-6)
    part = torch.zeros_like(full)
    head = [x[:100].contiguous() for x in dev]
    got = [_prefill(P, head, R.cu([100]), None, part, None, 0.1, 1e-6)]
    for i in range(100, 130):
        o = torch.zeros(1, 4, 128, device="cuda")
        assert P.redlite_delta_step(*[x[i:i + 1].contiguous() for x in dev], part, part, None, o, 0.1,
                                    1e-6) == P.REDLITE_OK
        got.append(o)
    ref, S, big = R.delta(*[_host(x) for x in dev], [130], np.zeros((1, 4, 128, 128)), 0.1, 1e-6)
    lim, slim = _limits(ref, big, [130], 0.1, 128, np.abs(_host(dev[2])).max(), torch.float32)
    for o, s in ((out, full), (torch.cat(got), part)):
        assert (np.abs(_host(o) - ref) <= lim).all() and (np.abs(_host(s) - S) <= slim).all()


@gpu
def test_strong_and_full_decay(P):
    """Log decays of -50 and -infinity clear the state; the tokens behind them are as after a fresh start."""
    rng = np.random.default_rng(3)
    for t in (torch.float32, torch.bfloat16):
        dev = _inputs(rng, t, 200, 1, 2, 128, 128, True, decay=0.01)
        dev[3][40:100:7, 0] = -50.0
        dev[3][90, 1] = float("-inf")
        dev[3][91, 1] = float("-inf")
        dev[3][130, :] = -3e8
        st = torch.tensor(rng.standard_normal((1, 2, 128, 128)), dtype=torch.float32).cuda()
        s = torch.zeros_like(st)
        out = _prefill(P, dev, R.cu([200]), st, s, None, 0.1, 1e-6)
        ref, S, big = R.delta(*[_host(x) for x in dev], [200], _host(st), 0.1, 1e-6)
        lim, slim = _limits(ref, big, [200], 0.1, 128, np.abs(_host(dev[2])).max(), t)
        assert (np.abs(_host(out) - ref) <= lim).all() and (np.abs(_host(s) - S) <= slim).all()


@gpu
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "beta"])
def test_non_finite_tokens_do_not_reach_back(P, t, what):
    """A NaN at one token leaves the outputs in front of it, other heads and other sequences as they were."""
    rng = np.random.default_rng(4)
    lens, bad = [150, 90], 100  # in the second chunk of the first sequence
    dev = _inputs(rng, t, 240, 2, 2, 128, 128, True)
    s0, s1 = (torch.zeros(2, 2, 128, 128, device="cuda") for _ in range(2))
    base = _prefill(P, dev, R.cu(lens), None, s0, None, 0.1, 1e-6)
    x = dev["qkv".index(what) if what in "qkv" else (3 if what == "g" else 4)]
    x[bad, 0] = float("nan")
    out = _prefill(P, dev, R.cu(lens), None, s1, None, 0.1, 1e-6)
    ref, S, big = R.delta(*[_host(y) for y in dev], lens, np.zeros((2, 2, 128, 128)), 0.1, 1e-6)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isfinite(_host(out)), fine)
    assert fine[:bad].all() and not fine[bad, 0].any()
    lim, _ = _limits(np.where(fine, ref, 0), big[np.isfinite(big)], lens, 0.1, 128, 6.0, t)
    assert (np.abs(_host(out) - ref)[fine] <= lim[fine]).all()
    assert torch.equal(out[:, 1], base[:, 1]) and torch.equal(out[150:], base[150:])
    assert torch.equal(s1[1], s0[1]) and torch.equal(s1[0, 1], s0[0, 1])
    assert np.array_equal(np.isfinite(_host(s1)), np.isfinite(S))


@gpu
def test_bad_slots_and_offsets(P):
    rng = np.random.default_rng(5)
    lens = [70, 10, 20, 5]
    dev = _inputs(rng, torch.float32, 105, 1, 2, 128, 128, True)
    good = torch.zeros(4, 2, 128, 128, device="cuda")
    base = _prefill(P, dev, R.cu(lens), None, good, None, 0.1, 1e-6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = torch.full_like(good, 2.0)
    slots = torch.tensor([2, -1, 2, 4], dtype=torch.int32, device="cuda")  # twice, and out of range on both sides
    out = _prefill(P, dev, R.cu(lens), None, state, slots, 0.1, 1e-6, status)
    assert int(status) == P.REDLITE_STATUS_BAD_SLOT
    assert torch.equal(out[:70], base[:70]) and bool((out[70:] == 0).all())
    assert torch.equal(state[2], good[0]) and bool((state[[0, 1, 3]] == 2.0).all())
    status.zero_()
    state.fill_(2.0)
    one = [x[:4].contiguous() for x in dev]
    o = torch.full((4, 2, 128), 9.0, device="cuda")
    assert P.redlite_delta_step(*one, None, state, slots, o, 0.1, 1e-6, status) == P.REDLITE_OK
    assert int(status) == P.REDLITE_STATUS_BAD_SLOT
    assert bool((o[1:] == 0).all()) and bool((o[0] != 9).any()) and bool((state[[0, 1, 3]] == 2.0).all())
    # offsets that do not ascend, or leave the rows
    for cu in ([0, 70, 60, 100, 105], [0, 70, 80, 100, 106], [-1, 70, 80, 100, 105]):
        status.zero_()
        state.fill_(2.0)
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        _prefill(P, dev, c, None, state, None, 0.1, 1e-6, status)
        assert int(status) == P.REDLITE_STATUS_BAD_LENGTH
        broken = [s for s in range(4) if not 0 <= cu[s] <= cu[s + 1] <= 105]
        assert bool((state[broken] == 2.0).all())


@gpu
def test_graphs_streams_strides_and_empty_calls(P):
    rng = np.random.default_rng(6)
    lens = [100, 0, 37]
    T, hk, hv = 137, 2, 4
    dev = _inputs(rng, torch.bfloat16, T, hk, hv, 128, 128, True)
    st = torch.tensor(rng.standard_normal((3, hv, 128, 128)), dtype=torch.float32).cuda()
    s0 = torch.zeros_like(st)
    base = _prefill(P, dev, R.cu(lens), st, s0, None, 0.1, 1e-6)
    assert torch.equal(s0[1], st[1])  # no tokens: the state is copied
    # q, k, v as slices of one projection; out as a slice
    joint = torch.cat([dev[0].reshape(T, -1), dev[1].reshape(T, -1), dev[2].reshape(T, -1)], 1)
    q, k, v = (x.view(T, -1, 128) for x in joint.split([hk * 128, hk * 128, hv * 128], 1))
    wide = torch.full((T, hv + 2, 128), 4.0, dtype=torch.bfloat16, device="cuda")
    s1 = torch.zeros_like(st)
    got = _prefill(P, [q, k, v, dev[3], dev[4]], R.cu(lens), st, s1, None, 0.1, 1e-6, out=wide[:, 1:hv + 1])
    assert torch.equal(got, base) and torch.equal(s1, s0)
    assert bool((wide[:, 0] == 4).all()) and bool((wide[:, -1] == 4).all())
    # captured, replayed with other lengths on another stream
    cu = R.cu(lens)
    ws = torch.empty(P.redlite_delta_workspace_bytes(T, 3, hk, hv, 128, 128), dtype=torch.uint8, device="cuda")
    out, s2 = torch.zeros_like(base), torch.zeros_like(st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        assert P.redlite_delta_prefill(*dev, cu, st, s2, None, out, ws, 0.1, 1e-6) == P.REDLITE_OK
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    assert torch.equal(out, base) and torch.equal(s2, s0)
    cu.copy_(torch.tensor([0, 1, 66, 130], dtype=torch.int32))
    out.fill_(7.0)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    n = [1, 65, 64]
    ref, S, big = R.delta(*[_host(x)[:130] for x in dev], n, _host(st), 0.1, 1e-6)
    lim, slim = _limits(ref, big, n, 0.1, 128, np.abs(_host(dev[2])).max(), torch.bfloat16)
    assert (np.abs(_host(out)[:130] - ref) <= lim).all() and (np.abs(_host(s2) - S) <= slim).all()
    assert bool((out[130:] == 7.0).all())
    # no rows at all: states are copied
    none = [x[:0] for x in dev]
    s3 = torch.zeros_like(st)
    _prefill(P, none, R.cu([0, 0, 0]), st, s3, None, 0.1, 1e-6)
    assert torch.equal(s3, st)
