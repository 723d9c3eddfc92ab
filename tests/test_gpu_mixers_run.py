"""The token mixers and the MoE block together, as a two-layer model would call
them: a packed prompt (attention over it and into the 4-bit cache; the chunked
delta rule), then single tokens (append and one-query attention; one delta
step), a block behind each.  Calls follow each other without a wait between
them, also as replayed graphs, and give the bits that they give one at a time;
the mixers' results are held against 64-bit references on the inputs that they
saw."""
import numpy as np
import pytest
import torch

import fixtures
import mixer_refs as R

pytestmark = pytest.mark.gpu

H, E, F, TOPK = 512, 16, 256, 4        # block
HQ, HK, D = 4, 2, 128                  # attention heads
KH, VH, DK = 2, 4, 128                 # delta heads
LENS = [70, 1, 130]
STEPS, PAGE = 6, 32


@pytest.fixture(scope="module")
def P():
    from routed_expert_ffn_iq2_b200 import build

    build.build()
    import routed_expert_ffn_iq2_b200 as P

    return P


class Model:
    def __init__(self, P, seed=5):
        self.P = P
        rng = np.random.default_rng(seed)
        T, B = sum(LENS), len(LENS)

        def w(n_in, n_out):
            return torch.tensor(rng.standard_normal((n_in, n_out)) / np.sqrt(n_in), dtype=torch.float32).cuda()

        self.x0 = torch.tensor(rng.standard_normal((T, H)), dtype=torch.float32).cuda()
        self.tokens = torch.tensor(rng.standard_normal((STEPS, B, H)), dtype=torch.float32).cuda()
        self.w_att, self.w_o = w(H, (HQ + 2 * HK) * D), w(HQ * D, H)
        self.w_del, self.w_do = w(H, (2 * KH + VH) * DK), w(VH * DK, H)
        self.w_gate = w(H, 2 * VH)
        g2, g1 = fixtures.make_grid(seed, 1), fixtures.make_grid(seed, 2)
        self.moe = P.MoeLayer(H, E, F, T, TOPK, g2, g1, pool_bytes=(E + 1) * fixtures.expert_bytes(1, H, F) + 4096)
        assert self.moe.upload(list(range(E)), [fixtures.make_expert(seed, 1 + e % 2, H, F, e) for e in range(E)]) == 0
        self.gamma = torch.ones(H, device="cuda")
        self.router = torch.tensor(0.05 * rng.standard_normal((E, H)), dtype=torch.float32).cuda()
        self.scratch = torch.zeros(P.redlite_moe_block_scratch_bytes(H, E, T, TOPK), dtype=torch.uint8, device="cuda")
        n, tab = R.table(rng, [a + STEPS for a in LENS], PAGE)
        self.table = torch.tensor(tab).cuda()
        self.cache = torch.zeros(n, HK, PAGE // 16, 20 * D, dtype=torch.uint8, device="cuda")
        self.state = torch.zeros(B, VH, DK, DK, device="cuda")
        self.cu = R.cu(LENS)
        self.zero = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ones = R.cu([1] * B)
        self.pos = torch.tensor(LENS, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws_dec = torch.empty(P.redlite_kv4_decode_workspace_bytes(B, HQ, HK, D), dtype=torch.uint8, device="cuda")
        self.ws_del = torch.empty(P.redlite_delta_workspace_bytes(T, B, KH, VH, DK, DK), dtype=torch.uint8, device="cuda")
        self.scale = D ** -0.5
        self.sync = False
        self.log, self.blocks = {}, []

    def did(self, rc):
        assert rc == 0
        if self.sync:
            torch.cuda.synchronize()

    def block(self, x):
        # the layer adds its experts up in any order: its last bits are not
        # the same twice, so what goes on is x and what is compared is rounded
        out = torch.full_like(x, float("nan"))
        self.did(self.P.redlite_moe_block(x, x.shape[0], self.gamma, 1e-6, self.router, TOPK, self.moe.table, None, out,
                                          self.scratch))
        self.blocks.append(out)
        return x + 0.0 * out

    def gates(self, x):
        y = x @ self.w_gate
        return (-torch.nn.functional.softplus(y[:, :VH])).contiguous(), torch.sigmoid(y[:, VH:]).contiguous()

    def prompt(self):
        P, T = self.P, sum(LENS)
        y = (self.x0 @ self.w_att).to(torch.bfloat16).view(T, HQ + 2 * HK, D)
        q, k, v = y[:, :HQ], y[:, HQ:HQ + HK], y[:, HQ + HK:]
        a = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.did(P.redlite_attn_prefill(q, k, v, self.cu, self.cu, a, self.scale, self.status))
        self.did(P.redlite_kv4_append(k, v, self.cu, self.zero, self.table, self.cache, PAGE, self.status))
        x = self.block(self.x0 + a.float().view(T, -1) @ self.w_o)
        y = (x @ self.w_del).view(T, 2 * KH + VH, DK)
        g, beta = self.gates(x)
        o = torch.empty(T, VH, DK, device="cuda")
        self.did(P.redlite_delta_prefill(y[:, :KH], y[:, KH:2 * KH], y[:, 2 * KH:], g, beta, self.cu, None, self.state, None,
                                         o, self.ws_del, self.scale, 1e-6, self.status))
        self.log.update(q=q, k=k, v=v, attn=a, dy=y, g=g, beta=beta, delta=o)
        return self.block(x + o.view(T, -1) @ self.w_do)

    def token(self, x):
        P, B = self.P, len(LENS)
        y = (x @ self.w_att).to(torch.bfloat16).view(B, HQ + 2 * HK, D)
        self.did(P.redlite_kv4_append(y[:, HQ:HQ + HK], y[:, HQ + HK:], self.ones, self.pos, self.table, self.cache, PAGE,
                                      self.status))
        self.pos += 1
        a = torch.empty(B, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.did(P.redlite_kv4_decode(y[:, :HQ], self.cache, PAGE, self.table, self.pos, a, self.ws_dec, self.scale,
                                      self.status))
        x = self.block(x + a.float().view(B, -1) @ self.w_o)
        z = (x @ self.w_del).view(B, 2 * KH + VH, DK)
        g, beta = self.gates(x)
        o = torch.empty(B, VH, DK, device="cuda")
        self.did(P.redlite_delta_step(z[:, :KH], z[:, KH:2 * KH], z[:, 2 * KH:], g, beta, self.state, self.state, None, o,
                                      self.scale, 1e-6, self.status))
        self.log.update(tq=y[:, :HQ], tattn=a, tz=z, tg=g, tbeta=beta, tdelta=o)
        return self.block(x + o.view(B, -1) @ self.w_do)

    def reset(self):
        self.cache.zero_()
        self.state.zero_()
        self.pos.copy_(torch.tensor(LENS, dtype=torch.int32))


def _run(m):
    m.reset()
    m.blocks.clear()
    outs = [m.prompt()]
    for i in range(STEPS):
        outs.append(m.token(m.tokens[i]))
    torch.cuda.synchronize()
    assert int(m.status) == 0 and m.moe.read_status() == 0
    return [o.clone() for o in outs], m.cache.clone(), m.state.clone(), [o.clone() for o in m.blocks]


def _same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    for x, y in zip(a[3], b[3]):
        assert float((x - y).abs().max()) <= 1e-4 * float(y.abs().max())


def test_calls_in_a_row_give_what_single_calls_give(P):
    m = Model(P)
    m.sync = True
    one = _run(m)
    m.sync = False
    for _ in range(5):
        _same(_run(m), one)
    assert all(bool(torch.isfinite(o).all()) for o in one[0])


def test_replayed_token_graph(P):
    m = Model(P, 6)
    want = _run(m)
    m.reset()
    m.prompt()
    x, side = torch.zeros(len(LENS), H, device="cuda"), torch.cuda.Stream()
    keep = (m.cache.clone(), m.state.clone(), m.pos.clone())
    # the layer's table names the stream it runs on: capture there
    m.moe.table.stream = side.cuda_stream
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = m.token(x)
    m.cache.copy_(keep[0]), m.state.copy_(keep[1]), m.pos.copy_(keep[2])
    for i in range(STEPS):
        x.copy_(m.tokens[i])
        graph.replay()
        assert torch.equal(out, want[0][1 + i])
    torch.cuda.synchronize()
    assert torch.equal(m.cache, want[1]) and torch.equal(m.state, want[2]) and int(m.status) == 0


def test_mixers_against_references(P):
    m = Model(P, 7)
    m.reset()
    m.prompt()
    torch.cuda.synchronize()
    h = {k: v.double().cpu().numpy() for k, v in m.log.items()}
    # attention over the prompt: probabilities rounded to bf16 (2^-8 of sum p |v|), scores and sums to 2^-14 of
    # max |v| (fp32, scores up to 2^6), half a step of the output
    t = 0
    for n in LENS:
        for hd in range(HQ):
            kk, vv = h["k"][t:t + n, hd // 2], h["v"][t:t + n, hd // 2]
            for i in range(n):
                p = R.softmax(m.scale * (kk[:i + 1] @ h["q"][t + i, hd]))
                ref = p @ vv[:i + 1]
                lim = 2.0 ** -8 * (p @ np.abs(vv[:i + 1])) + 2.0 ** -14 * np.abs(vv[:i + 1]).max()
                assert (np.abs(h["attn"][t + i, hd] - ref) <= lim + (np.abs(ref) + lim) * 2.0 ** -8).all()
        t += n
    # the delta rule: every product's operands are held to 2^-22; 130 tokens of |k| = 1, beta < 1 contract, so errors
    # add up at most linearly: 130 x 2^-22 x 128 of the largest state entry and value
    y = h["dy"]
    ref, S, big = R.delta(y[:, :KH], y[:, KH:2 * KH], y[:, 2 * KH:], h["g"], h["beta"], LENS,
                          np.zeros((len(LENS), VH, DK, DK)), m.scale, 1e-6)
    e = 130 * 2.0 ** -22 * 128 * max(big.max(), np.abs(y).max())
    assert np.abs(h["delta"] - ref).max() <= e and np.abs(m.state.double().cpu().numpy() - S).max() <= e
    # one token: attention over what the cache holds, then a step on the state as it was
    before = m.state.double().cpu().numpy()
    m.token(m.tokens[0])
    torch.cuda.synchronize()
    n = [a + 1 for a in LENS]
    ko = torch.empty(sum(n), HK, D, device="cuda")
    vo = torch.empty_like(ko)
    assert P.redlite_kv4_load(m.cache, PAGE, m.table, R.cu(n), m.zero, ko, vo, m.status) == 0
    h = {k: v.double().cpu().numpy() for k, v in m.log.items()}
    ko, vo, t = ko.double().cpu().numpy(), vo.double().cpu().numpy(), 0
    for b, c in enumerate(n):
        for hd in range(HQ):
            kk, vv = ko[t:t + c, hd // 2], vo[t:t + c, hd // 2]
            p = R.softmax(m.scale * (kk @ h["tq"][b, hd]))
            ref = p @ vv
            # p d is one fp16 product (two roundings of 2^-11) of up to 8 steps, the steps at most 2 max |v| / 15
            lim = 2.0 ** -10 * 8 * 2 * np.abs(vv).max() / 15 + 2.0 ** -12 * np.abs(vv).max()
            assert (np.abs(h["tattn"][b, hd] - ref) <= lim + (np.abs(ref) + lim) * 2.0 ** -8).all()
        t += c
    z = h["tz"]
    ref, S, big = R.delta(z[:, :KH], z[:, KH:2 * KH], z[:, 2 * KH:], h["tg"], h["tbeta"], [1] * len(LENS), before, m.scale,
                          1e-6)
    e = 2.0 ** -24 * 16 * np.sqrt(DK) * (big.max() + np.abs(z).max())
    assert np.abs(h["tdelta"] - ref).max() <= e and np.abs(m.state.double().cpu().numpy() - S).max() <= e
