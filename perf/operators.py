"""Cases and plain forms of the token mixers around the routed layer.

Six operators, reached through the package's same-named calls:

  prompt   redlite_attn_prefill   causal attention over packed prompts, grouped heads
  append   redlite_kv4_append     new keys and values into a paged 4-bit cache
           redlite_kv4_load       (and back out as the values the cache stands for)
  decode   redlite_kv4_decode     one query token per sequence over the 4-bit cache
  delta    redlite_delta_prefill  the gated delta rule over packed prompts (chunked)
  step     redlite_delta_step     the gated delta rule, one token per sequence

Head shapes are those of the model whose layers this package serves (16
query heads on 2 key/value heads of 256; 16 key heads and 32 value heads of
128 for the delta rule) and generic ones.  `own` selects the package's calls;
otherwise `run` computes the same results from elementary torch operations in
32 bits.
"""

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # a few short prompts that arrive together: launch and latency count
        dict(name="prompt_short", op="prompt", type="bf16", dim=256, q_heads=16, kv_heads=2, lens="37,5,1", extra="0,0,0",
             joint=True),
        # ragged batch in fp16 on the generic head shape, two of them with keys from an earlier part
        dict(name="prompt_packed", op="prompt", type="f16", dim=128, q_heads=32, kv_heads=8,
             lens="1000,513,0,2047,64,333", extra="0,129,0,0,1000,0", joint=False),
        # one long document
        dict(name="prompt_long", op="prompt", type="bf16", dim=256, q_heads=16, kv_heads=2, lens="16384", extra="0",
             joint=True),
        # every step of serving 16 streams: one token each, fp32 activations
        dict(name="append_step", op="append", type="f32", dim=256, kv_heads=2, page=64,
             lens=",".join(["1"] * 16), start=",".join(str(97 * i + 13) for i in range(16))),
        # prompts written into the cache
        dict(name="append_prompt", op="append", type="bf16", dim=256, kv_heads=2, page=64, lens="4096,1037,2,2961",
             start="0,0,77,1"),
        # one stream, a short context, fp32 activations: latency
        dict(name="decode_one", op="decode", type="f32", dim=256, q_heads=16, kv_heads=2, page=64, lens="700"),
        # a serving batch of ragged contexts
        dict(name="decode_batch", op="decode", type="bf16", dim=256, q_heads=16, kv_heads=2, page=64,
             lens=",".join(str(1 + (i * i * 37) % 8191) for i in range(64))),
        # long contexts on the generic head shape
        dict(name="decode_long", op="decode", type="f16", dim=128, q_heads=32, kv_heads=8, page=32,
             lens=",".join(str(65536 - 1111 * i) for i in range(16))),
        # packed prompts, fp32 activations, raw queries and keys normalised inside
        dict(name="delta_packed", op="delta", type="f32", k_heads=16, v_heads=32, dk=128, dv=128, norm=True,
             lens="1000,63,0,1,300,64,129,2048"),
        # one long document
        dict(name="delta_long", op="delta", type="bf16", k_heads=16, v_heads=32, dk=128, dv=128, norm=True,
             lens="16384"),
        # one stream, one token: latency
        dict(name="step_one", op="step", type="f32", k_heads=16, v_heads=32, dk=128, dv=128, norm=True, seqs=1),
        # one token for every stream of a large batch
        dict(name="step_batch", op="step", type="bf16", k_heads=16, v_heads=32, dk=128, dv=128, norm=True, seqs=200),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _lens(rng, n, hi, total, zero=0.0):
    """n lengths spread over 1..hi (logarithmically), at most `total` together, some of them 0."""
    out = []
    left = total
    for _ in range(n):
        v = 0 if rng.random() < zero else min(_log(rng, 1, hi), left)
        out.append(v)
        left -= v
    if not any(out):
        out[0] = 1
    return out


def _text(v):
    return ",".join(str(x) for x in v)


def _nums(s):
    return [int(x) for x in s.split(",")]


def draw(rng):
    op = rng.choice(["prompt", "append", "decode", "delta", "step"])
    if op == "prompt":
        kv = rng.choice([1, 2, 3, 4, 8])
        ratio = rng.choice([r for r in (1, 2, 3, 4, 6, 8, 16) if r * kv <= 32])
        n = _log(rng, 1, 24)
        lens = _lens(rng, n, 6000, 12000, 0.1)
        joint = rng.random() < 0.4
        # keys from an earlier part of the sequence, or (rarely) fewer keys than queries
        extra = [0 if joint or rng.random() < 0.6 else _log(rng, 1, 1500) for _ in lens]
        extra = [-rng.randint(1, v) if not joint and v > 0 and rng.random() < 0.05 else e for v, e in zip(lens, extra)]
        return dict(op=op, type=rng.choice(["bf16", "f16"]), dim=rng.choice([128, 256]), q_heads=kv * ratio,
                    kv_heads=kv, lens=_text(lens), extra=_text(extra), joint=joint)
    if op == "append":
        n = _log(rng, 1, 64)
        lens = [1] * n if rng.random() < 0.4 else _lens(rng, n, 4096, 8192, 0.1)
        return dict(op=op, type=rng.choice(["f32", "bf16", "f16"]), dim=rng.choice([128, 256]),
                    kv_heads=rng.choice([1, 2, 3, 4, 8]), page=rng.choice([16, 32, 64, 128]), lens=_text(lens),
                    start=_text([rng.randint(0, 900) for _ in lens]))
    if op == "decode":
        kv = rng.choice([1, 2, 3, 4, 8])
        ratio = rng.choice([r for r in (1, 2, 3, 4, 5, 8, 12, 16) if r * kv <= 48])
        n = _log(rng, 1, 150)
        lens = _lens(rng, n, 50000, 700000 // kv, 0.05)
        return dict(op=op, type=rng.choice(["f32", "bf16", "f16"]), dim=rng.choice([128, 256]), q_heads=kv * ratio,
                    kv_heads=kv, page=rng.choice([16, 32, 64, 128]), lens=_text(lens))
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 2, 4] if hk < 16 else [1, 2])
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
    norm = rng.random() < 0.7
    if op == "delta":
        lens = _lens(rng, _log(rng, 1, 24), 8000, 12000, 0.1)
        return dict(op=op, type=rng.choice(["f32", "bf16", "f16"]), k_heads=hk, v_heads=hv, dk=dk, dv=dv, norm=norm,
                    lens=_text(lens))
    return dict(op=op, type=rng.choice(["f32", "bf16", "f16"]), k_heads=hk, v_heads=hv, dk=dk, dv=dv, norm=norm,
                seqs=_log(rng, 1, 200))


# ----------------------------------------------------------------- inputs


def _cu(lens):
    c = [0]
    for v in lens:
        c.append(c[-1] + v)
    return c


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(lens, page, gen):
    """A block table of randomly placed pages for sequences of these lengths (-1 beyond a sequence's last page)."""
    need = [-(-v // page) for v in lens]
    n = max(1, sum(need))
    order = torch.randperm(n, generator=gen, device="cuda").to(torch.int32).cpu().tolist()
    width = max(1, max(need))
    table, at = [], 0
    for c in need:
        table.append(order[at:at + c] + [-1] * (width - c))
        at += c
    return n, _i32(table)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    t = _TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    op = case["op"]
    s = dict(case=case, type=t)
    if op == "prompt":
        D, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
        ql = _nums(case["lens"])
        kl = [max(0, a + b) for a, b in zip(ql, _nums(case["extra"]))]
        T, K = sum(ql), sum(kl)
        if case["joint"]:  # q, k, v as they leave one joint projection
            x = normal(T, (hq + 2 * hk) * D).to(t)
            q = x[:, :hq * D].view(T, hq, D)
            k = x[:, hq * D:(hq + hk) * D].view(T, hk, D)
            v = x[:, (hq + hk) * D:].view(T, hk, D)
        else:
            q, k, v = normal(T, hq, D).to(t), normal(K, hk, D).to(t), normal(K, hk, D).to(t)
        s.update(q=q, k=k, v=v, ql=ql, kl=kl, cu_q=_i32(_cu(ql)), cu_k=_i32(_cu(kl)), scale=2.0 * D ** -0.5,
                 out=torch.empty(T, hq, D, dtype=t, device="cuda"))
    elif op == "append":
        D, hk, page = case["dim"], case["kv_heads"], case["page"]
        lens, start = _nums(case["lens"]), _nums(case["start"])
        T = sum(lens)
        # keys have channels that are far larger than the rest, and offsets
        k = normal(T, hk, D) * torch.exp(0.7 * normal(1, hk, D)) + 0.5 * normal(1, hk, D)
        n, table = _pages([a + b for a, b in zip(start, lens)], page, gen)
        s.update(k=k.to(t), v=normal(T, hk, D).to(t), cu=_i32(_cu(lens)), start=_i32(start), table=table, page=page,
                 cache=torch.zeros(n, hk, page // 16, 20 * D, dtype=torch.uint8, device="cuda"),
                 k_out=torch.empty(T, hk, D, device="cuda"), v_out=torch.empty(T, hk, D, device="cuda"))
    elif op == "decode":
        D, hq, hk, page = case["dim"], case["q_heads"], case["kv_heads"], case["page"]
        lens = _nums(case["lens"])
        n, table = _pages(lens, page, gen)
        # any bytes are codes; steps and minima as activations of unit variance give
        cache = torch.randint(0, 256, (n, hk, page // 16, 20 * D), generator=gen, device="cuda", dtype=torch.uint8)
        ng = D // 32

        def steps():
            d = 0.2 + 0.25 * torch.rand(n, hk, page // 16, 16 * ng, generator=gen, device="cuda")
            return d.half(), (-7.5 * d + 0.3 * normal(n, hk, page // 16, 16 * ng)).half()

        d, m = steps()
        cache[..., 8 * D:10 * D] = torch.stack([d, m], -1).flatten(-2).view(torch.uint8)
        d, m = steps()
        cache[..., 18 * D:19 * D] = d.view(torch.uint8)
        cache[..., 19 * D:] = m.view(torch.uint8)
        q = normal(len(lens), hq, D).to(t)
        s.update(q=q, cache=cache, table=table, lens=_i32(lens), ll=lens, page=page, scale=1.5 * D ** -0.5,
                 out=torch.empty_like(q))
        if own:
            import routed_expert_ffn_iq2_b200 as P

            ws = P.redlite_kv4_decode_workspace_bytes(len(lens), hq, hk, D)
            s["workspace"] = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
    else:
        hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["dk"], case["dv"]
        lens = _nums(case["lens"]) if op == "delta" else [1] * case["seqs"]
        T, B = sum(lens), len(lens)
        q, k = normal(T, hk, dk), normal(T, hk, dk)
        if not case["norm"]:
            q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
        # per-head decay rates from almost none to a few tokens' memory
        rate = torch.exp(-4.6 + 6.0 * torch.rand(hv, generator=gen, device="cuda"))
        s.update(q=q.to(t), k=k.to(t), v=normal(T, hv, dv).to(t),
                 g=-rate * torch.nn.functional.softplus(normal(T, hv) - 1.0), beta=torch.sigmoid(normal(T, hv)),
                 lens=lens, cu=_i32(_cu(lens)), state_in=0.3 * normal(B, hv, dk, dv),
                 state_out=torch.zeros(B, hv, dk, dv, device="cuda"),
                 slots=torch.randperm(B, generator=gen, device="cuda").to(torch.int32),
                 scale=dk ** -0.5, eps=1e-6 if case["norm"] else -1.0,
                 out=torch.empty(T, hv, dv, dtype=t, device="cuda"))
        s["slot_list"] = s["slots"].cpu().tolist()
        if own and op == "delta":
            import routed_expert_ffn_iq2_b200 as P

            ws = P.redlite_delta_workspace_bytes(T, B, hk, hv, dk, dv)
            s["workspace"] = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------- the package's calls


def _run_own(s):
    import routed_expert_ffn_iq2_b200 as P

    op = s["case"]["op"]
    if op == "prompt":
        rc = P.redlite_attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["scale"])
        res = s["out"]
    elif op == "append":
        rc = P.redlite_kv4_append(s["k"], s["v"], s["cu"], s["start"], s["table"], s["cache"], s["page"])
        rc = rc or P.redlite_kv4_load(s["cache"], s["page"], s["table"], s["cu"], s["start"], s["k_out"], s["v_out"])
        res = (s["k_out"], s["v_out"])
    elif op == "decode":
        rc = P.redlite_kv4_decode(s["q"], s["cache"], s["page"], s["table"], s["lens"], s["out"], s["workspace"],
                                  s["scale"])
        res = s["out"]
    elif op == "delta":
        rc = P.redlite_delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], s["state_in"], s["state_out"],
                                     s["slots"], s["out"], s["workspace"], s["scale"], s["eps"])
        res = (s["out"], s["state_out"])
    else:
        rc = P.redlite_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state_in"], s["state_out"], s["slots"],
                                  s["out"], s["scale"], s["eps"])
        res = (s["out"], s["state_out"])
    if rc != 0:
        raise RuntimeError(f"{op}: code {rc}")
    return res


# -------------------------------------------------------------- plain forms


def _plain_prompt(s):
    q, k, v, c = s["q"], s["k"], s["v"], s["case"]
    D, hq, hk = c["dim"], c["q_heads"], c["kv_heads"]
    out = torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    a = b = 0
    for nq, nk in zip(s["ql"], s["kl"]):
        for i in range(0, nq if nk else 0, 1024):
            e = min(nq, i + 1024)
            top = nk - nq + e  # keys the last of these queries sees
            if top <= 0:
                continue
            qq = q[a + i:a + e].float().view(e - i, hk, hq // hk, D).permute(1, 2, 0, 3)
            kk = k[b:b + top].float().permute(1, 2, 0)[:, None]
            vv = v[b:b + top].float().permute(1, 0, 2)[:, None]
            see = (torch.arange(top, device="cuda")[None, :]
                   <= torch.arange(i, e, device="cuda")[:, None] + (nk - nq))
            z = torch.matmul(qq, kk) * s["scale"]
            z = torch.where(see, z, torch.full_like(z, float("-inf")))
            m = z.amax(-1, keepdim=True)
            p = torch.exp(z - torch.where(m > float("-inf"), m, torch.zeros_like(m)))
            n = p.sum(-1, keepdim=True)
            y = torch.matmul(p, vv) / torch.where(n > 0, n, torch.ones_like(n))
            out[a + i:a + e] = y.permute(2, 0, 1, 3).reshape(e - i, hq, D).to(q.dtype)
        a, b = a + nq, b + nk
    return out


def _plain_quantise(x, fifteen):
    """The values the 4-bit cache holds for x [..., D]: groups of 32, m + d code."""
    g = x.float().clamp(-65504.0, 65504.0).unflatten(-1, (-1, 32))
    m = g.amin(-1, keepdim=True).half().float()
    d = ((g.amax(-1, keepdim=True) - m) / fifteen).half().float()
    # in 64 bits: a value next to the border between two codes
    code = torch.round((g.double() - m.double()) / torch.where(d > 0, d, torch.ones_like(d)).double())
    code = torch.where(d > 0, code.clamp(0, 15), torch.zeros_like(code)).float()
    return (m + d * code).flatten(-2)


def _unpack(tiles, D, t):
    """Keys and values [tokens, D] in type t of cache tiles [n, 20 D] (16 tokens each)."""
    n, ng = tiles.shape[0], D // 32

    def nibbles(b):  # [n, 16, D / 2] bytes -> [n * 16, D]
        return torch.stack([b & 15, b >> 4], -1).reshape(n * 16, D).to(t)

    kb = tiles[:, :8 * D].view(n, ng // 2, 8, 4, 4, 4).permute(0, 1, 4, 2, 3, 5).reshape(n, 2, ng, 8, 4, 4)
    k = nibbles(kb.permute(0, 1, 3, 2, 4, 5).reshape(n, 16, D // 2))
    dm = tiles[:, 8 * D:10 * D].contiguous().view(torch.float16).view(n * 16, ng, 2, 1).to(t)
    k = (dm[:, :, 1] + dm[:, :, 0] * k.view(n * 16, ng, 32)).view(n * 16, D)
    vb = tiles[:, 10 * D:18 * D].view(n, ng // 2, 8, 4, 8, 2).permute(0, 1, 4, 2, 3, 5).reshape(n, 2, 2, ng, 8, 4, 2)
    v = nibbles(vb.permute(0, 1, 5, 2, 3, 4, 6).reshape(n, 16, D // 2))
    d = tiles[:, 18 * D:19 * D].contiguous().view(torch.float16).view(n * 16, ng, 1).to(t)
    m = tiles[:, 19 * D:].contiguous().view(torch.float16).view(n * 16, ng, 1).to(t)
    v = (m + d * v.view(n * 16, ng, 32)).view(n * 16, D)
    return k, v


def _plain_decode(s):
    q, c, page = s["q"], s["case"], s["page"]
    D, hq, hk = c["dim"], c["q_heads"], c["kv_heads"]
    out = torch.zeros_like(q)
    for b, n in enumerate(s["ll"]):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        tiles = s["cache"][pages].transpose(0, 1).reshape(-1, 20 * D)
        k, v = _unpack(tiles, D, torch.float32)
        k, v = k.view(hk, -1, D)[:, :n], v.view(hk, -1, D)[:, :n]
        z = torch.matmul(q[b].float().view(hk, hq // hk, D), k.transpose(1, 2)) * s["scale"]
        p = torch.exp(z - z.amax(-1, keepdim=True))
        out[b] = (torch.matmul(p, v) / p.sum(-1, keepdim=True)).reshape(hq, D).to(q.dtype)
    return out


def _heads(s):
    """Queries (scaled), keys and values in 32 bits, one row per value head."""
    c = s["case"]
    r = c["v_heads"] // c["k_heads"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["norm"]:
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + s["eps"])
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + s["eps"])
    return (q * s["scale"]).repeat_interleave(r, 1), k.repeat_interleave(r, 1), v


def _plain_delta(s, C=64):
    q, k, v = _heads(s)
    out = torch.zeros_like(s["out"])
    state = torch.zeros_like(s["state_out"])
    at = 0
    for n, slot in zip(s["lens"], s["slot_list"]):
        S = s["state_in"][slot]  # [H, dk, dv]
        if n:
            N = -(-n // C)

            def chunks(x):  # [n, H, ...] -> [N, H, C, ...], zeros behind the end
                y = torch.zeros(N * C, *x.shape[1:], dtype=x.dtype, device="cuda")
                y[:n] = x[at:at + n]
                return y.unflatten(0, (N, C)).transpose(1, 2)

            Q, K, V = chunks(q), chunks(k), chunks(v)
            beta = chunks(s["beta"])
            # differences of long sums of the log decays: 64 bits
            cum = torch.cumsum(chunks(s["g"]).double(), -1)
            low = torch.tril(torch.ones(C, C, dtype=torch.bool, device="cuda"))
            diff = (cum[..., :, None] - cum[..., None, :])
            decay = torch.where(low, torch.exp(torch.where(low, diff, torch.zeros_like(diff))),
                                torch.zeros_like(diff)).float()
            A = torch.tril(torch.matmul(K, K.transpose(-1, -2)) * decay * beta[..., None], -1)
            T = torch.eye(C, device="cuda").expand_as(A).clone()
            for i in range(1, C):  # rows of the inverse of I + A, top down
                T[..., i, :i] = -torch.matmul(A[..., i:i + 1, :i], T[..., :i, :i])[..., 0, :]
            P = torch.matmul(Q, K.transpose(-1, -2)) * decay
            start = torch.exp(cum).float()
            rest = torch.exp(cum[..., -1:] - cum).float()
            last = torch.exp(cum[..., -1]).float()
            U = torch.matmul(T, V * beta[..., None])
            W = torch.matmul(T, K * (beta * start)[..., None])
            Q = Q * start[..., None]
            K = (K * rest[..., None]).transpose(-1, -2)
            O = torch.empty_like(V)
            for j in range(N):
                D = U[j] - torch.matmul(W[j], S)
                O[j] = torch.matmul(Q[j], S) + torch.matmul(P[j], D)
                S = S * last[j][:, None, None] + torch.matmul(K[j], D)
            out[at:at + n] = O.transpose(1, 2).reshape(N * C, *v.shape[1:])[:n].to(out.dtype)
        state[slot] = S
        at += n
    return out, state


def _plain_step(s):
    q, k, v = _heads(s)
    slot = s["slots"].long()
    S = s["state_in"][slot] * torch.exp(s["g"])[..., None, None]
    d = (v - (S * k[..., None]).sum(-2)) * s["beta"][..., None]
    S = S + k[..., None] * d[..., None, :]
    out = (S * q[..., None]).sum(-2).to(s["type"])
    state = torch.zeros_like(s["state_out"])
    state[slot] = S
    return out, state


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "prompt":
        return _plain_prompt(state)
    if op == "append":
        fifteen = torch.full((), 15.0, device="cuda").expand(1)  # a tensor: the quotient is rounded once
        return _plain_quantise(state["k"], fifteen), _plain_quantise(state["v"], fifteen)
    if op == "decode":
        return _plain_decode(state)
    return _plain_delta(state) if op == "delta" else _plain_step(state)


# --------------------------------------------------------------------- work


def work(case):
    e = torch.finfo(_TYPES[case["type"]]).bits // 8
    op = case["op"]
    if op == "prompt":
        ql = _nums(case["lens"])
        kl = [max(0, a + b) for a, b in zip(ql, _nums(case["extra"]))]
        # query i of a sequence sees max(0, nk - nq + i + 1) keys
        pairs = sum(sum(range(max(1, nk - nq + 1), nk + 1)) if nk - nq < 0 else nq * (2 * nk - nq + 1) // 2
                    for nq, nk in zip(ql, kl))
        rows = 2 * sum(ql) * case["q_heads"] + 2 * sum(kl) * case["kv_heads"]
        return {"bytes": e * case["dim"] * rows, "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    if op == "append":
        n = sum(_nums(case["lens"])) * case["kv_heads"]
        # in; out to the cache; in from it; out as values
        return {"bytes": n * case["dim"] * (2 * e + 2 * 1.25 + 8), "flops": n * case["dim"] * 2 * 8}
    if op == "decode":
        lens = _nums(case["lens"])
        return {"bytes": sum(lens) * case["kv_heads"] * 5 * case["dim"] // 4
                + 2 * e * len(lens) * case["q_heads"] * case["dim"],
                "flops": 4 * sum(lens) * case["q_heads"] * case["dim"]}
    hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["dk"], case["dv"]
    lens = _nums(case["lens"]) if op == "delta" else [1] * case["seqs"]
    T, B = sum(lens), len(lens)
    return {"bytes": T * (e * (2 * hk * dk + 2 * hv * dv) + 8 * hv) + 8 * B * hv * dk * dv,
            "flops": 6 * T * hv * dk * dv}


# ------------------------------------------------- the definitions in 64 bits


def _exact_prompt(s):
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    hq, hk = s["case"]["q_heads"], s["case"]["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    a = b = 0
    for nq, nk in zip(s["ql"], s["kl"]):
        for h in range(hq):
            kk, vv = k[b:b + nk, h // (hq // hk)], v[b:b + nk, h // (hq // hk)]
            for i in range(max(0, nq - nk), nq, 4096):  # the first nq - nk queries see no key
                e = min(nq, i + 4096)
                z = (q[a + i:a + e, h] @ kk.T) * s["scale"]
                z.masked_fill_(torch.triu(torch.ones(e - i, nk, dtype=torch.bool, device="cuda"),
                                          diagonal=nk - nq + i + 1), float("-inf"))
                out[a + i:a + e, h] = torch.softmax(z, -1) @ vv
        a, b = a + nq, b + nk
    return out


def _exact_append(x):
    # the format's own roundings (32-bit difference and quotient, 16-bit step and
    # minimum), each from a 64-bit result; codes from 64-bit quotients
    import numpy as np

    a = x.double().cpu().numpy()
    a = np.clip(a.reshape(*a.shape[:-1], -1, 32), -65504.0, 65504.0)
    m = a.min(-1, keepdims=True).astype(np.float32).astype(np.float16).astype(np.float64)
    span = (a.max(-1, keepdims=True) - m).astype(np.float32).astype(np.float64)
    d = (span / 15.0).astype(np.float32).astype(np.float16).astype(np.float64)
    code = np.clip(np.rint(np.divide(a - m, d, out=np.zeros_like(a), where=d > 0)), 0, 15)
    return torch.from_numpy((m + d * code).reshape(*x.shape)).cuda()


def _exact_decode(s):
    D, hq, hk = s["case"]["dim"], s["case"]["q_heads"], s["case"]["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["ll"]):
        for h in range(hk if n else 0):
            pages = s["table"][b, :(n + s["page"] - 1) // s["page"]].long()
            k, v = _unpack(s["cache"][pages, h].reshape(-1, 20 * D), D, torch.float64)
            r = hq // hk
            z = s["q"][b, h * r:(h + 1) * r].double() @ k[:n].T * s["scale"]
            out[b, h * r:(h + 1) * r] = torch.softmax(z, -1) @ v[:n]
    return out


def _exact_delta(s):
    # token by token: S <- a S; S <- S + k (beta (v - S^T k))^T; o = S^T q
    c = s["case"]
    r = c["v_heads"] // c["k_heads"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if c["norm"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + s["eps"])
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + s["eps"])
    q = q.repeat_interleave(r, 1) * s["scale"]
    k = k.repeat_interleave(r, 1)
    a, beta = torch.exp(s["g"].double()), s["beta"].double()
    out = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    state = torch.zeros(s["state_out"].shape, dtype=torch.float64, device="cuda")
    cu = _cu(s["lens"])
    # sequences go together while they last, longest first
    order = sorted(range(len(s["lens"])), key=lambda i: -s["lens"][i])
    slot = torch.tensor([s["slot_list"][i] for i in order], device="cuda")
    first = torch.tensor([cu[i] for i in order], device="cuda")
    S = s["state_in"][slot].double()
    for t in range(max(s["lens"])):
        n = sum(1 for i in order if s["lens"][i] > t)
        row = first[:n] + t
        x = S[:n] * a[row][..., None, None]
        kt = k[row]
        d = (v[row] - torch.matmul(kt[..., None, :], x)[..., 0, :]) * beta[row][..., None]
        x = x + kt[..., None] * d[..., None, :]
        S[:n] = x
        out[row] = torch.matmul(q[row][..., None, :], x)[..., 0, :]
    state[slot] = S
    return out, state


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt":
        return _exact_prompt(s)
    if op == "append":
        return _exact_append(s["k"]), _exact_append(s["v"])
    if op == "decode":
        return _exact_decode(s)
    return _exact_delta(s)
