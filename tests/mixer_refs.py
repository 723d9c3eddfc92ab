"""64-bit references of the token mixers and the stored form of the 4-bit
cache, from the definitions in include/redlite_moe.h; no code shared with the
library."""
import numpy as np
import torch

HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}


def cu(lens, device="cuda", first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + first, dtype=torch.int32, device=device)


# ------------------------------------------------------------ 4-bit cache


def quantise(x):
    """(codes, d, m) of x [..., D] (float64 array holding the inputs exactly)."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    broken = ~np.isfinite(g).all(-1)
    g = np.clip(np.where(broken[..., None], 0.0, g), -65504.0, 65504.0)
    m = g.min(-1).astype(np.float32).astype(np.float16)
    span = (g.max(-1) - m.astype(np.float64)).astype(np.float32)
    d = (span / np.float32(15)).astype(np.float32).astype(np.float16)
    d64, m64 = d.astype(np.float64)[..., None], m.astype(np.float64)[..., None]
    c = np.zeros_like(g)
    np.divide(g - m64, d64, out=c, where=d64 > 0)
    d[broken] = m[broken] = np.nan
    return np.clip(np.rint(c), 0, 15).astype(np.uint8), d, m


def dequantise(codes, d, m):
    v = m.astype(np.float64)[..., None] + d.astype(np.float64)[..., None] * codes
    return v.reshape(*v.shape[:-2], -1)


class Cache:
    """A cache filled by the reference: random codes and steps, laid out
    element by element as the header's stored form says."""

    @classmethod
    def zeros(cls, n_pages, heads, D, page):
        C = cls.__new__(cls)
        C.D, C.page, C.heads, C.n_pages = D, page, heads, n_pages
        shape = (n_pages, heads, page // 16, 16, D // 32)
        C.codes = [np.zeros(shape + (32,), np.uint8) for _ in range(2)]
        C.d = [np.zeros(shape, np.float16) for _ in range(2)]
        C.m = [np.zeros(shape, np.float16) for _ in range(2)]
        return C

    def __init__(self, rng, n_pages, heads, D, page, mag=1.0):
        self.D, self.page, self.heads, self.n_pages = D, page, heads, n_pages
        ng, nt = D // 32, page // 16
        shape = (n_pages, heads, nt, 16)
        self.codes = [rng.integers(0, 16, shape + (ng, 32), dtype=np.uint8) for _ in range(2)]
        self.d = [(mag * rng.uniform(0.05, 0.4, shape + (ng,))).astype(np.float16) for _ in range(2)]
        self.m = [(-7.5 * self.d[i].astype(np.float32) + mag * 0.3 * rng.standard_normal(shape + (ng,))).astype(np.float16)
                  for i in range(2)]
        self.pack()

    def pack(self):
        D, ng = self.D, self.D // 32
        n, h, nt = self.d[0].shape[:3]
        by = np.zeros((n, h, nt, 20 * D), np.uint8)
        for t in range(16):
            hh, r = t >> 3, t & 7
            for g in range(ng):
                for c in range(4):
                    y = hh * ng + g
                    at = 4 * ((y >> 2) * 128 + (4 * r + c) * 4 + (y & 3))
                    v = self.codes[0][..., t, g, 8 * c:8 * c + 8]
                    for e in range(4):
                        by[..., at + e] = v[..., 2 * e] | (v[..., 2 * e + 1] << 4)
                at = 8 * D + 4 * (t * ng + g)
                by[..., at:at + 2] = self.d[0][..., t, g, None].view(np.uint8)
                by[..., at + 2:at + 4] = self.m[0][..., t, g, None].view(np.uint8)
                for rr in range(8):
                    x = (2 * hh + (t & 1)) * ng + g
                    at = 10 * D + 2 * ((x >> 3) * 256 + (4 * rr + ((t & 7) >> 1)) * 8 + (x & 7))
                    v = self.codes[1][..., t, g, 4 * rr:4 * rr + 4]
                    by[..., at] = v[..., 0] | (v[..., 1] << 4)
                    by[..., at + 1] = v[..., 2] | (v[..., 3] << 4)
                at = 18 * D + 2 * (t * ng + g)
                by[..., at:at + 2] = self.d[1][..., t, g, None].view(np.uint8)
                by[..., at + D:at + D + 2] = self.m[1][..., t, g, None].view(np.uint8)
        self.bytes = by

    def values(self, which, pages, n, head):
        """[n, D] float64 values of the first n tokens on these pages."""
        k = dequantise(self.codes[which][pages, head], self.d[which][pages, head], self.m[which][pages, head])
        return k.reshape(-1, self.D)[:n]

    def steps(self, which, pages, n, head):
        d = self.d[which][pages, head].astype(np.float64).reshape(-1, self.D // 32)[:n]
        m = self.m[which][pages, head].astype(np.float64).reshape(-1, self.D // 32)[:n]
        return d, m


def table(rng, lens, page, spare=0):
    """(n_pages, int32 block table) with pages in random order, -1 where none is needed."""
    need = [-(-n // page) for n in lens]
    n = sum(need) + spare
    order = rng.permutation(max(n, 1))
    t = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for i, c in enumerate(need):
        t[i, :c] = order[at:at + c]
        at += c
    return max(n, 1), t


def softmax(z):
    p = np.exp(z - z.max(-1, keepdims=True))
    return p / p.sum(-1, keepdims=True)


# -------------------------------------------------------- gated delta rule


def delta(q, k, v, g, beta, lens, state, scale, eps):
    """(out, states, growth) in 64 bits, token by token.  q, k [T, Hk, dk], v [T, Hv, dv], g, beta [T, Hv],
    state [n, Hv, dk, dv]: the states in front of each sequence.  growth, per sequence and head: the largest
    norm the state reaches."""
    hv, r = v.shape[1], v.shape[1] // k.shape[1]
    if eps >= 0:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
    q, k = np.repeat(q, r, 1) * scale, np.repeat(k, r, 1)
    out, S_out = np.zeros(v.shape), state.copy()
    t = 0
    big = np.zeros((len(lens), hv))
    for s, n in enumerate(lens):
        S = S_out[s]
        big[s] = np.abs(S).max((1, 2))
        for _ in range(n):
            S *= np.exp(g[t])[:, None, None]
            d = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
            S += k[t][:, :, None] * d[:, None, :]
            out[t] = np.einsum("hkv,hk->hv", S, q[t])
            big[s] = np.maximum(big[s], np.abs(S).max((1, 2)))
            t += 1
    return out, S_out, big
