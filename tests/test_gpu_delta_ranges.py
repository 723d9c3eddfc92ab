"""The gated delta rule where a state comes and goes: what is left of it is scaled without leaving fp32."""
import numpy as np
import pytest
import torch

import mixer_refs as R
import test_gpu_delta as TD
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("t,top", [(torch.float16, 2.0 ** 15)] + [(t, 2.0 ** e) for t in TD.TYPES[:2]
                                                                    for e in (15, 40, 100)])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
@pytest.mark.parametrize("rest", [0.0, 2.0 ** -80])
def test_a_large_state_that_is_taken_back(P, t, dk, dv, rest, top):
    """A large value and its removal in one chunk (the state is exactly zero, or a small one in other rows), a chunk
    without updates, then ordinary tokens.  Every number up to there is a power of two, so nothing is rounded; what
    follows is held to the bounds of ordinary tokens."""
    rng = np.random.default_rng(dk)
    n, hv = 200, 2
    k = np.zeros((n, 1, dk))
    k[:128, 0, 0] = 1
    k[128:, 0] = rng.standard_normal((72, dk))
    k[128:] /= np.sqrt((k[128:] ** 2).sum(-1, keepdims=True))
    q = rng.standard_normal((n, 1, dk)) / np.sqrt(dk)
    v = np.zeros((n, hv, dv))
    v[0] = top
    v[128:] = rng.standard_normal((72, hv, dv))
    g, beta = np.zeros((n, hv)), np.zeros((n, hv))
    beta[:2] = 1
    beta[128:] = 0.5
    dev = [torch.tensor(x).to(t).cuda() for x in (q, k, v)]
    dev += [torch.tensor(x, dtype=torch.float32).cuda() for x in (g, beta)]
    state = torch.zeros(1, hv, dk, dv, device="cuda")
    state[:, :, 3:] = rest
    out_state = torch.zeros_like(state)
    out = TD._prefill(P, dev, R.cu([n]), state, out_state, None, 1.0, -1.0)
    ref, S, big = R.delta(*[TD._host(x) for x in dev], [n], TD._host(state), 1.0, -1.0)
    got, gs = TD._host(out), TD._host(out_state)
    assert np.isfinite(got).all() and np.isfinite(gs).all()
    # the first output is q top, the others up to the chunk's end nothing of it: two fp16 parts of each operand
    assert (np.abs(got[0] - ref[0]) <= (R.HALF_ULP[t] + 2.0 ** -11) * np.abs(ref[0])).all()
    lim, slim = TD._limits(ref[64:], np.abs(S).max((2, 3)), [136], 1.0, dk, np.abs(v[128:]).max(), t)
    assert (np.abs(got[64:] - ref[64:]) <= lim).all(), float((np.abs(got[64:] - ref[64:]) / lim).max())
    assert (np.abs(gs - S) <= slim).all(), float((np.abs(gs - S) / slim).max())
