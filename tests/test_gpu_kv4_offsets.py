"""Appending to and loading from the 4-bit cache with offsets that do not ascend within the rows: reported, nothing
out of range read or written."""
import numpy as np
import pytest
import torch

import mixer_refs as R
import test_gpu_kv4 as TK
from test_gpu_kv4 import P  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("cu", [
    [0, 20, 10, 60],               # falls
    [0, 20, 40, 61],               # past the rows
    [-1, 20, 40, 60],              # in front of them
    [60, 40, 20, 0],
    [0, 20, 2147483647, 60],
    [-2147483648, 20, 40, 60],
    [5, 5, 5, 4],
])
def test_offsets_that_do_not_ascend_are_reported(P, cu):
    rng = np.random.default_rng(1)
    lens, page = [20, 20, 20], 16
    k, v, tab, cache = TK._fill(P, rng, torch.float32, 128, 2, page, lens, [0, 0, 0])
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert P.redlite_kv4_append(k, v, c, st, tab, cache, page, status) == P.REDLITE_OK
    assert int(status) & P.REDLITE_STATUS_BAD_LENGTH
    status.zero_()
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    assert P.redlite_kv4_load(cache, page, tab, c, st, ko, vo, status) == P.REDLITE_OK
    assert int(status) & P.REDLITE_STATUS_BAD_LENGTH
    # a row is some token of its sequence, zeros (reported) or left alone
    for x, y in ((k, ko), (v, vo)):
        ref = torch.tensor(R.dequantise(*R.quantise(x.double().cpu().numpy())), dtype=torch.float32).cuda()
        same = (y == ref).flatten(1).all(1) | (y == 7).flatten(1).all(1) | (y == 0).flatten(1).all(1)
        assert bool(same.all()) or cu[0] != 0  # (rows of a sequence that starts in front of them lie further on)


@gpu
@pytest.mark.parametrize("n,broken", [(1, 0), (700, 0), (700, 256), (700, 699)])
def test_any_broken_sequence_is_reported(P, n, broken):
    """One offset past the rows among many; and none: no report."""
    lens = np.ones(n, int)
    k = torch.randn(n, 1, 128, device="cuda")
    tab = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    cache = torch.zeros(n, 1, 1, 2560, dtype=torch.uint8, device="cuda")
    st = torch.zeros(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = R.cu(lens)
    for load in (False, True):
        f = (lambda c: P.redlite_kv4_load(cache, 16, tab, c, st, k, k.clone(), status)) if load else \
            (lambda c: P.redlite_kv4_append(k, k, c, st, tab, cache, 16, status))
        assert f(cu) == P.REDLITE_OK and int(status) == 0
        bad = cu.clone()
        bad[broken + 1] = n + 1
        assert f(bad) == P.REDLITE_OK and int(status) == P.REDLITE_STATUS_BAD_LENGTH
        status.zero_()
