"""The native marshaller of the token mixers: arguments that do not fit
together are refused before anything reaches a device."""
import pytest
import torch


@pytest.fixture(scope="module")
def P():
    from routed_expert_ffn_iq2_b200 import build

    build.build()
    import routed_expert_ffn_iq2_b200 as P

    return P


def test_host_tensors_are_refused(P):
    f = torch.zeros(2, 2, 128)
    i = torch.zeros(2, dtype=torch.int32)
    b = torch.zeros(1, 2, 1, 2560, dtype=torch.uint8)
    t = torch.zeros(1, 1, dtype=torch.int32)
    g = torch.zeros(2, 2)
    S = torch.zeros(2, 2, 128, 128)
    h = f.half()
    assert P.redlite_attn_prefill(h, h, h, i, i, h, 1.0) == P.REDLITE_EINVAL
    assert P.redlite_kv4_append(f, f, i, i[:1], t, b, 16) == P.REDLITE_EINVAL
    assert P.redlite_kv4_load(b, 16, t, i, i[:1], f, f) == P.REDLITE_EINVAL
    assert P.redlite_kv4_decode(f, b, 16, t, i, f, b, 1.0) == P.REDLITE_EINVAL
    assert P.redlite_delta_prefill(f, f, f, g, g, i, None, S, None, f, b, 1.0) == P.REDLITE_EINVAL
    assert P.redlite_delta_step(f, f, f, g, g, None, S, None, f, 1.0) == P.REDLITE_EINVAL


def test_what_is_no_tensor_raises(P):
    f = torch.zeros(2, 2, 128, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        P.redlite_attn_prefill(None, f, f, i, i, f, 1.0)
    with pytest.raises(TypeError):
        P.redlite_attn_prefill(f, f, [1], i, i, f, 1.0)
    with pytest.raises(TypeError):
        P._native._marshal().attn_prefill(f, f)


@pytest.mark.gpu
def test_arguments_that_do_not_fit(P):
    f = torch.zeros(2, 2, 128, device="cuda")
    h = f.half()
    i = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        P.redlite_attn_prefill(h, h, h, i, i, h, "x")
    for a in ((f.double(),) * 3, (h, h, f), (h, h, h[0]), (h, h.cpu(), h), (h, h, h[:, :, ::2])):
        assert P.redlite_attn_prefill(a[0], a[1], a[2], i, i, a[0], 1.0) == P.REDLITE_EINVAL
    assert P.redlite_attn_prefill(h, h, h, i.cpu(), i, h, 1.0) == P.REDLITE_EINVAL
    assert P.redlite_attn_prefill(h, h, h, i[:0], i[:0], h, 1.0) == P.REDLITE_EINVAL
    assert P.redlite_attn_prefill(h, h, h, i, i, h, 1.0, status=i.long()) == P.REDLITE_EINVAL
    b = torch.zeros(1, 2, 1, 2560, dtype=torch.uint8, device="cuda")
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    for page in (1 << 40, 0, 24):
        assert P.redlite_kv4_append(f, f, i, z, t, b, page) != P.REDLITE_OK
    assert P.redlite_kv4_append(f, f, i, z, t, b[..., :-1].contiguous(), 16) == P.REDLITE_EINVAL
    assert P.redlite_kv4_append(f, f, i, z, t[0], b, 16) == P.REDLITE_EINVAL
    assert P.redlite_kv4_append(f, f, i, i, t, b, 16) == P.REDLITE_EINVAL
    g = torch.zeros(2, 2, device="cuda")
    S = torch.zeros(2, 2, 128, 128, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for kw in (dict(g=g[:1]), dict(g=g.half()), dict(S=S[:, :, :64].contiguous()), dict(S=S[0]), dict(sl=i[:1])):
        a = dict(dict(g=g, S=S, sl=None), **kw)
        assert P.redlite_delta_step(f, f, f, a["g"], g, None, a["S"], a["sl"], f, 1.0) == P.REDLITE_EINVAL, kw
    assert P.redlite_delta_prefill(f, f, f, g, g, i, None, S, None, f, ws, 1.0) == P.REDLITE_ENOMEM
