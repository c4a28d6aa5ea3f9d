"""Host side of the paged-cache, chunk-attention and distillation entry
points (no GPU): refusals of the C ABI before any launch, refusals of the
binding, and the 64-bit formulas the GPU tests compare with, checked against
differences and against torch."""
import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import operators_ref as ref

P16 = 1 << 20  # any non-null 16-byte aligned address: refused before use


def cache(**kw):
    a = dict(k=P16, v=P16, dt=api.SD_BF16, num_pages=4, page_size=16, heads=2,
             head_dim=64, page_stride=2048, token_stride=128, head_stride=64,
             block_table=P16, max_pages=3)
    a.update(kw)
    return api._PagedKVStruct(*[a[f] for f, _ in api._PagedKVStruct._fields_])


def append(c=None, **kw):
    a = dict(k=P16, ks=128, v=P16, vs=128, q=P16, qs=256, hq=4, start=P16,
             kv=P16, pos=None, cs=P16, max_pos=64, rot=64, inter=0, B=2,
             total=3, out=P16)
    a.update(kw)
    st = c if c is not None else cache()
    return api.lib().sd_kv_append(
        ctypes.addressof(st), a["k"], a["ks"], a["v"], a["vs"], a["q"],
        a["qs"], a["hq"], a["start"], a["kv"], a["pos"], a["cs"],
        a["max_pos"], a["rot"], a["inter"], a["B"], a["total"], a["out"],
        None, None)


def attend(c=None, **kw):
    a = dict(q=P16, qs=256, hq=4, start=P16, kv=P16, mask=None, words=0, B=2,
             total=3, max_q=2, scale=0.125, out=P16, ws=P16, nws=1 << 40)
    a.update(kw)
    st = c if c is not None else cache()
    return api.lib().sd_paged_attention(
        a["q"], a["qs"], a["hq"], ctypes.addressof(st), a["start"], a["kv"],
        a["mask"], a["words"], a["B"], a["total"], a["max_q"], a["scale"],
        a["out"], None, None, a["ws"], a["nws"], None)


BAD_CACHES = [
    (dict(dt=api.SD_F32), api.SD_ERR_INVALID_ARG),
    (dict(num_pages=-1), api.SD_ERR_INVALID_ARG),
    (dict(page_size=0), api.SD_ERR_INVALID_ARG),
    (dict(page_size=12), api.SD_ERR_UNSUPPORTED),
    (dict(heads=0), api.SD_ERR_INVALID_ARG),
    (dict(head_dim=0), api.SD_ERR_INVALID_ARG),
    (dict(max_pages=-1), api.SD_ERR_INVALID_ARG),
    (dict(max_pages=1 << 28), api.SD_ERR_INVALID_ARG),
    (dict(head_stride=-64), api.SD_ERR_INVALID_ARG),
    (dict(k=None), api.SD_ERR_INVALID_ARG),
    (dict(block_table=None), api.SD_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_cache_descriptions_are_refused(bad, code):
    assert append(cache(**bad)) == code
    assert attend(cache(**bad)) == code


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(total=-1), dict(hq=-1), dict(q=None), dict(out=None),
    dict(rot=63), dict(rot=66), dict(rot=0), dict(max_pos=0), dict(k=None),
    dict(start=None), dict(kv=None), dict(ks=127), dict(vs=127),
    dict(qs=255)])
def test_append_refusals(bad):
    assert append(**bad) == api.SD_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(total=-1), dict(max_q=-1), dict(hq=3), dict(hq=0),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(mask=P16, words=0), dict(q=None),
    dict(out=None), dict(q=P16 + 2), dict(qs=252), dict(qs=260),
    dict(out=P16 + 8), dict(out=P16 + 16), dict(ws=None), dict(nws=1000),
    dict(ws=P16 + 16), dict(scale=3e38), dict(total=1 << 30)])
def test_attention_refusals(bad):
    assert attend(**bad) == api.SD_ERR_INVALID_ARG


def test_attention_limits():
    assert attend(cache(head_dim=96), qs=4 * 96) == api.SD_ERR_UNSUPPORTED
    assert b"96" in api.lib().sd_last_error()
    assert attend(cache(k=P16 + 8)) == api.SD_ERR_INVALID_ARG
    assert attend(cache(token_stride=132)) == api.SD_ERR_INVALID_ARG


def test_empty_paged_calls_are_no_ops():
    for kw in (dict(B=0), dict(total=0)):
        assert append(**kw) == api.SD_OK
        assert attend(**kw) == api.SD_OK


@pytest.mark.parametrize("bad", [
    dict(dt=2), dict(N=-1), dict(V=0), dict(V=1 << 25), dict(K=0),
    dict(K=257), dict(T=0.0), dict(T=-1.0), dict(T=float("nan")),
    dict(stride=99), dict(z=None), dict(tl=None), dict(ti=None),
    dict(gstride=99), dict(g=None), dict(grad=None), dict(lse=None)])
def test_distill_refusals(bad):
    a = dict(z=P16, stride=100, dt=0, tl=P16, ti=P16, N=2, V=100, K=5, T=1.0,
             g=P16, loss=P16, lse=P16, grad=P16, gstride=100)
    a.update(bad)
    L = api.lib()
    back = L.sd_distill_topk_backward(
        a["z"], a["stride"], a["dt"], a["lse"], a["tl"], a["ti"], None,
        a["g"], a["N"], a["V"], a["K"], a["T"], a["grad"], a["gstride"],
        None, None)
    step = L.sd_distill_topk_step(
        a["z"], a["stride"], a["dt"], a["tl"], a["ti"], None, a["g"], a["N"],
        a["V"], a["K"], a["T"], a["loss"], a["lse"], a["grad"], a["gstride"],
        None, None)
    assert back == step == api.SD_ERR_INVALID_ARG
    if not set(bad) & {"gstride", "g", "grad"}:
        assert L.sd_distill_topk(
            a["z"], a["stride"], a["dt"], a["tl"], a["ti"], None, a["N"],
            a["V"], a["K"], a["T"], a["loss"], a["lse"], None,
            None) == api.SD_ERR_INVALID_ARG


def test_empty_distillation_is_a_no_op():
    assert api.lib().sd_distill_topk(None, 10, 0, None, None, None, 0, 10, 3,
                                     1.0, None, None, None, None) == api.SD_OK


def test_binding_refuses_host_tensors():
    z, tl = torch.zeros(2, 10), torch.zeros(2, 3)
    ti = torch.zeros(2, 3, dtype=torch.int32)
    w = torch.zeros(2)
    c = torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: api.distill_topk(z, tl, ti),
                 lambda: api.distill_topk_backward(z, w, tl, ti, w),
                 lambda: api.distill_topk_step(z, tl, ti, w),
                 lambda: api.PagedKV(c, c, torch.zeros(
                     1, 1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("T", [0.7, 1.0, 2.0])
@pytest.mark.parametrize("full", [False, True])
def test_gradient_formula_against_differences(T, full):
    """Central differences of the 64-bit loss, repeated and padded entries
    included: the error of a difference is h^2 / 6 times the third
    derivative, itself at most P / T^3."""
    r = np.random.default_rng(5)
    z = r.normal(size=(2, 17)) * 2
    logit = r.normal(size=(2, 6)) * 2
    ids = np.array([[3, 3, 0, 16, -1, 5], [1, 2, 2, 2, 9, 40]])
    tl = np.array([4.0, 3.5]) if full else None
    g = np.array([0.8, -1.3])
    got = ref.distill(z, logit, ids, T, tl, g)["grad"]
    P = 1.0 if tl is None else np.exp(logit / T - tl[:, None]).sum(1).max()
    h = 1e-4
    for n in range(2):
        for j in range(17):
            zp, zm = z.copy(), z.copy()
            zp[n, j] += h
            zm[n, j] -= h
            d = g[n] * (ref.distill(zp, logit, ids, T, tl)["loss"][n] -
                        ref.distill(zm, logit, ids, T, tl)["loss"][n]) / 2 / h
            assert abs(d - got[n, j]) < abs(g[n]) * P * h * h / T ** 3 + 1e-10


def test_formulas_against_torch():
    """The references against torch's own 64-bit operators: autograd of the
    KL, softmax attention, and rotation as complex multiplication."""
    g = torch.Generator().manual_seed(3)
    z = torch.randn(3, 40, generator=g, dtype=torch.float64,
                    requires_grad=True)
    t = torch.randn(3, 40, generator=g, dtype=torch.float64)
    top = t.topk(5, 1)
    p = torch.softmax(top.values / 0.9, 1)
    loss = (p * (p.log() - torch.log_softmax(z / 0.9, 1).gather(
        1, top.indices))).sum(1)
    loss.sum().backward()
    r = ref.distill(z.detach().numpy(), top.values.numpy(),
                    top.indices.numpy(), 0.9, None, np.ones(3))
    np.testing.assert_allclose(r["loss"], loss.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(r["grad"], z.grad.numpy(), atol=1e-14)

    P = ref.Paged([3, 2], [9, 20], 2, 64, 8, torch.bfloat16, 1,
                  device="cpu")
    q = P.rows(4)
    out, lse, _, _ = ref.attention(P, q, 0.2)
    for b in range(2):
        k = torch.tensor(P.gather(P.k, b)).repeat_interleave(2, 1)
        v = torch.tensor(P.gather(P.v, b)).repeat_interleave(2, 1)
        lo, n = P.start[b], P.n[b]
        s = torch.einsum("ihd,jhd->hij", q[lo:lo + n].double(), k) * 0.2
        mask = torch.ones(n, P.kv[b], dtype=torch.bool).tril(P.kv[b] - n)
        s = s.masked_fill(~mask, -np.inf)
        want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v)
        np.testing.assert_allclose(out[lo:lo + n], want.numpy(), atol=1e-12)
        np.testing.assert_allclose(lse[lo:lo + n],
                                   s.logsumexp(-1).T.numpy(), atol=1e-12)

    x = np.random.default_rng(0).normal(size=(2, 3, 10))
    tab = ref.f64(ref.cos_sin_table(7, 8))
    for inter in (False, True):
        y, _ = ref.rotate(x, tab, [6, 2], inter)
        for r_, pos in enumerate([6, 2]):
            a = x[r_][:, 0:8:2] if inter else x[r_][:, :4]
            b = x[r_][:, 1:8:2] if inter else x[r_][:, 4:8]
            w = (a + 1j * b) * (tab[pos, :4] + 1j * tab[pos, 4:])
            ya = y[r_][:, 0:8:2] if inter else y[r_][:, :4]
            yb = y[r_][:, 1:8:2] if inter else y[r_][:, 4:8]
            np.testing.assert_allclose(ya + 1j * yb, w, atol=1e-14)
        np.testing.assert_array_equal(y[:, :, 8:], x[:, :, 8:])


def test_workspace_buffers_are_not_shared(monkeypatch):
    """A device, stream and thread each have their own buffer, and one that a
    call outgrows stays allocated (a captured graph may write to it)."""
    import gc
    import threading
    import weakref
    stream = [1]
    monkeypatch.setattr(api, "_raw_stream", lambda device: stream[0])
    ws, dev = api.Workspace(), torch.device("cpu")
    a = ws.get(dev, 1000)
    assert ws.get(dev, 1000) is a and ws.get(dev, 10) is a
    stream[0] = 2
    b = ws.get(dev, 1000)
    assert b.data_ptr() != a.data_ptr()
    other = []
    t = threading.Thread(target=lambda: other.append(ws.get(dev, 1000)))
    t.start()
    t.join()
    assert other[0].data_ptr() not in (a.data_ptr(), b.data_ptr())
    stream[0] = 1
    assert ws.get(dev, 1000) is a
    old = weakref.ref(a)
    del a
    c = ws.get(dev, 5000)
    gc.collect()
    assert c.numel() >= 5000 and old() is not None
    assert ws.get(dev, 5000) is c


@pytest.mark.parametrize("name", ["k", "v", "block_table"])
def test_a_cache_keeps_the_tensors_it_describes(name):
    """Its C description holds their addresses: assigning another tensor would
    leave the old address in use after the old tensor is gone."""
    cache = api.PagedKV.__new__(api.PagedKV)
    with pytest.raises(AttributeError):
        setattr(cache, name, torch.zeros(1))
