"""Host side of the 4-bit cache (no GPU): refusals of the C ABI before any
launch, refusals of the binding, and the plain quantisation that the GPU
tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import kv4_ref as ref

P16 = 1 << 20  # any non-null 16-byte aligned address: refused before use


def cache(**kw):
    a = dict(k=P16, v=P16, k_scale=P16, v_scale=P16, dt=api.SD_BF16,
             num_pages=4, page_size=16, heads=2, head_dim=64, group=32,
             page_stride=1024, scale_stride=256, block_table=P16, max_pages=3)
    a.update(kw)
    return api._PagedKV4Struct(*[a[f] for f, _ in
                                 api._PagedKV4Struct._fields_])


def append(c=None, **kw):
    a = dict(k=P16, ks=128, v=P16, vs=128, q=P16, qs=256, hq=4, start=P16,
             kv=P16, pos=None, cs=P16, max_pos=64, rot=64, inter=0, B=2,
             total=3, out=P16)
    a.update(kw)
    st = c if c is not None else cache()
    return api.lib().sd_kv4_append(
        ctypes.addressof(st), a["k"], a["ks"], a["v"], a["vs"], a["q"],
        a["qs"], a["hq"], a["start"], a["kv"], a["pos"], a["cs"],
        a["max_pos"], a["rot"], a["inter"], a["B"], a["total"], a["out"],
        None, None)


def read(c=None, **kw):
    a = dict(start=P16, kv=P16, B=2, total=3, k=P16, ks=128, v=P16, vs=128)
    a.update(kw)
    st = c if c is not None else cache()
    return api.lib().sd_kv4_read(
        ctypes.addressof(st), a["start"], a["kv"], a["B"], a["total"],
        a["k"], a["ks"], a["v"], a["vs"], None, None)


def attend(c=None, **kw):
    a = dict(q=P16, qs=256, hq=4, start=P16, kv=P16, mask=None, words=0, B=2,
             total=3, max_q=2, scale=0.125, out=P16, ws=P16, nws=1 << 40)
    a.update(kw)
    st = c if c is not None else cache()
    return api.lib().sd_kv4_attention(
        a["q"], a["qs"], a["hq"], ctypes.addressof(st), a["start"], a["kv"],
        a["mask"], a["words"], a["B"], a["total"], a["max_q"], a["scale"],
        a["out"], None, None, a["ws"], a["nws"], None)


INVALID, UNSUPPORTED = api.SD_ERR_INVALID_ARG, api.SD_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad,code", [
    (dict(dt=api.SD_F32), INVALID), (dict(num_pages=-1), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=12), UNSUPPORTED),
    (dict(heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=0), UNSUPPORTED), (dict(group=16), INVALID),
    (dict(group=0), INVALID), (dict(group=128), INVALID),
    (dict(max_pages=-1), INVALID), (dict(max_pages=1 << 28), INVALID),
    (dict(page_stride=1008), INVALID), (dict(page_stride=1032), INVALID),
    (dict(scale_stride=240), INVALID), (dict(scale_stride=264), INVALID),
    (dict(page_stride=-1024, num_pages=1), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k_scale=None), INVALID), (dict(v_scale=P16 + 8), INVALID),
    (dict(block_table=None), INVALID)])
def test_bad_cache_descriptions_are_refused(bad, code):
    assert append(cache(**bad)) == code
    assert read(cache(**bad)) == code
    assert attend(cache(**bad)) == code


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(total=-1), dict(hq=-1), dict(q=None), dict(out=None),
    dict(rot=63), dict(rot=66), dict(rot=0), dict(max_pos=0), dict(k=None),
    dict(start=None), dict(kv=None), dict(ks=127), dict(vs=127),
    dict(qs=255)])
def test_append_refusals(bad):
    assert append(**bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(total=-1), dict(start=None), dict(kv=None), dict(k=None),
    dict(v=None), dict(ks=112), dict(vs=136), dict(k=P16 + 16)])
def test_read_refusals(bad):
    assert read(**bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(total=-1), dict(max_q=-1), dict(hq=3), dict(hq=0),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(mask=P16, words=0), dict(q=None),
    dict(out=None), dict(q=P16 + 2), dict(qs=252), dict(qs=260),
    dict(out=P16 + 16), dict(ws=None), dict(nws=1000), dict(ws=P16 + 16),
    dict(scale=3e38), dict(total=1 << 30)])
def test_attention_refusals(bad):
    assert attend(**bad) == INVALID


def test_empty_calls_are_no_ops():
    for kw in (dict(B=0), dict(total=0)):
        assert append(**kw) == api.SD_OK
        assert read(**kw) == api.SD_OK
        assert attend(**kw) == api.SD_OK


def test_the_binding_refuses():
    table = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.PagedKV4.empty(2, 16, 1, 64, table, torch.bfloat16)
    with pytest.raises(ValueError, match="group"):
        api.PagedKV4.empty(2, 16, 1, 64, table, torch.bfloat16, group=128)
    for f in (api.kv4_append, api.kv4_attention):
        with pytest.raises(TypeError, match="PagedKV4"):
            f(object.__new__(api.PagedKV), *[table] * 4) \
                if f is api.kv4_append else \
                f(table, object.__new__(api.PagedKV), table, table)
    with pytest.raises(TypeError, match="PagedKV4"):
        api.kv4_read(object.__new__(api.PagedKV), table, table, 1)
    four = object.__new__(api.PagedKV4)
    with pytest.raises(TypeError, match="a PagedKV$"):
        api.kv_append(four, table, table, table, table)
    with pytest.raises(TypeError, match="a PagedKV$"):
        api.paged_attention(table, four, table, table)


# -------------------------------------------------- the plain quantisation
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("by", [1e-3, 1.0, 300.0])
def test_quantised_numbers_are_half_a_step_away(group, by):
    r = np.random.default_rng(group)
    x = (r.standard_normal((50, 128)) * by).astype(np.float32)
    n, pair = ref.quantise(x, group)
    y = ref.values(n, pair)
    g = x.reshape(50, -1, group).astype(np.float64)
    step = (g.max(-1) - g.min(-1)) / 15
    # half a step; b is rounded to 1/32 of a step (72 steps and the group's
    # offset, at most 15 more, lie below 2^7 steps, where fp16 numbers are
    # 2^-4 apart), a moves the ends by 15 steps x 2^-11 and, near fp16's least
    # numbers, 15 x 2^-25; the number itself is rounded
    tol = step * (0.5 + 1 / 32 + 15 * 2.0 ** -11) + 80 * 2.0 ** -25
    err = np.abs(y - x).reshape(50, -1, group).max(-1)
    assert (err <= tol + 2.0 ** -11 * np.abs(g).max(-1)).all()
    assert n.max() == 15 and n.min() == 0


def test_codes_survive_packing():
    n = np.random.default_rng(1).integers(0, 16, (7, 64)).astype(np.uint8)
    np.testing.assert_array_equal(ref.unpack(ref.pack(n)), n)
    word = ref.pack(np.arange(8, dtype=np.uint8)).view("<u4")
    assert int(word[0]) == 0x75316420


def test_groups_at_the_ends():
    x = np.zeros((6, 32))
    x[1] = 7.25               # one number: held exactly
    x[2, 3] = np.nan
    x[3, 3] = np.inf
    x[4, :2] = 1e6, -1e6      # beyond what a group holds
    x[5] = 1e-9               # below fp16
    n, pair = ref.quantise(x, 32)
    y = ref.values(n, pair)
    assert (y[0] == 0).all() and (y[1] == 7.25).all() and (y[5] == 0).all()
    assert np.isnan(y[2]).all() and np.isnan(y[3]).all()
    # a is rounded to 0.5 (numbers from 512 on), b to 32: 15 and 79 of them
    assert abs(y[4, 0] - 6144) <= 64 and abs(y[4, 1] + 6144) <= 64
