"""sd_kv_append against the 64-bit formula: types, both pairings, partial
rotation, strided rows, page orders, positions, lengths of zero and one,
and data it has to refuse row by row."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import operators_ref as ref
from tests.test_gpu_canaries import GuardedTorch

pytestmark = pytest.mark.gpu


def run(P, Hq, rot, *, interleaved=False, positions=None, fused=True,
        max_pos=None, guard=None):
    """Append the batch's chunks; compare everything: q_out, the written
    slots, and that no other slot changed."""
    Hkv, D, dt = P.heads, P.dim, P.dtype
    k0, v0 = P.to_gpu(P.k), P.to_gpu(P.v)
    cache = api.PagedKV(k0, v0, P.table.cuda())
    x = P.rows(Hq + 2 * Hkv)
    start, kv = P.lengths()
    tab = None
    if rot:
        tab = ref.cos_sin_table(max_pos or max(P.kv + [1]), rot)
    g = x.cuda()
    q, k, v = g[:, :Hq], g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.kv_append(
        cache, k, v, start, kv, q=q if Hq else None,
        cos_sin=None if tab is None else tab.cuda(),
        positions=None if positions is None else torch.tensor(
            positions, dtype=torch.int32, device="cuda"),
        interleaved=interleaved, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    index = np.concatenate([np.arange(m - n, m) for n, m in zip(P.n, P.kv)]
                           or [[]]).astype(int)
    pos = index if positions is None else positions
    x64 = ref.f64(x)
    if rot:
        y, size = ref.rotate(x64[:, :Hq + Hkv], ref.f64(tab), pos,
                             interleaved)
    else:
        y, size = x64[:, :Hq + Hkv], np.zeros_like(x64[:, :Hq + Hkv])
    tol = ref.append_tol(y, size, dt)
    if not rot:
        tol = np.zeros_like(tol)
    if Hq:
        assert (np.abs(ref.f64(out) - y[:, :Hq]) <= tol[:, :Hq]).all()
    kc, vc = ref.f64(cache.k), ref.f64(cache.v)
    ok, ov = ref.f64(P.k), ref.f64(P.v)
    seq = np.repeat(np.arange(len(P.n)), P.n)
    for r, (b, j) in enumerate(zip(seq, index)):
        p, t = P.slot(b, j)
        assert (np.abs(kc[p, t] - y[r, Hq:]) <= tol[r, Hq:]).all()
        np.testing.assert_array_equal(vc[p, t], x64[r, Hq + Hkv:])
        kc[p, t], vc[p, t] = ok[p, t], ov[p, t]
    np.testing.assert_array_equal(kc, ok)
    np.testing.assert_array_equal(vc, ov)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (128, 64), (64, 24),
                                   (80, 80), (96, 20), (72, 0), (10, 6),
                                   (9, 4), (256, 256)])
def test_types_and_rotations(dtype, interleaved, D, rot):
    P = ref.Paged([1, 3, 0, 5], [7, 3, 4, 30], 2, D, 8, dtype, seed=D + rot)
    run(P, 6, rot, interleaved=interleaved)


@pytest.mark.parametrize("Hq,Hkv", [(0, 1), (1, 1), (5, 1), (71, 1), (12, 4),
                                    (3, 3)])
@pytest.mark.parametrize("fused", [False, True])
def test_heads_and_strides(Hq, Hkv, fused):
    P = ref.Paged([2, 1], [2, 17], Hkv, 64, 16, torch.bfloat16, seed=Hq)
    run(P, Hq, 64, fused=fused)


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("page", [8, 24, 128])
def test_page_orders(head_major, page):
    P = ref.Paged([17, 1, 40], [50, 129, 40], 3, 64, page, torch.float16,
                  seed=page, head_major=head_major)
    run(P, 3, 32)


def test_one_token_of_one_sequence_and_many_tokens():
    run(ref.Paged([1], [1], 1, 64, 8, torch.bfloat16, seed=1), 1, 64)
    run(ref.Paged([700, 1], [700, 3], 2, 128, 64, torch.bfloat16, seed=2), 4,
        128)


def test_many_sequences():
    r = np.random.default_rng(6)
    n = r.integers(0, 3, 1100)
    run(ref.Paged(n.tolist(), (n + r.integers(0, 20, 1100)).tolist(), 1, 64,
                  8, torch.bfloat16, seed=21), 1, 64)


def test_tree_positions():
    """Nodes of a token tree rotate by depth, not by slot."""
    P = ref.Paged([5, 3], [25, 3], 2, 64, 8, torch.bfloat16, seed=9)
    run(P, 4, 64, positions=[20, 21, 21, 22, 22, 0, 1, 1], max_pos=23)


def test_rows_it_cannot_place():
    """A bad page, a bad position, a bad key count and an uncovered row: the
    cache is untouched there, q_out is zero, the bits are set; the other
    sequences are as ever."""
    B, H, D = 4, 1, 64
    P = ref.Paged([2, 2, 2, 2], [4, 12, 4, 4], H, D, 8, torch.bfloat16,
                  seed=4, fill=0.0)
    table = P.table.clone()
    table[1, 1] = 10 ** 6  # its keys 8..: the chunk's own page
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), table.cuda())
    start, kv = P.lengths()
    kv[2] = 1  # fewer keys than new tokens
    x = P.rows(3 * H)
    x = torch.cat([x, torch.ones(1, 3 * H, D, dtype=x.dtype)]).cuda()
    tab = ref.cos_sin_table(50, D).cuda()
    pos = torch.tensor([2, 3, 10, 11, 0, 1, 49, 50, 0], dtype=torch.int32,
                       device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = cache.k.clone(), cache.v.clone()
    out = api.kv_append(cache, x[:, 1:2], x[:, 2:], start, kv, q=x[:, :1],
                        cos_sin=tab, positions=pos, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == api.DEV_BAD_PAGE | api.DEV_BAD_LENGTH | \
        api.DEV_BAD_POSITION
    assert bool((out[[2, 3, 4, 5, 7]] == 0).all())
    assert bool((out[[0, 1, 6]] != 0).any(-1).all())
    changed = ((cache.k != before[0]) | (cache.v != before[1])).any(-1).any(-1)
    want = {P.slot(0, 2), P.slot(0, 3), P.slot(3, 2)}
    assert {tuple(i) for i in changed.nonzero().tolist()} == want


@pytest.mark.parametrize("D,rot", [(64, 64), (10, 6), (96, 20)])
def test_no_write_outside_the_buffers(monkeypatch, D, rot):
    guard = GuardedTorch()
    monkeypatch.setattr(api, "torch", guard)
    P = ref.Paged([3, 1], [19, 8], 2, D, 8, torch.bfloat16, seed=6)
    shape = P.k.shape
    k = guard.empty(shape, dtype=P.dtype, device="cuda")
    v = guard.empty(shape, dtype=P.dtype, device="cuda")
    k.copy_(P.k)
    v.copy_(P.v)
    x = P.rows(8).cuda()
    start, kv = P.lengths()
    api.kv_append(api.PagedKV(k, v, P.table.cuda()), x[:, 4:6], x[:, 6:],
                  start, kv, q=x[:, :4],
                  cos_sin=ref.cos_sin_table(19, rot).cuda())
    assert guard.check() == 3


def test_another_stream():
    """The call runs on the current stream, after what is queued there."""
    P = ref.Paged([64], [64], 2, 64, 16, torch.bfloat16, seed=8, fill=0.0)
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    x = P.rows(4).cuda()
    start, kv = P.lengths()
    want = None
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(5):
            big = (big @ big) * 1e-3
        y = x + (big[0, 0] * 0).to(x.dtype)
        api.kv_append(cache, y[:, :2], y[:, 2:], start, kv)
    s.synchronize()
    got = cache.k[P.table[0, :4].cuda().long()].reshape(64, 2, 64)
    want = x[:, :2] + (big[0, 0] * 0).to(x.dtype)
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


@pytest.mark.parametrize("bad,err", [
    (lambda: torch.zeros(1, dtype=torch.int32), ValueError),
    (lambda: torch.zeros(1, dtype=torch.int64, device="cuda"), TypeError),
    (lambda: torch.zeros(0, dtype=torch.int32, device="cuda"), ValueError),
    (lambda: torch.zeros(4, dtype=torch.int32, device="cuda")[::2],
     ValueError)])
def test_status_words_are_checked(bad, err):
    """By every call that this binding has around the verify step: the kernels
    write to the status word's address."""
    P = ref.Paged([1], [1], 1, 64, 8, torch.bfloat16, seed=1, fill=0.0)
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    x, st = P.rows(1).cuda(), bad()
    z = torch.zeros(2, 50, device="cuda")
    w = torch.zeros(2, device="cuda")
    top = z[:, :3].contiguous(), torch.zeros(2, 3, dtype=torch.int32,
                                             device="cuda")
    for call in (lambda: api.kv_append(cache, x, x, *P.lengths(), status=st),
                 lambda: api.paged_attention(x, cache, *P.lengths(),
                                             status=st),
                 lambda: api.distill_topk(z, *top, status=st),
                 lambda: api.distill_topk_backward(z, w, *top, w, status=st),
                 lambda: api.distill_topk_step(z, *top, w, status=st)):
        with pytest.raises(err, match="status"):
            call()
