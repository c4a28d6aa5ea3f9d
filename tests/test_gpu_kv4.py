"""The 4-bit cache on the GPU: the append's codes bit for bit against the
plain quantisation, the read-back's numbers, attention against the 64-bit
formula over the numbers that the codes stand for, data that is refused, and
the three together.  Pairs of numbers that no key owns are NaN."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import kv4_ref as ref
from tests import operators_ref as oref
from tests.test_gpu_canaries import GuardedTorch

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def lengths(n, kv):
    return (torch.tensor(np.concatenate([[0], np.cumsum(n)]),
                         dtype=torch.int32, device="cuda"),
            torch.tensor(kv, dtype=torch.int32, device="cuda"))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append
def rotate32(x, tab, pos, interleaved):
    """The rotation in 32-bit steps, each rounded by itself."""
    rot = tab.shape[1]
    h = rot // 2
    y = x.copy()
    c, s = tab[pos][:, None, :h], tab[pos][:, None, h:]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = ref.to32(ref.to32(a * c) - ref.to32(b * s))
    y[..., ib] = ref.to32(ref.to32(a * s) + ref.to32(b * c))
    return y


def run_append(P, Hq, rot, *, interleaved=False, positions=None, fused=True,
               x=None, apart_rows=0):
    """Append the batch's chunks and compare all of the cache: codes and pairs
    of the new tokens bit for bit, everything else as it was."""
    Hkv, D, dt = P.heads, P.dim, P.dtype
    cache = P.cache(api)
    was = [t.clone() for t in (cache.k, cache.v, cache.k_scale,
                               cache.v_scale)]
    if x is None:
        x = P.rows(Hq + 2 * Hkv)
    start, kv = P.lengths()
    tab = oref.cos_sin_table(max(P.kv + [1]), rot) if rot else None
    g = x.cuda()
    q, k, v = g[:, :Hq], g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.kv4_append(
        cache, k, v, start, kv, q=q if Hq else None,
        cos_sin=None if tab is None else tab.cuda(),
        positions=None if positions is None else i32(positions),
        interleaved=interleaved, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    index = np.concatenate([np.arange(m - n, m) for n, m in zip(P.n, P.kv)]
                           or [[]]).astype(int)
    pos = index if positions is None else np.array(positions)
    x64 = oref.f64(x)
    if rot:
        turned = rotate32(x64[:, :Hq + Hkv], oref.f64(tab), pos, interleaved)
        y, size = oref.rotate(x64[:, :Hq + Hkv], oref.f64(tab), pos,
                              interleaved)
        tol = oref.append_tol(y, size, dt)
    else:
        turned = y = x64[:, :Hq + Hkv]
        tol = np.zeros_like(y)
    if Hq:
        assert (np.abs(oref.f64(out) - y[:, :Hq]) <= tol[:, :Hq]).all()
    kn, kp = ref.quantise(turned[:, Hq:], P.group)
    vn, vp = ref.quantise(x64[:, Hq + Hkv:], P.group)
    want = [t.cpu() for t in was]
    seq = np.repeat(np.arange(len(P.n)), P.n)
    for r, (b, j) in enumerate(zip(seq, index)):
        p, t = P.slot(b, j)
        for w, c in ((want[0], kn), (want[1], vn)):
            w[p, :, t] = torch.tensor(ref.pack(c[r]))
        for w, c in ((want[2], kp), (want[3], vp)):
            w[p, :, t] = torch.tensor(c[r]).half()
    for w, got in zip(want, (cache.k, cache.v, cache.k_scale,
                             cache.v_scale)):
        np.testing.assert_array_equal(got.cpu().numpy(), w.numpy())
    return cache, out


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64),
                                     (128, 128)])
@pytest.mark.parametrize("rot,interleaved", [(1, False), (1, True),
                                             (2, False), (0, False)])
def test_append_types_groups_pairings(dtype, D, group, rot, interleaved):
    P = ref.Paged4([1, 0, 9, 3], [1, 4, 40, 100], 2, D, 16, dtype, 5, group)
    run_append(P, 6, rot and D // rot, interleaved=interleaved)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot", [2, 6, 20, 34, 48])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_any_rotation(D, rot, interleaved):
    P = ref.Paged4([5, 2], [9, 30], 3, D, 8, BF, 6, 32)
    run_append(P, 3, rot, interleaved=interleaved)


@pytest.mark.parametrize("Hkv,Hq", [(1, 0), (1, 1), (3, 5), (8, 64), (40, 0),
                                    (5, 71)])
def test_append_head_layouts(Hkv, Hq):
    P = ref.Paged4([3, 1], [20, 1], Hkv, 64, 8, HF, 7, 64)
    run_append(P, Hq, 64, fused=bool(Hq % 2))


@pytest.mark.parametrize("page", [8, 24, 64, 320])
def test_append_pages_apart(page):
    P = ref.Paged4([30, 1], [90, 200], 2, 64, page, BF, 8, 32, apart=48)
    cache, _ = run_append(P, 2, 32)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        between = t._base[:, t[0].numel():]
        assert between.numel() * between.element_size() == 48 * t.shape[0]
        assert bool((between == 255).all() if t.dtype == torch.uint8
                    else torch.isnan(between).all())


def test_append_positions_and_odd_rows():
    """A tree's positions; rows that are not 16-byte aligned."""
    P = ref.Paged4([4, 2], [30, 9], 2, 64, 8, BF, 9, 32)
    run_append(P, 4, 64, positions=[26, 27, 27, 28, 7, 0])
    cache = P.cache(api)
    start, kv = P.lengths()
    wide = torch.randn((6, 4 * 64 + 3), device="cuda").to(BF)
    odd = wide[:, 1:257].unflatten(1, (4, 64))
    api.kv4_append(cache, odd[:, :2], odd[:, 2:], start, kv)
    a = ref.held(cache)
    cache = P.cache(api)
    even = odd.contiguous()
    api.kv4_append(cache, even[:, :2], even[:, 2:], start, kv)
    for x, y in zip(a, ref.held(cache)):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,group,rot", [(128, 64, 128), (64, 32, 32)])
def test_append_many_rows_bit_for_bit(dtype, interleaved, D, group, rot):
    """Millions of elements: no product of the rotation is fused with its sum
    (a code in 10^5 would change), on one to eight warps a row."""
    H, page = 8, 64
    for total in (40, 700, 3001, 9000):
        cols = -(-total // page)
        g = torch.Generator(device="cuda").manual_seed(total)
        table = torch.randperm(cols, generator=g,
                               device="cuda").int().view(1, cols)
        cache = api.PagedKV4.empty(cols, page, H, D, table, dtype, group)
        x = torch.randn((total, 2 * H, D), generator=g,
                        device="cuda").to(dtype)
        tab = oref.cos_sin_table(total, rot).cuda()
        start, kv = lengths([total], [total])
        api.kv4_append(cache, x[:, :H], x[:, H:], start, kv, cos_sin=tab,
                       interleaved=interleaved)
        y = x.float()
        c, s = (t[:, None] for t in tab.split(rot // 2, 1))
        at = torch.arange(rot // 2, device="cuda")
        i, j = (2 * at, 2 * at + 1) if interleaved else (at, at + rot // 2)
        a, b = y[:, :H, i], y[:, :H, j]
        y[:, :H, i], y[:, :H, j] = a * c - b * s, a * s + b * c
        y = y.unflatten(-1, (-1, group))
        lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
        step = ((hi - lo) * float(np.float32(1 / 15))).half()
        base = (lo - step.float() * 64).half()
        n = ((y - base.float()) * step.float().reciprocal()).round() - 64
        n = n.clamp(0, 15).to(torch.uint8).flatten(-2)
        w = n.unflatten(-1, (-1, 8))[..., torch.tensor(ref.ORDER).cuda()]
        codes = (w[..., 0::2] | w[..., 1::2] << 4).flatten(-2)
        pos = torch.arange(total, device="cuda")
        p, t = table[0, pos // page].long(), pos % page
        pair = torch.cat([step, base], -1)
        for got, want in ((cache.k, codes[:, :H]), (cache.v, codes[:, H:]),
                          (cache.k_scale, pair[:, :H]),
                          (cache.v_scale, pair[:, H:])):
            assert torch.equal(got[p, :, t], want)


def test_append_numbers_at_the_ends():
    """One number a group, NaN, infinities, numbers beyond 6144 and below
    fp16's least, groups far from zero."""
    P = ref.Paged4([8], [8], 1, 64, 8, BF, 10, 32)
    x = P.rows(2)
    x[0] = 7.25
    x[1, 0, 3] = float("nan")
    x[2, 1, 40] = float("inf")
    x[3, 0, 5] = -float("inf")
    x[4, :, :2] = 1e30
    x[4, :, 2] = -7000.0
    x[5] = x[5] * 1e-8
    x[6] = x[6] * 0.01 + 500
    x[7] = 0
    cache, _ = run_append(P, 0, 0, x=x)
    k, v = ref.held(cache)
    p, t = P.slot(0, 1)
    assert np.isnan(k[p, t, 0, :32]).all()
    assert np.isfinite(k[p, t, 0, 32:]).all()


def test_append_refuses_rows():
    """Unusable lengths, bad pages and positions: nothing written, q zero;
    rows of no sequence left as they are."""
    P = ref.Paged4([2, 2, 2, 2], [40, 50, 60, 30], 1, 64, 16, BF, 11, 32)
    x = P.rows(4).cuda()
    start, kv = P.lengths()
    tab = oref.cos_sin_table(64, 64).cuda()

    def call(P_table, kv, pos=None, start=start):
        cache = P.cache(api, table=P_table)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = api.kv4_append(cache, x[:, 2:3], x[:, 3:], start, kv, q=x[:, :2],
                           cos_sin=tab, status=st,
                           positions=None if pos is None else i32(pos))
        return ref.held(cache), q, int(st.item())

    good, gq, st = call(P.table, kv)
    before = ref.held(P.cache(api))
    assert st == 0

    def same(held, q, bad_rows, want_bits, st):
        assert st == want_bits
        seq = np.repeat(np.arange(4), 2)
        for r in range(8):
            b = seq[r]
            j = P.kv[b] - 2 + r % 2
            p, t = P.slot(b, j)
            for h, g_, w in zip(held, good, before):
                np.testing.assert_array_equal(
                    h[p, t], w[p, t] if r in bad_rows else g_[p, t])
            assert torch.equal(q[r], torch.zeros_like(q[r])
                               if r in bad_rows else gq[r])

    bad = kv.clone()
    bad[1] = 1
    same(*call(P.table, bad)[:2], [2, 3], api.DEV_BAD_LENGTH,
         call(P.table, bad)[2])
    bad[1] = 10 ** 6
    same(*call(P.table, bad)[:2], [2, 3], api.DEV_BAD_LENGTH,
         call(P.table, bad)[2])
    table = P.table.clone()
    table[2, 59 // 16] = 10 ** 6
    h, q, st = call(table, kv)
    same(h, q, [4, 5], api.DEV_BAD_PAGE, st)
    h, q, st = call(P.table, kv, [38, 39, 48, 49, 58, 59, 64, -1])
    same(h, q, [6, 7], api.DEV_BAD_POSITION, st)
    short = start.clone()
    short[4] = 7  # the last row belongs to no sequence
    cache = P.cache(api)
    q = torch.full_like(gq, 3.0)
    rows = x.contiguous()
    rc = api.lib().sd_kv4_append(
        cache._addr, rows[:, 2].data_ptr(), 4 * 64, rows[:, 3].data_ptr(),
        4 * 64, rows.data_ptr(), 4 * 64, 2, short.data_ptr(), kv.data_ptr(),
        None, None, 0, 0, 0, 4, 8, q.data_ptr(), None,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and bool((q[7] == 3).all()) and bool((q[6] != 3).any())


# -------------------------------------------------------------------- read
def run_read(P, n, kv):
    cache = P.cache(api)
    start, lens = lengths(n, kv)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    total = int(sum(n))
    r = api.kv4_read(cache, start, lens, total, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    lo = 0
    for b, (a, m) in enumerate(zip(n, kv)):
        for name, held in (("k", P.k), ("v", P.v)):
            want = P.gather(held, b)[m - a:m]
            want = torch.tensor(want).float().to(P.dtype)
            assert torch.equal(r[name][lo:lo + a].cpu(), want)
        lo += a


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64),
                                     (128, 128)])
@pytest.mark.parametrize("heads", [1, 5])
def test_read_types_and_ranges(dtype, D, group, heads):
    kv = [130, 1, 40, 9]
    P = ref.Paged4([0] * 4, kv, heads, D, 24, dtype, 21, group, by=3.0)
    run_read(P, kv, kv)
    run_read(P, [7, 0, 1, 9], [100, 1, 33, 9])  # parts of the sequences


def test_read_pages_apart_and_bad_rows():
    P = ref.Paged4([0] * 3, [70, 20, 33], 2, 64, 16, BF, 22, 64, apart=32)
    run_read(P, [70, 20, 33], [70, 20, 33])
    table = P.table.clone()
    table[0, 2] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    start, kv = lengths([70, 20, 4], [70, 10, 33])
    r = api.kv4_read(P.cache(api, table=table), start, kv, 94, status=st)
    assert int(st.item()) == api.DEV_BAD_PAGE | api.DEV_BAD_LENGTH
    nan = torch.isnan(r["k"]).flatten(1).all(1).cpu().numpy()
    want = np.zeros(94, bool)
    want[32:48] = True   # the missing page
    want[70:90] = True   # 20 rows of 10 keys
    np.testing.assert_array_equal(nan, want)
    assert bool(torch.isfinite(r["v"][want == 0]).all())


def test_read_leaves_rows_of_no_sequence():
    P = ref.Paged4([0] * 2, [5, 8], 1, 64, 8, HF, 23, 32)
    k = torch.full((20, 64), 3.0, dtype=HF, device="cuda")
    v = torch.full((20, 64), 3.0, dtype=HF, device="cuda")
    start, kv = i32([2, 7, 15]), i32([5, 8])
    cache = P.cache(api)
    rc = api.lib().sd_kv4_read(
        cache._addr, start.data_ptr(), kv.data_ptr(), 2, 20, k.data_ptr(),
        64, v.data_ptr(), 64, None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    for t in (k, v):
        assert bool((t[:2] == 3).all()) and bool((t[15:] == 3).all())
    assert torch.equal(k[2:7].cpu().double(),
                       torch.tensor(P.gather(P.k, 0)[:, 0]))


# --------------------------------------------------------------- attention
def random_trees(n, seed):
    r = np.random.default_rng(seed)
    see = []
    for m in n:
        t = np.zeros((m, m), bool)
        for i in range(m):
            if i:
                t[i] = t[r.integers(max(0, i - 6), i)]
            t[i, i] = True
        see.append(t)
    return see


def run(P, Hq, *, see=None, max_q=None, scale=None, by=2.0, q=None):
    cache = P.cache(api)
    q = P.rows(Hq, by=by) if q is None else q
    start, kv = P.lengths()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.kv4_attention(
        q.cuda(), cache, start, kv, max_q=max_q, scale=scale,
        tree_mask=None if see is None else oref.pack_mask(see),
        want_lse=True, status=st, workspace=api.Workspace())
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    out, lse, tol, ltol = ref.attention(P, q, scale or P.dim ** -0.5, see)
    g, gl = oref.f64(got["out"]), oref.f64(got["lse"])
    assert np.isfinite(g).all()
    assert (np.abs(g - out) <= tol).all(), (np.abs(g - out) / tol).max()
    fine = np.isfinite(lse)
    assert (gl[~fine] == lse[~fine]).all()
    assert (np.abs(gl - lse)[fine] <= ltol[fine]).all()
    return got


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64),
                                     (128, 128)])
@pytest.mark.parametrize("n,kv", [
    ([1], [1]), ([1], [2]), ([5], [100]), ([1, 1, 1], [129, 128, 127]),
    ([0, 3, 0], [5, 3, 0]), ([9, 9], [300, 9]), ([17, 1, 40], [140, 513, 40]),
    ([130], [257]), ([1], [1000])])
def test_attention_lengths(dtype, D, group, n, kv):
    run(ref.Paged4(n, kv, 2, D, 16, dtype, sum(kv) + D, group), 4,
        max_q=max(n))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 5), (10, 2), (8, 1),
                                    (16, 1), (17, 1), (71, 1), (130, 1),
                                    (14, 2), (300, 1)])
@pytest.mark.parametrize("n", [1, 4])
def test_attention_head_layouts(Hq, Hkv, n):
    run(ref.Paged4([n, n], [n, 200], Hkv, 64, 8, BF, Hq, 32), Hq, max_q=n)


@pytest.mark.parametrize("page", [8, 24, 48, 64, 128, 256, 320])
@pytest.mark.parametrize("Hq", [8, 40])
def test_attention_pages(page, Hq):
    """Pages that end inside a key tile, tiles that end inside a page, pages
    apart."""
    run(ref.Paged4([3, 1], [401, 130], 2, 128, page, HF, page, 64,
                   apart=page * 2), Hq, max_q=3)


@pytest.mark.parametrize("hint", [None, 0, 1, 3, 5, 64, 4096])
def test_attention_the_hint_changes_no_result(hint):
    run(ref.Paged4([40, 1, 3], [170, 300, 3], 2, 64, 16, BF, 3, 32), 6,
        max_q=hint)


@pytest.mark.parametrize("n,kv,Hq", [([64, 64], [300, 64], 8),
                                     ([31, 33, 1], [200, 40, 9], 2),
                                     ([130], [300], 2), ([1, 2], [1, 2], 4),
                                     ([5, 4], [90, 33], 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_token_trees(n, kv, Hq, D):
    run(ref.Paged4(n, kv, 2, D, 32, HF, sum(kv), 64), Hq, max_q=max(n),
        see=random_trees(n, 5))


@pytest.mark.parametrize("hint", [2, 40, 4096])
def test_attention_masks_that_leave_rows_empty(hint):
    see = random_trees([5, 40, 3], 7)
    see[0][2] = False
    see[1][:, :] = False
    see[1][3, 0] = see[1][39, 38] = True
    P = ref.Paged4([5, 40, 3], [5, 40, 20], 2, 64, 16, BF, 11, 32)
    got = run(P, 4, max_q=hint, see=see)
    assert bool((got["out"][2] == 0).all())
    assert bool((got["lse"][2] == -float("inf")).all())
    assert bool((got["out"][5:8] == 0).all())
    # bits past the chunk count for nothing
    ahead = [np.ones((3, 3), bool)]
    P = ref.Paged4([3], [130], 1, 64, 8, BF, 12, 32)
    run(P, 2, max_q=hint, see=ahead)
    q = P.rows(2).cuda()
    start, kv = P.lengths()
    full = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    a, b = (api.kv4_attention(q, P.cache(api), start, kv, tree_mask=m,
                              max_q=hint)["out"]
            for m in (full, oref.pack_mask(ahead)))
    assert torch.equal(a, b)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 2)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_parts_of_prompts(D, Hq, Hkv, dtype):
    run(ref.Paged4([300, 257, 1], [300, 700, 650], Hkv, D, 64, dtype, 21, 64),
        Hq, max_q=300)


def test_attention_long_prefixes_are_split_and_joined():
    run(ref.Paged4([1, 2], [6000, 150], 1, 64, 32, BF, 31, 32), 4, max_q=2)
    run(ref.Paged4([9], [5000], 2, 128, 16, HF, 32, 128), 8, max_q=9)
    run(ref.Paged4([1] * 40, list(range(1, 2000, 50)), 1, 64, 16, BF, 33, 64),
        8, max_q=1)


@pytest.mark.parametrize("by", [0.0, 20.0])
def test_attention_flat_and_steep_scores(by):
    run(ref.Paged4([2, 3], [700, 40], 2, 64, 16, BF, 41, 32), 4, by=by)
    run(ref.Paged4([40], [200], 1, 128, 16, HF, 42, 64), 4, by=by)


@pytest.mark.parametrize("n,Hq", [(1, 2), (1, 16), (20, 2), (200, 2)])
def test_attention_rising_and_falling_scores(n, Hq):
    """Key after key scores lie above (below) the ones before, by hundreds
    over the sequence."""
    for sign in (1, -1):
        P = ref.Paged4([n], [900], 1, 64, 16, BF, 43, 32)
        d = torch.randn(64, generator=P.gen).numpy()
        d /= np.linalg.norm(d)
        for j in range(900):
            p, t = P.slot(0, j)
            P.kn[p, t], P.kp[p, t] = ref.quantise(
                ref.to32(d[None] * (sign * j / 20)), 32)
        P.k = torch.tensor(ref.values(P.kn, P.kp))
        q = torch.tensor(d * 8).to(BF).view(1, 1, 64).repeat(n, Hq, 1)
        run(P, Hq, scale=1.0, q=q, max_q=n)


@pytest.mark.parametrize("n,Hq", [(1, 2), (1, 16), (20, 2), (200, 2)])
def test_attention_a_heavy_key_beside_many_light_ones(n, Hq):
    """A key 2^14 above the others, its value 0: the others' sum is the
    result."""
    P = ref.Paged4([n], [3000], 1, 64, 16, BF, 44, 32)
    P.kn[:], P.kp[:] = ref.quantise(np.zeros_like(P.kn, np.float64), 32)
    p, t = P.slot(0, 5)
    heavy = np.zeros((1, 64))
    heavy[0, 0] = 14 * np.log(2)
    P.kn[p, t], P.kp[p, t] = ref.quantise(ref.to32(heavy), 32)
    P.vn[p, t], P.vp[p, t] = ref.quantise(np.zeros((1, 64)), 32)
    P.k, P.v = (torch.tensor(ref.values(*x))
                for x in ((P.kn, P.kp), (P.vn, P.vp)))
    q = torch.zeros((n, Hq, 64), dtype=BF)
    q[..., 0] = 1
    # keys that nobody owns keep their NaN
    run(P, Hq, scale=1.0, q=q, max_q=n)


@pytest.mark.parametrize("by", [1e-30, 1e-6, 1e6, 1e30])
def test_attention_queries_of_any_size(by):
    """bf16 queries far outside fp16's range."""
    P = ref.Paged4([1, 3], [200, 30], 1, 64, 16, BF, 45, 32)
    q = P.rows(4, by=by)
    q[:, :, 3] = 0
    run(P, 4, scale=0.3 / by, q=q)
    P = ref.Paged4([40], [60], 1, 128, 16, BF, 46, 32)
    run(P, 4, scale=0.3 / by, q=P.rows(4, by=by))


def test_attention_queries_that_are_not_finite():
    """NaN for the row alone."""
    for n, Hq in ((1, 4), (5, 8), (64, 4)):
        for dt in (BF, HF):
            P = ref.Paged4([n], [150], 1, 64, 16, dt, 47, 32)
            q = P.rows(Hq)
            want = ref.attention(P, q, 0.125)[0]
            q[0, 1, 7] = float("inf")
            q[0, 2, 9] = float("nan")
            start, kv = P.lengths()
            got = oref.f64(api.kv4_attention(q.cuda(), P.cache(api), start,
                                             kv, max_q=n)["out"])
            nan = np.isnan(got).any(-1)
            rows = np.zeros_like(nan)
            rows[0, 1:3] = True
            np.testing.assert_array_equal(nan, rows)
            assert np.abs(got - want)[~rows].max() < 0.05


def test_attention_scale_and_strided_queries():
    P = ref.Paged4([4, 2], [90, 33], 2, 64, 16, BF, 51, 32)
    run(P, 4, scale=0.3)
    start, kv = P.lengths()
    wide = P.rows(9).cuda()
    a, b = (api.kv4_attention(w, P.cache(api), start, kv)["out"]
            for w in (wide[:, 2:6], wide[:, 2:6].contiguous()))
    assert torch.equal(a, b)


@pytest.mark.parametrize("hint", [2, 40, 4096])
def test_attention_unusable_sequences(hint):
    """A key count below the chunk, one above the table, a bad page among
    those read, a mask too short: NaN for that sequence, bits set, the other
    sequences as without them."""
    n, kv = [2, 2, 2, 2, 40], [40, 50, 60, 30, 40]
    P = ref.Paged4(n, kv, 1, 64, 16, BF, 61, 32)
    q = P.rows(4).cuda()
    start, kvt = P.lengths()
    rows = np.repeat(np.arange(5), n)

    def call(table, kvt, mask=None):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = api.kv4_attention(q, P.cache(api, table=table), start, kvt,
                              tree_mask=mask, want_lse=True, status=st,
                              max_q=hint)
        return oref.f64(r["out"]), oref.f64(r["lse"]), int(st.item())

    good, glse, st = call(P.table, kvt)
    assert st == 0 and np.isfinite(good).all()
    want, _, tol, _ = ref.attention(P, q, 0.125)

    def check(got, seq, bits):
        out, lse, st = got
        assert st == bits
        bad = rows == seq
        assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
        assert (np.abs(out - want)[~bad] <= tol[~bad]).all()

    for b, m in ((1, 1), (3, 10 ** 6)):
        k2 = kvt.clone()
        k2[b] = m
        check(call(P.table, k2), b, api.DEV_BAD_LENGTH)
    for page in (-1, 10 ** 6):
        table = P.table.clone()
        table[2, 1] = page
        check(call(table, kvt), 2, api.DEV_BAD_PAGE)
    see = [np.tril(np.ones((m, m), bool)) for m in n]
    short = oref.pack_mask(see)[:, :1].contiguous()
    check(call(P.table, kvt, short), 4, api.DEV_BAD_LENGTH)


@pytest.mark.parametrize("n,Hq", [([1, 2], 4), ([40, 3], 4), ([200, 3], 4)])
def test_attention_leaves_rows_of_no_sequence(n, Hq):
    P = ref.Paged4(n, [250, 30], 1, 64, 16, BF, 62, 32)
    total = P.total + 5
    q = torch.randn((total, Hq, 64), device="cuda").to(BF)
    start = torch.tensor(P.start + 2, dtype=torch.int32, device="cuda")
    kv = i32(P.kv)
    out = torch.full((total, Hq, 64), 3.0, dtype=BF, device="cuda")
    lse = torch.full((total, Hq), 3.0, device="cuda")
    need = api.lib().sd_kv4_attention_workspace(Hq, 1, 64, max(n))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    cache = P.cache(api)
    rc = api.lib().sd_kv4_attention(
        q.data_ptr(), Hq * 64, Hq, cache._addr, start.data_ptr(),
        kv.data_ptr(), None, 0, 2, total, max(n), 0.125, out.data_ptr(),
        lse.data_ptr(), None, ws.data_ptr(), need,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    for t in (out, lse):
        assert bool((t[:2] == 3).all()) and bool((t[-3:] == 3).all())
        assert bool((t[2:-3] != 3).flatten(1).any(1).all())


def test_attention_keys_that_are_not_finite_reach_who_sees_them():
    """A NaN group in the last of the chunk's keys: the token itself has NaN,
    a sequence beside it does not."""
    for n, Hq in ((3, 2), (40, 2), (200, 2)):
        P = ref.Paged4([n, 1], [n + 50, 60], 1, 64, 16, BF, 63, 32)
        p, t = P.slot(0, n + 49)
        P.kp[p, t, 0, 1] = np.nan
        start, kv = P.lengths()
        out = api.kv4_attention(P.rows(Hq).cuda(), P.cache(api), start, kv,
                                max_q=n)["out"]
        assert bool(torch.isnan(out[n - 1]).all())
        assert bool(torch.isfinite(out[n]).all())


def test_attention_bits_do_not_change():
    """Calls in a row, on another stream, and a replayed graph: same bits."""
    for n, Hq, D in ((1, 8, 128), (9, 32, 128), (9, 16, 64), (150, 4, 128)):
        P = ref.Paged4([n, n, 1], [900, n + 3, 2000], 2, D, 16, BF, 71, 64)
        cache, q = P.cache(api), P.rows(Hq).cuda()
        start, kv = P.lengths()
        ws = api.Workspace()

        def call():
            return api.kv4_attention(q, cache, start, kv, max_q=n,
                                     workspace=ws)["out"]
        first = call()
        for _ in range(20):
            assert torch.equal(call(), first)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert torch.equal(call(), first)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = call()
        q2 = q.clone()
        q.copy_(-q2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()) and not torch.equal(out, first)
        q.copy_(q2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,group", [(BF, 64), (HF, 32)])
def test_drafting_from_a_4_bit_copy(dtype, group):
    """A prompt is appended to a 16-bit and a 4-bit cache, tokens are added
    one at a time, then a round of drafts at once: attention over the 4-bit
    cache is attention over what it reads back as, and near attention over
    the 16-bit one."""
    B, Hq, Hkv, D, page = 3, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randperm(B * 8, generator=g,
                           device="cuda").int().view(B, 8)
    shape = (B * 8, page, Hkv, D)
    wide = api.PagedKV(torch.zeros(shape, dtype=dtype, device="cuda"),
                       torch.zeros(shape, dtype=dtype, device="cuda"), table)
    four = api.PagedKV4.empty(B * 8, page, Hkv, D, table, dtype, group)
    tab = oref.cos_sin_table(128, D).cuda()
    have = np.zeros(B, int)
    for n in ([60, 33, 90], [1, 1, 1], [1, 0, 1], [5, 5, 5]):
        have += n
        start, kv = lengths(n, have)
        total = int(sum(n))
        x = torch.randn((total, Hq + 2 * Hkv, D), generator=g,
                        device="cuda").to(dtype)
        k, v = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        q = api.kv4_append(four, k, v, start, kv, q=x[:, :Hq], cos_sin=tab)
        q16 = api.kv_append(wide, k, v, start, kv, q=x[:, :Hq], cos_sin=tab)
        assert bool(((q.float() - q16.float()).abs() <= 2 * oref.U[dtype] *
                     q16.float().abs() + 1e-5).all())
        got = api.kv4_attention(q, four, start, kv, max_q=max(n))["out"]
        near = api.paged_attention(q, wide, start, kv, max_q=max(n))["out"]
        # 16-bit rows of all keys, in order, as a cache of their own
        s_all, kv_all = lengths(have, have)
        r = api.kv4_read(four, s_all, kv_all, int(sum(have)))
        lo = at = 0
        for b in range(B):
            kk, vv = (oref.f64(r[c][at:at + have[b]]) for c in "kv")
            at += have[b]
            for i in range(n[b]):
                m = have[b] - n[b] + i + 1
                for h in range(Hq):
                    s = kk[:m, h // 4] @ oref.f64(q[lo + i, h]) * D ** -0.5
                    w = np.exp(s - s.max())
                    want = w @ vv[:m, h // 4] / w.sum()
                    # the read rows are rounded to the type once more: scores
                    # by u |q||k| (added up at random: sqrt(D) of D), values
                    # and the result by u
                    u = oref.U[dtype]
                    ds = u * D ** -0.5 * (np.abs(kk[:m, h // 4]) @
                                          np.abs(oref.f64(q[lo + i, h]))).max()
                    err = np.abs(oref.f64(got[lo + i, h]) - want)
                    assert (err <= (2 * ds + 2 * u + 2.0 ** -10) *
                            np.abs(vv[:m, h // 4]).max() + 1e-4).all()
            lo += n[b]
        # 4 bits: a step is a fifteenth of a group's range, about 5; scores
        # move by a tenth or two, values by 0.1
        assert float((got.float() - near.float()).abs().mean()) < 0.2


def test_offsets_past_32_bits():
    """Pages more than 4 GB into the cache: the same bits as at its start."""
    H, D, page, n = 8, 128, 64, 140000
    shape = (n, H, page, D // 2)
    k, v = (torch.empty(shape, dtype=torch.uint8, device="cuda")
            for _ in range(2))
    ks, vs = (torch.empty((n, H, page, 2, 2), dtype=torch.float16,
                          device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(9)
    total = 300
    x = torch.randn((total, 2 * H + 32, D), generator=g, device="cuda").to(BF)
    start, kv = lengths([total], [total])
    out = []
    for first in (0, n - 8):
        table = (first + torch.arange(8, device="cuda")).int().view(1, 8)
        cache = api.PagedKV4(k, v, ks, vs, table, BF)
        api.kv4_append(cache, x[:, :H], x[:, H:2 * H], start, kv)
        r = [*api.kv4_read(cache, start, kv, total).values()]
        for m in (1, 3, 9, 300):  # each kernel
            s0, kv0 = lengths([m], [total])
            q = x[:m, 2 * H:].contiguous()
            r.append(api.kv4_attention(q, cache, s0, kv0, max_q=m)["out"])
        out.append(r)
    for a, b in zip(*out):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())


def test_calls_on_two_streams_at_once():
    """Calls that overlap on the GPU share nothing."""
    P = ref.Paged4([9, 9, 1], [900, 400, 2000], 2, 128, 16, BF, 81, 64)
    cache = P.cache(api)
    start, kv = P.lengths()
    qs = [P.rows(h).cuda() for h in (4, 16, 128)]
    want = [api.kv4_attention(q, cache, start, kv, max_q=9)["out"]
            for q in qs]
    side = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for q, s in zip(qs, side):
            with torch.cuda.stream(s):
                got.append(api.kv4_attention(q, cache, start, kv,
                                             max_q=9)["out"])
    torch.cuda.synchronize()
    for i, a in enumerate(got):
        assert torch.equal(a, want[i % 3])


@pytest.mark.parametrize("n,kv,Hq", [([3, 1], [3000, 70], 4),
                                     ([3, 1], [3000, 70], 8),
                                     ([9, 1], [3000, 70], 6),
                                     ([200], [300], 6)])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32)])
def test_no_write_outside_the_buffers(monkeypatch, n, kv, Hq, D, group):
    """Outputs and workspaces lie between guards."""
    P = ref.Paged4(n, kv, 2, D, 16, BF, 91, group)
    cache, q = P.cache(api), P.rows(Hq).cuda()
    start, lens = P.lengths()
    x = P.rows(4).cuda()
    guard = GuardedTorch()
    monkeypatch.setattr(api, "torch", guard)
    api.kv4_attention(q, cache, start, lens, max_q=max(n), want_lse=True,
                      workspace=api.Workspace())
    assert guard.check() == 3
    api.kv4_append(cache, x[:, :2], x[:, 2:], start, lens, q=q)
    api.kv4_read(cache, start, lens, P.total)
    assert guard.check() == 3
