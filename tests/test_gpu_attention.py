"""sd_paged_attention against the 64-bit formula, under bounds derived from
the types' roundings (tests/operators_ref.py).  The caches hold NaN wherever
no key of a sequence lies."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import operators_ref as ref
from tests.test_gpu_canaries import GuardedTorch

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


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


def run(P, Hq, *, see=None, max_q=None, scale=None, by=2.0, ws=None):
    cache = api.PagedKV(P.to_gpu(P.k), P.to_gpu(P.v), P.table.cuda())
    q = P.rows(Hq, by=by)
    start, kv = P.lengths()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.paged_attention(
        q.cuda(), cache, start, kv, max_q=max_q, scale=scale,
        tree_mask=None if see is None else ref.pack_mask(see), want_lse=True,
        status=st, workspace=ws or api.Workspace())
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    out, lse, tol, ltol = ref.attention(P, q, scale or P.dim ** -0.5, see)
    g, gl = ref.f64(got["out"]), ref.f64(got["lse"])
    assert np.isfinite(g).all()
    assert (np.abs(g - out) <= tol).all(), np.abs(g - out).max()
    fine = np.isfinite(lse)
    assert (gl[~fine] == lse[~fine]).all()
    assert (np.abs(gl - lse)[fine] <= ltol[fine]).all()
    return got


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,kv", [
    ([1], [1]), ([1], [2]), ([5], [100]), ([1, 1, 1], [129, 128, 127]),
    ([0, 3, 0], [5, 3, 0]), ([9, 9], [300, 9]), ([17, 1, 40], [140, 513, 40]),
    ([130], [257]), ([1], [1000])])
def test_lengths(dtype, D, n, kv):
    run(ref.Paged(n, kv, 2, D, 16, dtype, seed=sum(kv) + D), 4,
        max_q=max(n))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,kv,Hq", [([1], [700], 4), ([9, 3], [260, 1000], 8),
                                     ([64], [64], 4), ([5], [100], 2)])
def test_few_rows_are_off_by_the_outputs_rounding(dtype, D, n, kv, Hq):
    """With up to 128 rows a head the weights keep twice the type's bits."""
    P = ref.Paged(n, kv, 2, D, 16, dtype, seed=sum(kv) + Hq)
    q = P.rows(Hq, by=2.0)
    start, lens = P.lengths()
    got = api.paged_attention(
        q.cuda(), api.PagedKV(P.to_gpu(P.k), P.to_gpu(P.v), P.table.cuda()),
        start, lens, max_q=max(n), workspace=api.Workspace())
    out, _, tol, _ = ref.attention(P, q, D ** -0.5, split=True)
    assert (np.abs(ref.f64(got["out"] if isinstance(got, dict) else got)
                   - out) <= tol).all()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 5), (10, 2), (16, 1),
                                    (71, 1), (130, 1), (14, 2)])
@pytest.mark.parametrize("n", [1, 4])
def test_head_layouts(Hq, Hkv, n):
    run(ref.Paged([n, n], [n, 200], Hkv, 64, 8, BF, seed=Hq), Hq, max_q=n)


@pytest.mark.parametrize("page", [8, 24, 48, 64, 128, 256, 320])
@pytest.mark.parametrize("head_major", [False, True])
def test_pages(page, head_major):
    """Pages that end inside a key tile, tiles that end inside a page."""
    P = ref.Paged([3, 1], [401, 130], 2, 128, page, HF, seed=page,
                  head_major=head_major)
    run(P, 8, max_q=3)


@pytest.mark.parametrize("hint", [None, 0, 1, 5, 64, 4096])
def test_the_hint_changes_no_result(hint):
    """Any max_q: the chunk lengths are what q_start says."""
    run(ref.Paged([40, 1, 3], [170, 300, 3], 2, 64, 16, BF, seed=3), 6,
        max_q=hint)


@pytest.mark.parametrize("n,kv,Hq", [([64, 64], [300, 64], 8),
                                     ([31, 33, 1], [200, 40, 9], 2),
                                     ([130], [300], 2), ([1, 2], [1, 2], 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_token_trees(n, kv, Hq, D):
    run(ref.Paged(n, kv, 2, D, 32, HF, seed=sum(kv)), Hq, max_q=max(n),
        see=random_trees(n, 5))


def test_masks_that_leave_rows_empty():
    """No prefix and no bit: out 0, lse -inf; rows beside them as ever.  Bits
    past the chunk count for nothing."""
    see = random_trees([5, 40, 3], 7)
    see[0][2] = False
    see[1][:, :] = False
    see[1][3, 0] = see[1][39, 38] = True
    P = ref.Paged([5, 40, 3], [5, 40, 20], 2, 64, 16, BF, seed=11)
    got = run(P, 4, max_q=40, see=see)
    assert bool((got["out"][2] == 0).all())
    assert bool((got["lse"][2] == -float("inf")).all())
    assert bool((got["out"][5:8] == 0).all())
    # a mask that looks ahead, and one past the chunk
    ahead = [np.ones((3, 3), bool)]
    P = ref.Paged([3], [130], 1, 64, 8, BF, seed=12)
    want = run(P, 2, max_q=3, see=ahead)["out"]
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    P.gen.manual_seed(1)
    q = P.rows(2).cuda()
    start, kv = P.lengths()
    full = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    a = api.paged_attention(q, cache, start, kv, tree_mask=full)["out"]
    b = api.paged_attention(q, cache, start, kv,
                            tree_mask=ref.pack_mask(ahead))["out"]
    assert torch.equal(a, b) and want.shape == a.shape


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 2)])
def test_parts_of_prompts(D, Hq, Hkv):
    """Chunks of several hundred tokens: many row tiles, causal limits inside
    key tiles, work shared between several CTAs."""
    run(ref.Paged([300, 257, 1], [300, 700, 650], Hkv, D, 64, BF, seed=21),
        Hq, max_q=300)


def test_long_prefixes_are_split_and_joined():
    run(ref.Paged([1, 2], [6000, 150], 1, 64, 32, BF, seed=31), 4, max_q=2)
    run(ref.Paged([9], [5000], 2, 128, 16, HF, seed=32), 8, max_q=9)


@pytest.mark.parametrize("by", [0.0, 20.0])
def test_flat_and_steep_scores(by):
    """Equal weights, and maxima that move by hundreds along the keys."""
    run(ref.Paged([2, 3], [700, 40], 2, 64, 16, BF, seed=41), 4, by=by)
    run(ref.Paged([40], [200], 1, 128, 16, HF, seed=42), 4, by=by)


def test_rising_maximum():
    """Every key tile's scores lie above the last one's."""
    P = ref.Paged([1], [640], 1, 64, 16, BF, seed=43)
    d = torch.randn(64, generator=P.gen)
    for j in range(640):
        p, t = P.slot(0, j)
        P.k[p, t, 0] = (d * (j / 64.0) / d.norm()).to(BF)
    q = (d * 8).to(BF).view(1, 1, 64).repeat(1, 2, 1)
    P.rows = lambda *a, **k: q
    run(P, 2, scale=1.0)


def test_scale_and_strided_queries():
    P = ref.Paged([4, 2], [90, 33], 2, 64, 16, BF, seed=51)
    run(P, 4, scale=0.3)
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    start, kv = P.lengths()
    wide = P.rows(9).cuda()
    a = api.paged_attention(wide[:, 2:6], cache, start, kv)["out"]
    b = api.paged_attention(wide[:, 2:6].contiguous(), cache, start,
                            kv)["out"]
    assert torch.equal(a, b)


def test_unusable_sequences():
    """A key count below the chunk, one above the table, a bad page among
    those read, a mask too short: NaN for that sequence, bits set, the other
    sequences the same bits as without them."""
    n, kv = [2, 2, 2, 2, 40], [40, 50, 60, 30, 40]
    P = ref.Paged(n, kv, 1, 64, 16, BF, seed=61)
    q = P.rows(4).cuda()
    start, kvt = P.lengths()

    def call(table, kvt, mask=None):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = api.paged_attention(
            q, api.PagedKV(P.k.cuda(), P.v.cuda(), table.cuda()), start, kvt,
            tree_mask=mask, want_lse=True, status=st, max_q=40)
        return r["out"], r["lse"], int(st.item())

    out, lse, st = call(P.table, kvt)
    assert st == 0 and bool(torch.isfinite(out).all())
    bad_kv = kvt.clone()
    bad_kv[0], bad_kv[1] = 1, 10 ** 6
    table = P.table.clone()
    table[2, 1] = -1
    table[3, 0] = 10 ** 6
    table[4, 3] = 10 ** 6  # past its 40 keys: never read
    o2, l2, st = call(table, bad_kv)
    assert st == api.DEV_BAD_LENGTH | api.DEV_BAD_PAGE
    assert bool(torch.isnan(o2[:8]).all()) and bool(torch.isnan(l2[:8]).all())
    assert torch.equal(o2[8:], out[8:]) and torch.equal(l2[8:], lse[8:])
    mask = torch.full((48, 1), -1, dtype=torch.int32, device="cuda")
    o3, _, st = call(P.table, kvt, mask)
    assert st == api.DEV_BAD_LENGTH
    assert bool(torch.isnan(o3[8:]).all())
    assert bool(torch.isfinite(o3[:8]).all())


def test_a_nan_key_reaches_who_sees_it():
    P = ref.Paged([2, 2], [150, 150], 2, 64, 16, BF, seed=71)
    p, t = P.slot(0, 7)
    P.k[p, t, 1] = np.nan
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    q = P.rows(4).cuda()
    o = api.paged_attention(q, cache, *P.lengths())["out"]
    assert bool(torch.isnan(o[:2, 2:]).all())
    assert bool(torch.isfinite(o[:2, :2]).all())
    assert bool(torch.isfinite(o[2:]).all())


def test_same_bits_twice_and_on_another_stream():
    P = ref.Paged([9, 1, 30], [3000, 700, 900], 2, 128, 16, BF, seed=81)
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    q = P.rows(8).cuda()
    start, kv = P.lengths()
    ws = api.Workspace()
    a = api.paged_attention(q, cache, start, kv, workspace=ws)["out"]
    for _ in range(3):
        b = api.paged_attention(q, cache, start, kv, workspace=ws)["out"]
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = api.paged_attention(q, cache, start, kv,
                                workspace=api.Workspace())["out"]
    s.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("n,kv,hint", [([9, 1], [3000, 70], 9),
                                       ([200], [300], 200)])
def test_no_write_outside_the_buffers(monkeypatch, n, kv, hint):
    guard = GuardedTorch()
    monkeypatch.setattr(api, "torch", guard)
    P = ref.Paged(n, kv, 2, 64, 16, BF, seed=91)
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    api.paged_attention(P.rows(6).cuda(), cache, *P.lengths(), max_q=hint,
                        want_lse=True, workspace=api.Workspace())
    assert guard.check() >= 2


def test_rows_of_no_sequence_are_left_alone(monkeypatch):
    """total above q_start[B]: those rows keep what they held."""
    guard = GuardedTorch()  # its buffers start as the sentinel
    monkeypatch.setattr(api, "torch", guard)
    P = ref.Paged([2, 1], [20, 300], 2, 64, 16, BF, seed=95)
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    q = torch.cat([P.rows(4), torch.ones(3, 4, 64, dtype=BF)]).cuda()
    out = api.paged_attention(q, cache, *P.lengths(),
                              workspace=api.Workspace())["out"]
    torch.cuda.synchronize()
    assert bool((out[3:].view(torch.uint8) == 0xA5).all())
    assert bool(torch.isfinite(out[:3]).all())


def test_cache_offsets_past_32_bits():
    """Pages whose element offsets do not fit 32 bits (a strided view of a
    larger buffer): the last pages of a cache of 2^32 + elements."""
    page, H, D = 16, 1, 64
    pages = 2
    stride = (1 << 32) // 1 + 1024  # elements between the two pages
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    n = stride + page * H * D
    kb = torch.empty(n, dtype=BF, device="cuda")
    vb = torch.empty(n, dtype=BF, device="cuda")
    view = (pages, page, H, D), (stride, H * D, D, 1)
    k, v = kb.as_strided(*view), vb.as_strided(*view)
    g = torch.Generator().manual_seed(1)
    P = ref.Paged([1], [30], H, D, page, BF, seed=1, extra_cols=0)
    P.table = torch.tensor([[1, 0]], dtype=torch.int32)
    P.k = torch.randn(pages, page, H, D, generator=g).to(BF)
    P.v = torch.randn(pages, page, H, D, generator=g).to(BF)
    k.copy_(P.k)
    v.copy_(P.v)
    P.to_gpu = lambda t: k if t is P.k else v
    run(P, 2)


@pytest.mark.parametrize("page", [16, 64])
def test_many_calls_in_a_row_keep_their_bits(page):
    """A ragged verify round over long prefixes (72 rows a unit, units cut
    between CTAs), queued a hundred times without waiting: the tile rings of
    the two streams stay in step whatever order the copies land in."""
    g = torch.Generator(device="cuda").manual_seed(page)
    B, n, Hkv, G, D, kv = 24, 9, 8, 8, 128, 4096
    per = kv // page
    k = torch.randn(B * per, page, Hkv, D, generator=g, device="cuda").to(BF)
    v = torch.randn(B * per, page, Hkv, D, generator=g, device="cuda").to(BF)
    table = torch.randperm(B * per, generator=g, device="cuda").to(
        torch.int32).view(B, per)
    cache = api.PagedKV(k, v, table)
    start = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    kvl = (torch.rand(B, generator=g, device="cuda") * (kv - n) + n).to(
        torch.int32)
    q = torch.randn(B * n, G * Hkv, D, generator=g, device="cuda").to(BF)
    ws = api.Workspace()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [api.paged_attention(q, cache, start, kvl, max_q=n, workspace=ws,
                                status=st)["out"] for _ in range(100)]
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert all(torch.equal(o, outs[0]) for o in outs)
    b, t, h = 3, 4, 11  # one row against 64 bits
    last = int(kvl[b]) - n + t + 1
    kk = k[table[b].long()].flatten(0, 1)[:last, h // G].double()
    vv = v[table[b].long()].flatten(0, 1)[:last, h // G].double()
    p = torch.softmax(kk @ q[b * n + t, h].double() * D ** -0.5, 0)
    err = (outs[0][b * n + t, h].double() - p @ vv).abs()
    assert bool((err <= 2.0 ** -7 * (p @ vv.abs()) + 1e-4).all())


@pytest.mark.parametrize("hint", [1, 200])
def test_many_sequences(hint):
    """More sequences than a CTA looks over at once, empty ones and unusable
    ones among them."""
    r = np.random.default_rng(5)
    B = 700
    n = r.integers(0, 4, B)
    kv = n + r.integers(0, 30, B)
    n[300], kv[300] = 3, 400
    P = ref.Paged(n.tolist(), kv.tolist(), 1, 64, 8, BF, seed=101)
    run(P, 2, max_q=hint)
    q = P.rows(2).cuda()
    start, kvt = P.lengths()
    cache = api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda())
    want = api.paged_attention(q, cache, start, kvt, max_q=hint)["out"]
    bad = [b for b in (10, 290, 600, 699) if n[b] > 0]
    kvt[bad] = 10 ** 7
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.paged_attention(q, cache, start, kvt, max_q=hint,
                              status=st)["out"]
    assert int(st.item()) == (api.DEV_BAD_LENGTH if bad else 0)
    rows = torch.zeros(P.total, dtype=torch.bool, device="cuda")
    for b in bad:
        rows[P.start[b]:P.start[b + 1]] = True
    assert bool(torch.isnan(got[rows]).all())
    # the shares move, so a unit may be cut elsewhere: another order of sums
    err = (got[~rows].float() - want[~rows].float()).abs()
    assert bool((err <= 2.0 ** -7 * want[~rows].float().abs() + 1e-3).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("many", [False, True])
def test_units_of_one_tile_among_longer_ones(D, many):
    """Sequences of one key tile, of which one stream of a unit has nothing,
    between sequences of two and more; several units an SM, calls queued
    without waiting: no wait gives up, and every call has the same bits."""
    r = np.random.default_rng(D + many)
    B = 1200 if many else 300
    kv = np.where(r.random(B) < 0.8, r.integers(1, 129, B),
                  r.integers(129, 600, B)).tolist()
    P = ref.Paged([1] * B, kv, 2, D, 64, BF, seed=D)
    got = run(P, 4, max_q=1) if not many else None
    cache = api.PagedKV(P.to_gpu(P.k), P.to_gpu(P.v), P.table.cuda())
    q = P.rows(4, by=2.0).cuda()
    start, lens = P.lengths()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = api.Workspace()
    outs = [api.paged_attention(q, cache, start, lens, max_q=1, status=st,
                                workspace=ws)["out"] for _ in range(60)]
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool(torch.isfinite(outs[0]).all())
    assert all(torch.equal(o, outs[0]) for o in outs)
    assert many or got["out"].shape == outs[0].shape


def test_two_streams_without_a_workspace():
    """Calls of different shapes queued on two streams at once, whose units
    are cut (each leaves records and partial sums to a second kernel)."""
    calls = []
    for n, kv, heads, D in (([9], [6000], 2, 64),
                            ([2, 1], [3000, 900], 1, 128)):
        P = ref.Paged(n, kv, heads, D, 16, BF, seed=D)
        calls.append((P.rows(4 * heads).cuda(), api.PagedKV(
            P.k.cuda(), P.v.cuda(), P.table.cuda()), *P.lengths()))
    want = [api.paged_attention(*c)["out"] for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(api.paged_attention(*calls[i])["out"])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_a_graph_keeps_its_workspace():
    """A captured call, replayed after a larger call on the same Workspace and
    stream and after new tensors have taken what was free: the same bits, and
    nothing is written into those tensors."""
    small = ref.Paged([9], [3000], 1, 64, 16, BF, seed=3)
    large = ref.Paged([80], [700], 2, 128, 16, BF, seed=4)

    def args(P, Hq):
        return (P.rows(Hq).cuda(), api.PagedKV(
            P.k.cuda(), P.v.cuda(), P.table.cuda()), *P.lengths())
    a, b = args(small, 4), args(large, 8)
    ws, s = api.Workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        want = api.paged_attention(*a, workspace=ws)["out"]
        first = ws.get(a[1].device, 1)
        size = first.numel()
        del first
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = api.paged_attention(*a, workspace=ws)["out"]
        api.paged_attention(*b, workspace=ws)
        assert ws.get(a[1].device, 1).numel() > size
        torch.cuda.synchronize()
        taken = [torch.full((size,), 7, dtype=torch.uint8, device="cuda")
                 for _ in range(4)]
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((t == 7).all()) for t in taken)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hint", [1, 400])
@pytest.mark.parametrize("heavy", [(0,), (4095,), (0, 1700, 1701, 3000)])
@pytest.mark.parametrize("below,size", [(11.5, 1.0), (17.3, 8.0),
                                        (24.0, 4096.0), (36.0, 4096.0),
                                        (60.0, 4096.0)])
def test_few_heavy_keys_of_no_value_over_thousands(D, hint, heavy, below,
                                                   size):
    """fp16, a few keys whose values are 0 and thousands of others `below`
    nats under them (to 2^-34 of their weight), which are the whole result.

    Bound: a weight is off by its rounding (u; as two numbers less) and by
    2^-17 of the largest of its 64 keys, which lie within 2 nats of each other
    unless a heavy one is among them: then by 2^-28 of that, and by no more
    than itself; scores off by d; the sums; the output's rounding."""
    B, H, G, kv, page = 20, 8, 2, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(D + hint)
    score = torch.rand(B, kv, H, generator=g, device="cuda") * 2 - 1 - below
    score[:, list(heavy)] = 0
    k = torch.zeros(B, kv, H, D, device="cuda")
    k[..., 3] = (score + 12) * 0.25
    v = (torch.rand(B, kv, H, D, generator=g, device="cuda") + 0.5) * size
    v[:, list(heavy)] = 0
    k, v = k.to(HF), v.to(HF)
    q = torch.zeros(B, G * H, D, device="cuda", dtype=HF)
    q[..., 3] = 4.0
    table = torch.randperm(B * kv // page, generator=g, device="cuda").to(
        torch.int32)
    pages = [torch.empty(B * kv // page, page, H, D, dtype=HF, device="cuda")
             for _ in range(2)]
    for p, x in zip(pages, (k, v)):
        p[table.long()] = x.view(-1, page, H, D)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.paged_attention(
        q, api.PagedKV(*pages, table.view(B, -1)),
        torch.arange(B + 1, dtype=torch.int32, device="cuda"),
        torch.full((B,), kv, dtype=torch.int32, device="cuda"), max_q=hint,
        scale=1.0, want_lse=True, status=st, workspace=api.Workspace())
    assert int(st.item()) == 0
    s = torch.einsum("bhgd,bjhd->bhgj", q.view(B, H, G, D).double(),
                     k.double())
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[..., None])
    out = torch.einsum("bhgj,bjhd->bhgd", w, v.double())
    u = ref.U[HF]
    top = s.abs().max().item()
    d = 2 * ref.U32 * (D + 8) * top + 2.0 ** -20 + top * 4 * ref.U32
    # v >= 0: out is also the sum of the terms' sizes
    tol = out * (u * 1.01 + 2 * d + 2 * kv * ref.U32 + 2.0 ** -17 * np.e ** 2)
    tol += 64 * len(heavy) * min(2.0 ** -28, np.exp(1 - below)) * \
        v.max().item()
    tol += u * 1.01 * out + 2.0 ** -24
    err = (got["out"].view(B, H, G, D).double() - out).abs()
    assert bool((err <= tol).all()), (err / out).max().item()
    ltol = d + kv * ref.U32 + 128 * ref.U32
    assert bool(((got["lse"].view(B, H, G).double() - lse).abs()
                 <= ltol).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hint", [1, 200])
@pytest.mark.parametrize("n", [40, 300])
def test_empty_rows_beside_values_that_are_not_finite(D, hint, n):
    """Rows that see no key give 0 and -inf whatever the values of other rows'
    keys are: the mask leaves all rows empty but two, which see an infinity
    and a NaN."""
    P = ref.Paged([n, 3], [n, 20], 2, D, 16, BF, seed=n + D)
    see = [np.zeros((n, n), bool), np.tril(np.ones((3, 3), bool))]
    see[0][3, 0] = see[0][n - 1, n - 2] = True
    for j, x in ((0, np.inf), (n - 2, np.nan)):
        p, t = P.slot(0, j)
        P.v[p, t] = x
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = api.paged_attention(
        P.rows(8).cuda(), api.PagedKV(P.k.cuda(), P.v.cuda(), P.table.cuda()),
        *P.lengths(), max_q=hint, tree_mask=ref.pack_mask(see), want_lse=True,
        status=st, workspace=api.Workspace())
    assert int(st.item()) == 0
    empty = torch.ones(n + 3, dtype=torch.bool)
    empty[[3, n - 1, n, n + 1, n + 2]] = False
    assert bool((r["out"][empty.cuda()] == 0).all())
    assert bool((r["lse"][empty.cuda()] == -float("inf")).all())
    assert bool(torch.isinf(r["out"][3]).all() | torch.isnan(r["out"][3]).all())
    assert bool(torch.isnan(r["out"][n - 1]).all())
    assert bool(torch.isfinite(r["out"][n:]).all())
