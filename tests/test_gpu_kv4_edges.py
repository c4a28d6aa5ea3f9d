"""The 4-bit cache on the GPU at the ends of its ranges: queries near the
type's least and greatest numbers, values beyond what a group holds, tables
and rows at any address, batches past one block of sequences."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import kv4_ref as ref
from tests import operators_ref as oref
from tests.test_gpu_kv4 import run

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
# chunk and query heads of one cache head: the kernels of 8, 16, 128 and 256
# rows
SHAPES = [(1, 4), (3, 4), (20, 4), (70, 4)]


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("by", [1e-35, 1e-36, 1e-37, 1e-38])
@pytest.mark.parametrize("n,Hq", SHAPES)
def test_attention_queries_near_the_least_numbers(n, Hq, by):
    """bf16 rows down to its subnormal numbers, scores of a usual size."""
    P = ref.Paged4([n, 1], [n + 150, 30], 1, 64, 16, BF, 45, 32)
    run(P, Hq, scale=0.3 / by, q=P.rows(Hq, by=by), max_q=n)


@pytest.mark.parametrize("n,Hq", SHAPES)
def test_attention_a_factor_beyond_32_bits(n, Hq):
    """Scale times the queries' power of two is above 3.4e38, the scores are
    0: every key seen counts alike."""
    P = ref.Paged4([n, 1], [n + 150, 30], 1, 64, 16, BF, 46, 32)
    P.kn[:], P.kp[:] = ref.quantise(np.zeros_like(P.kn, np.float64), 32)
    P.k = torch.tensor(ref.values(P.kn, P.kp))
    q = torch.full((P.total, Hq, 64), 2.0 ** 127, dtype=BF)
    run(P, Hq, scale=2.0 ** 20, q=q, max_q=n)


def weight_bound(P, q, scale):
    """out, and a bound with weights that keep 22 bits (2^-21 of their own
    size counts twice that) and 2^-28 of the row's largest: what is left is
    the scores' and sums' 32 bits and the output's own rounding."""
    u, u32, D = oref.U[P.dtype], oref.U32, P.dim
    q64 = oref.f64(q)
    Hq = q64.shape[1]
    out, tol = np.zeros((P.total, Hq, D)), np.zeros((P.total, Hq, D))
    for b, (n, kv) in enumerate(zip(P.n, P.kv)):
        k, v = P.gather(P.k, b), P.gather(P.v, b)
        for i in range(n):
            m, r = kv - n + i + 1, P.start[b] + i
            for h in range(Hq):
                kh, vh = (x[:m, h // (Hq // P.heads)] for x in (k, v))
                s = kh @ q64[r, h] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                d = scale * 2 * u32 * (D + 8) * \
                    (np.abs(kh) @ np.abs(q64[r, h])).max() + 2.0 ** -20 + \
                    np.abs(s).max() * 4 * u32
                out[r, h] = w @ vh
                tol[r, h] = w @ np.abs(vh) * (2.0 ** -21 + 2 * d +
                                              2 * m * u32) + \
                    u * np.abs(out[r, h]) * 1.01 + 2.0 ** -24 + \
                    m * 2.0 ** -28 * np.abs(vh).max()
    return out, tol


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq", SHAPES[:3])
def test_attention_weights_keep_more_bits_than_the_type(n, Hq, D):
    """Up to 128 rows a head a weight is two fp16 numbers: where values cancel
    the result is off by less than one would leave."""
    P = ref.Paged4([n, n], [n + 2, n + 40], 1, D, 16, HF, 47, 32)
    q = P.rows(Hq, by=0.5)
    start, kv = P.lengths()
    got = oref.f64(api.kv4_attention(q.cuda(), P.cache(api), start, kv,
                                     max_q=n)["out"])
    out, tol = weight_bound(P, q, D ** -0.5)
    assert (np.abs(got - out) <= tol).all(), (np.abs(got - out) / tol).max()


@pytest.mark.parametrize("hint", [2, 4, 30, 100])
@pytest.mark.parametrize("masked", [False, True])
def test_attention_more_sequences_than_a_block_takes_at_once(hint, masked):
    """601 short ragged sequences, some of them empty, planned 256 at a time;
    hints that pick each kernel."""
    r = np.random.default_rng(8)
    n = r.integers(0, 4, 601)
    n[::7] = 0
    kv = n + r.integers(0, 90, 601)
    kv[5::50] += 300
    P = ref.Paged4(n.tolist(), kv.tolist(), 2, 64, 16, BF, 48, 32)
    see = None
    if masked:
        see = [np.tril(np.ones((m, m), bool)) for m in n]
        for t in see[::3]:
            t[:, :-1] = False  # the last token sees itself, others only keys
    run(P, 8, max_q=hint, see=see)


# ------------------------------------------------------------------ append
def inside(x):
    """x as a group of finite numbers holds it."""
    return np.clip(x, -ref.MOST, ref.MOST)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("at", [6144, -6144])
def test_append_beyond_the_end_in_narrow_groups(dtype, D, group, at):
    """Numbers near +-6144 and some beyond: the codes are those of the numbers
    kept inside, and what is held stays within their own rounding of them."""
    sign = 1 if at > 0 else -1
    P = ref.Paged4([16], [16], 1, D, 16, dtype, 12, group)
    g = np.random.default_rng(3)
    x = sign * (6144 - g.integers(0, 9, (16, 2, D)) * g.integers(
        0, 9, (16, 1, 1)).astype(np.float64))
    beyond = g.random((16, 2, D)) < 0.1
    x[beyond] = sign * g.choice([6150.0, 7000.0, 60000.0], beyond.sum())
    x[3] = np.where(g.random((2, D)) < 0.5, 7000.0, -60000.0)
    t = torch.tensor(x).to(dtype)
    cache = P.cache(api)
    start, kv = P.lengths()
    api.kv4_append(cache, t[:, :1].cuda(), t[:, 1:].cuda(), start, kv)
    y = inside(oref.f64(t))
    for i, (codes, pairs) in enumerate(((cache.k, cache.k_scale),
                                        (cache.v, cache.v_scale))):
        want, pair = ref.quantise(y[:, i], group)
        p = P.table[0, 0]
        np.testing.assert_array_equal(pairs.cpu().numpy()[p, 0],
                                      pair.astype(np.float16))
        np.testing.assert_array_equal(codes.cpu().numpy()[p, 0],
                                      ref.pack(want))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 48)])
def test_append_an_angle_table_at_any_address(interleaved, D, rot):
    """A table that starts 4, 8 or 12 bytes past 16-byte alignment: the bits
    of the aligned one, keys, values and queries."""
    P = ref.Paged4([40, 1, 7], [90, 30, 7], 2, D, 16, BF, 13, 32)
    x = P.rows(8).cuda()
    start, kv = P.lengths()
    tab = oref.cos_sin_table(90, rot).cuda()

    def call(table):
        cache = P.cache(api)
        q = api.kv4_append(cache, x[:, 4:6], x[:, 6:], start, kv, q=x[:, :4],
                           cos_sin=table, interleaved=interleaved)
        return [q, cache.k, cache.v, cache.k_scale.view(torch.int16),
                cache.v_scale.view(torch.int16)]

    want = call(tab)
    for off in (1, 2, 3):
        store = torch.full((tab.numel() + 4,), float("nan"), device="cuda")
        odd = store[off:off + tab.numel()].view(tab.shape)
        odd.copy_(tab)
        assert odd.data_ptr() % 16 == 4 * off
        for a, b in zip(call(odd), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 32, 34])
def test_append_rotated_rows_at_any_address(dtype, interleaved, rot):
    """Rows that are not 16-byte aligned, turned: the bits of aligned ones."""
    P = ref.Paged4([30, 2], [70, 9], 2, 64, 8, dtype, 14, 32)
    start, kv = P.lengths()
    tab = oref.cos_sin_table(70, rot).cuda()
    wide = torch.randn((32, 8 * 64 + 3), device="cuda").to(dtype)
    odd = wide[:, 1:513].unflatten(1, (8, 64))
    got = []
    for x in (odd, odd.contiguous()):
        cache = P.cache(api)
        q = api.kv4_append(cache, x[:, 4:6], x[:, 6:], start, kv, q=x[:, :4],
                           cos_sin=tab, interleaved=interleaved)
        got.append([q, cache.k, cache.v, cache.k_scale.view(torch.int16),
                    cache.v_scale.view(torch.int16)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
