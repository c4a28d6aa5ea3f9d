"""Plain 64-bit implementation (numpy) of the 4-bit cache: its numbers, its
quantisation as 32-bit steps, and the bounds that attention over it is
compared under."""
import numpy as np
import torch

from tests import operators_ref as ref

MOST = 6144.0
ORDER = np.array([0, 2, 4, 6, 1, 3, 5, 7])


def to32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def to16(x):
    with np.errstate(over="ignore"):
        return to32(x).astype(np.float32).astype(np.float16).astype(
            np.float64)


def quantise(x, group):
    """x [..., D] (32-bit numbers): codes [..., D] and pairs [..., D / group,
    2] (fp16 numbers)."""
    y = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, group))
    bad = ~np.isfinite(y).all(-1, keepdims=True)
    y = np.where(bad, 0.0, y)
    lo = np.clip(y.min(-1, keepdims=True), -MOST, MOST)
    hi = np.clip(y.max(-1, keepdims=True), -MOST, MOST)
    a = to16(to32(to32(hi - lo) * np.float64(np.float32(1 / 15))))
    b = to16(to32(lo - 64 * a))
    r = to32(1 / np.where(a > 0, a, 1))
    n = np.clip(np.rint(to32(to32(y - b) * r)) - 64, 0, 15)
    n = np.where((a > 0) & ~bad, n, 0).astype(np.uint8)
    pair = np.where(bad, np.nan, np.concatenate([a, b], -1))
    return n.reshape(x.shape), pair


def pack(n):
    w = n.reshape(n.shape[:-1] + (-1, 8))[..., ORDER]
    return (w[..., 0::2] | w[..., 1::2] << 4).reshape(
        n.shape[:-1] + (n.shape[-1] // 2,))


def unpack(codes):
    w = np.stack([codes & 15, codes >> 4], -1).reshape(
        codes.shape[:-1] + (-1, 8))
    n = np.empty_like(w)
    n[..., ORDER] = w
    return n.reshape(codes.shape[:-1] + (codes.shape[-1] * 2,))


def values(n, pair):
    """What codes [..., D] stand for."""
    g = n.shape[-1] // pair.shape[-2]
    y = n.reshape(n.shape[:-1] + (-1, g)).astype(np.float64)
    return to16(pair[..., 1:] + (64 + y) * pair[..., :1]).reshape(n.shape)


class Paged4(ref.Paged):
    """A batch of sequences over a shuffled 4-bit cache.  Every pair outside
    the sequences' own keys is NaN: nothing may read it into a result.
    k and v are the numbers the codes stand for."""

    def __init__(self, n, kv, heads, dim, page, dtype, seed, group=32, *,
                 by=1.0, device="cuda", apart=0):
        super().__init__(n, kv, heads, dim, page, torch.float32, seed,
                         device=device)
        self.dtype, self.group, self.apart = dtype, group, apart
        out = []
        for t in (self.k, self.v):
            x = t.numpy().astype(np.float64) * by  # [pages, page, heads, dim]
            code, pair = quantise(x, group)
            out.append((code, pair, torch.tensor(values(code, pair))))
        (self.kn, self.kp, self.k), (self.vn, self.vp, self.v) = out

    def cache(self, api, table=None):
        """The cache on the GPU, pages `apart` bytes apart."""
        def lay(x, dt):  # [pages, page, heads, row] -> head-major pages
            x = torch.tensor(np.ascontiguousarray(x.swapaxes(1, 2)))
            x = x.to(dt)
            per = x[0].numel()
            gap = self.apart // x.element_size()
            store = torch.full((x.shape[0], per + gap), 255 if dt ==
                               torch.uint8 else float("nan"), dtype=dt,
                               device=self.device)
            t = store[:, :per].view(x.shape)
            t.copy_(x)
            return t
        H = torch.float16
        return api.PagedKV4(
            lay(pack(self.kn), torch.uint8), lay(pack(self.vn), torch.uint8),
            lay(self.kp, H), lay(self.vp, H),
            (self.table if table is None else table).to(self.device),
            self.dtype)


def held(cache):
    """The numbers a PagedKV4 holds: k, v [pages, page, heads, dim]."""
    r = []
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        n = unpack(c.cpu().numpy()).swapaxes(1, 2)
        r.append(values(n, s.cpu().numpy().astype(np.float64).swapaxes(1, 2)))
    return r


def attention(P, q, scale, see=None):
    """64-bit attention over the numbers of a Paged4 batch, and bounds.
    Products of fp16 numbers are exact in fp32 and their sums rounded (in any
    order, perhaps with truncation); weights are fp16, rounded once, those
    2^-24 and less of the row's largest to a multiple of 2^-25 of it at most;
    the output is rounded to its type."""
    u, uw, u32 = ref.U[P.dtype], 2.0 ** -11, ref.U32
    q64 = ref.f64(q)
    Hq, D = q64.shape[1:]
    G = Hq // P.heads
    out = np.zeros((P.total, Hq, D))
    lse = np.full((P.total, Hq), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros((P.total, Hq))
    for b, (n, kv) in enumerate(zip(P.n, P.kv)):
        k, v = P.gather(P.k, b), P.gather(P.v, b)
        ok = np.zeros((n, kv), bool)
        ok[:, :kv - n] = True
        ok[:, kv - n:] = np.tril(np.ones((n, n), bool)) if see is None \
            else see[b]
        rows = slice(P.start[b], P.start[b] + n)
        for h in range(Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            qh = q64[rows, h]
            s = qh @ kh.T * scale
            ds = scale * (2 * u32 * (D + 8) * (np.abs(qh) @ np.abs(kh).T) +
                          2.0 ** -38 * np.abs(qh).max(-1, keepdims=True) *
                          np.abs(kh).sum(-1)[None])
            s = np.where(ok, s, -np.inf)
            for i in range(n):
                if not ok[i].any():
                    continue
                m = s[i].max()
                w = np.exp(s[i] - m)
                l = w.sum()
                r = P.start[b] + i
                out[r, h] = w @ vh / l
                lse[r, h] = m + np.log(l)
                d = np.where(ok[i], ds[i], 0).max() + 2.0 ** -20 + \
                    np.abs(m) * 4 * u32
                size = w @ np.abs(vh) / l
                tol[r, h] = size * (uw * 1.01 + 2 * d + 2 * kv * u32) + \
                    u * np.abs(out[r, h]) * 1.01 + \
                    ok[i].sum() * 2.0 ** -25 * np.abs(vh[ok[i]]).max() + \
                    (2.0 ** -24 if P.dtype == torch.float16 else 0)
                ltol[r, h] = d + kv * u32 + 8 * u32 * (1 + abs(lse[r, h]))
    return out, lse, tol, ltol
