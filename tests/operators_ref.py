"""Plain 64-bit implementations (numpy) of the paged-cache append, the
chunk attention and the distillation loss with its gradient, written from
their formulas, and the rounding bounds the GPU tests compare under.

Unit roundoffs: bf16 has 8 significand bits (u = 2^-8), fp16 11 (2^-11),
fp32 24 (2^-24)."""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11,
     torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


# ------------------------------------------------------------ paged cache
class Paged:
    """A batch of sequences over a shuffled paged cache: n new tokens and kv
    keys each.  Every cache element outside the sequences' own keys is
    `fill` (NaN by default): nothing may read it into a result."""

    def __init__(self, n, kv, heads, dim, page, dtype, seed, *, fill=np.nan,
                 head_major=False, extra_cols=1, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.n, self.kv, self.page, self.dtype = list(n), list(kv), page, dtype
        self.heads, self.dim, self.device = heads, dim, device
        need = [-(-x // page) for x in kv]
        num = sum(need) + 2
        ids = torch.randperm(num, generator=g).tolist()
        cols = max(need + [0]) + extra_cols
        table = torch.full((len(kv), cols), -1, dtype=torch.int32)
        shape = (num, heads, page, dim) if head_major \
            else (num, page, heads, dim)
        kc = torch.full(shape, fill, dtype=dtype)
        vc = torch.full(shape, fill, dtype=dtype)
        if head_major:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        at = 0
        for b, m in enumerate(need):
            mine = ids[at:at + m]
            at += m
            table[b, :m] = torch.tensor(mine, dtype=torch.int32)
            for j in range(kv[b]):
                p, t = mine[j // page], j % page
                kc[p, t] = torch.randn((heads, dim), generator=g).to(dtype)
                vc[p, t] = torch.randn((heads, dim), generator=g).to(dtype)
        self.k, self.v = kc, vc
        self.table = table
        self.start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.total = int(self.start[-1])
        self.gen = g

    def rows(self, heads, by=1.0, dtype=None):
        return (torch.randn((self.total, heads, self.dim), generator=self.gen)
                * by).to(dtype or self.dtype)

    def to_gpu(self, t):
        """The tensor on the GPU with the same strides."""
        if t.is_contiguous():
            return t.to(self.device)
        return t.transpose(1, 2).contiguous().to(self.device).transpose(1, 2)

    def lengths(self):
        return (torch.tensor(self.start, dtype=torch.int32,
                             device=self.device),
                torch.tensor(self.kv, dtype=torch.int32, device=self.device))

    def slot(self, b, j):
        return int(self.table[b, j // self.page]), j % self.page

    def gather(self, cache, b):
        """Keys (or values) of sequence b: [kv, heads, dim], 64 bits."""
        if self.kv[b] == 0:
            return np.zeros((0, self.heads, self.dim))
        pages = self.table[b, :-(-self.kv[b] // self.page)].long()
        return f64(cache[pages].reshape(-1, self.heads, self.dim)
                   [:self.kv[b]])


def cos_sin_table(max_pos, rot, base=10000.0):
    f = base ** (-np.arange(rot // 2) * 2.0 / rot)
    a = np.arange(max_pos)[:, None] * f
    return torch.tensor(np.concatenate([np.cos(a), np.sin(a)], 1),
                        dtype=torch.float32)


def rotate(x, table, pos, interleaved):
    """x [rows, heads, dim] in 64 bits, table [max_pos, rot], pos [rows]:
    the rotated rows and |x| |c| + |y| |s| of every element."""
    rot = table.shape[1]
    h = rot // 2
    y, size = x.copy(), np.abs(x)
    for r, p in enumerate(pos):
        c, s = table[p, :h], table[p, h:]
        ia = np.arange(0, rot, 2) if interleaved else np.arange(h)
        ib = ia + 1 if interleaved else ia + h
        a, b = x[r][:, ia], x[r][:, ib]
        y[r][:, ia], y[r][:, ib] = a * c - b * s, a * s + b * c
        size[r][:, ia] = np.abs(a * c) + np.abs(b * s)
        size[r][:, ib] = np.abs(a * s) + np.abs(b * c)
    return y, size


def append_tol(exact, size, dtype):
    """fp32 products and sum (three roundings of the terms' size), then one
    rounding to the type; half an fp16 subnormal step."""
    return U[dtype] * (np.abs(exact) + 4 * U32 * size) + 4 * U32 * size + \
        (2.0 ** -25 if dtype == torch.float16 else 0.0)


def attention(P, q, scale, see=None, split=False):
    """64-bit attention of a Paged batch: out, lse and the bounds of their
    errors.  see: list of [n, n] truth tables of the chunk (None: causal).
    split: weights are sums of two numbers of the type, the first perhaps cut
    off (2 u away at most) and the second rounded (u of that)."""
    q64 = f64(q)
    Hq, D = q64.shape[1:]
    G = Hq // P.heads
    out = np.zeros((P.total, Hq, D))
    lse = np.full((P.total, Hq), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros((P.total, Hq))
    u = U[P.dtype]
    uw = 2 * u * u if split else u
    for b, (n, kv) in enumerate(zip(P.n, P.kv)):
        k, v = P.gather(P.k, b), P.gather(P.v, b)
        ok = np.zeros((n, kv), bool)
        ok[:, :kv - n] = True
        ok[:, kv - n:] = np.tril(np.ones((n, n), bool)) if see is None \
            else see[b]
        rows = slice(P.start[b], P.start[b] + n)
        for h in range(Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            s = q64[rows, h] @ kh.T * scale
            # products summed in fp32 in any order, possibly with truncation
            ds = scale * 2 * U32 * (D + 8) * (np.abs(q64[rows, h])
                                              @ np.abs(kh).T)
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
                    np.abs(m) * 4 * U32
                size = w @ np.abs(vh) / l
                # weights rounded to the type (fp16 also in its subnormal
                # range), their exponents off by d, the sums, the output
                tol[r, h] = size * (uw * 1.01 + 2 * d + 2 * kv * U32) + \
                    u * np.abs(out[r, h]) * 1.01 + \
                    (ok[i].sum() * 2.0 ** -24 * np.abs(vh[ok[i]]).max()
                     + 2.0 ** -24 if P.dtype == torch.float16 else 0)
                ltol[r, h] = d + kv * U32 + 8 * U32 * (1 + abs(lse[r, h]))
    return out, lse, tol, ltol


def pack_mask(see, device="cuda"):
    """List of [n, n] truth tables -> [total, words] int32."""
    words = max(1, -(-max([x.shape[0] for x in see] + [1]) // 32))
    rows = []
    for m in see:
        n = m.shape[0]
        bits = np.zeros((n, words * 32), np.uint64)
        bits[:, :n] = m
        w = (bits.reshape(n, words, 32)
             << np.arange(32, dtype=np.uint64)).sum(-1)
        rows.append(w.astype(np.uint32).view(np.int32))
    return torch.tensor(np.concatenate(rows), device=device)


# ----------------------------------------------------------- distillation
def distill(student, logit, ids, T, teacher_lse=None, g=None):
    """64-bit loss, lse and gradient of every row, and their bounds."""
    z = np.asarray(student, np.float64) / T
    N, V = z.shape
    t = np.asarray(logit, np.float64) / T
    r = {k: np.zeros(N) for k in ("loss", "lse", "loss_tol", "lse_tol")}
    grad, gtol = np.zeros((N, V)), np.zeros((N, V))
    for n in range(N):
        zf = z[n]
        m = zf.max()
        lse = m + np.log(np.exp(zf - m).sum())
        size = np.abs(zf[np.isfinite(zf)]).max()
        # at most V / 256 + 64 terms summed one after the other in fp32,
        # each 2^x to 2^-22 and its argument to a few roundings of `size`
        lse_tol = (V / 256 + 64) * U32 + 8 * U32 * (1 + size + abs(lse))
        use = (ids[n] >= 0) & (ids[n] < V) & (t[n] > -np.inf)
        p = np.zeros(V)
        loss = ltol = 0.0
        P = 0.0
        if use.any():
            tk = t[n][use]
            ref = teacher_lse[n] if teacher_lse is not None else \
                tk.max() + np.log(np.exp(tk - tk.max()).sum())
            tsize = np.abs(tk).max() + abs(ref)
            rel = 16 * U32 * (1 + tsize) + 256 * U32
            for i, x in zip(ids[n][use], tk):
                pk = np.exp(x - ref)
                if pk > 0:
                    loss += pk * ((x - ref) - (zf[i] - lse))
                    ltol += pk * (rel * (1 + abs(x - ref) + abs(zf[i] - lse))
                                  + 8 * U32 * (abs(zf[i]) + abs(lse)))
                p[i] += pk
                P += pk
        r["loss"][n], r["lse"][n], r["lse_tol"][n] = loss, lse, lse_tol
        r["loss_tol"][n] = ltol + P * lse_tol if use.any() else 0.0
        if g is not None and use.any():
            q = np.exp(zf - lse)
            grad[n] = g[n] / T * (P * q - p)
            dz = np.where(np.isfinite(zf), np.abs(zf - lse), 0)
            gtol[n] = abs(g[n]) / T * (
                P * q * (rel + lse_tol + 16 * U32 * (1 + dz)) +
                p * (rel + 64 * U32))
    r["grad"], r["grad_tol"] = grad, gtol
    return r
