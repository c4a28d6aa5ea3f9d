"""Cases of the 4-bit paged cache: what drafting over long contexts is bound by
are the cache's bytes, so keys and values are held in 4 bits.

    store   keys and values of new tokens quantised into the cache as they
            are written, keys and queries rotated by position on the way, and
            what the cache then stands for read back (a prompt's attention
            computed on the values that later steps will see)
    read    tokens of the cache back as 16-bit rows
    attend  attention of a chunk of new tokens (one token, gamma + 1 drafts,
            a token tree, part of a prompt) over the cache

A group of 32, 64 or 128 neighbours of a head's row has a pair (a, b) of fp16
numbers, and a code n in 0 .. 15 stands for the fp16 number nearest to
b + (64 + n) a.  `run` computes an operator in its plain form (elementary torch
operations in 32 bits) or, where `own` is true, through the library's entry
points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
#: what a value beyond is held as: 64 + 15 steps of a group stay below fp16's end
MOST = 6144.0
#: element of each nibble of a 32-bit word of codes, lowest nibble first
ORDER = [0, 2, 4, 6, 1, 3, 5, 7]


def _api():
    from speculative_decoding_verification_temperature_gb300 import api
    return api


# ---------------------------------------------------------------- the cases
def _case(name, op, dtype, B, q, kv, Hq, Hkv, D, page, group, *, ragged=True,
          tree=False, rot=0, interleaved=False, lse=False):
    """q: new tokens of the longest sequence ("read": tokens read of it); kv:
    keys of the longest one, those tokens among them.  ragged: the other
    sequences are shorter."""
    return {"name": name, "op": op, "dtype": dtype, "B": B, "q": q, "kv": kv,
            "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "group": group,
            "ragged": ragged, "tree": tree, "rot": rot,
            "interleaved": interleaved, "lse": lse}


def listed():
    return [
        # one sequence takes one more token: the smallest call there is
        _case("store-one", "store", "bf16", 1, 1, 300, 32, 8, 128, 16, 32,
              rot=128),
        # a round: gamma = 8 drafts and the root of 32 sequences
        _case("store-round", "store", "bf16", 32, 9, 1024, 64, 8, 128, 64,
              64, ragged=False, rot=128),
        # ragged prompts, half of each head rotated, neighbours as pairs
        _case("store-prompts", "store", "f16", 8, 4000, 4000, 32, 8, 128, 48,
              128, rot=64, interleaved=True),
        # a short prefix of an odd length, read back for a prompt's next part
        _case("read-short", "read", "bf16", 1, 777, 777, 8, 8, 64, 16, 32),
        # the prefixes of a batch back in 16 bits
        _case("read-prefixes", "read", "bf16", 16, 8192, 8192, 32, 8, 128,
              64, 64),
        # a short chat of a small model without shared heads: gamma = 4
        _case("attend-small", "attend", "bf16", 1, 5, 100, 8, 8, 64, 16, 32),
        # drafting of a ragged batch, one token a sequence
        _case("attend-single", "attend", "bf16", 64, 1, 8192, 32, 8, 128, 16,
              64),
        # drafting of one sequence behind a very long prefix
        _case("attend-long", "attend", "bf16", 1, 1, 262144, 32, 8, 128, 128,
              128),
        # a verify round over the same cache; the log-sum-exp too, for a
        # caller that joins this with attention over newer keys in 16 bits
        _case("attend-round", "attend", "bf16", 32, 9, 8192, 64, 8, 128, 64,
              64, lse=True),
        # token trees of 64 nodes, each node sees its ancestors
        _case("attend-tree", "attend", "f16", 16, 64, 4096, 32, 8, 128, 32,
              32, tree=True),
        # parts of two prompts over what is cached of them
        _case("attend-prompt", "attend", "bf16", 2, 4096, 12288, 32, 8, 128,
              64, 64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


#: A drawn case has no more bytes and operations than the largest listed ones,
#: and no more values in a plain form's score matrix or padded cache.
MOST_BYTES, MOST_FLOPS, MOST_SCORES, MOST_CACHE = 4.5e8, 1.2e12, 3.0e9, 1.0e9


def draw(rng):
    while True:
        op = rng.choice(["store", "read", "attend", "attend", "attend"])
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        kind = rng.choice({"store": ["one", "round", "prompt"],
                           "read": ["prompt"],
                           "attend": ["one", "round", "tree", "prompt"]}[op])
        q = {"one": 1, "round": rng.randint(2, 17),
             "tree": rng.randint(3, 130),
             "prompt": _log_int(rng, 18, 8192 if op == "read" else 4096)}[kind]
        B = _log_int(rng, 1, 8 if kind == "prompt" else 64)
        kv = _log_int(rng, q, {"store": 4096, "read": 8192,
                               "attend": 131072}[op] if q <= 4096 else 8192)
        c = _case("", op, rng.choice(["bf16", "bf16", "f16"]), B, q, kv,
                  rng.choice([1, 2, 3, 4, 5, 8, 16]) * Hkv, Hkv, D,
                  rng.choice([8, 16, 24, 32, 64, 128]),
                  rng.choice([g for g in (32, 64, 128) if g <= D]),
                  ragged=rng.random() < 0.7, tree=kind == "tree",
                  rot=rng.choice([D, D // 2, 0]) if op == "store" else 0,
                  interleaved=op == "store" and rng.random() < 0.4,
                  lse=op == "attend" and rng.random() < 0.4)
        if op == "attend" and B * c["Hq"] * q * kv > MOST_SCORES or \
                B * kv * Hkv * D > MOST_CACHE:
            continue
        w = work(c)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            del c["name"]
            return c


# ---------------------------------------------------------------- the inputs
def _lengths(case):
    """New tokens and keys of each sequence (by the case alone)."""
    B, q, kv = case["B"], case["q"], case["kv"]
    ql, kl = [q] * B, [kv] * B
    if case["ragged"]:
        r = random.Random(B * 1000003 + q * 1009 + kv)
        for b in range(1, B):
            if q > 17 and not case["tree"]:
                ql[b] = r.randint(max(1, q // 2), q)
            kl[b] = max(ql[b], int(kv * r.uniform(0.25, 1.0)))
            if case["op"] != "attend" and q == kv:
                kl[b] = ql[b]
    return ql, kl


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, by=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * by).to(dtype)


def _ancestors(B, q, seed):
    """Random trees: [B, q, q] truth values, node i sees its ancestors and
    itself; parents are among the eight nodes before it."""
    r = random.Random(int(seed))
    see = torch.zeros(B, q, q, dtype=torch.bool)
    for b in range(B):
        for i in range(q):
            if i:
                see[b, i] = see[b, r.randrange(max(0, i - 8), i)]
            see[b, i, i] = True
    return see


def _pack_mask(see):
    """Bits of [B, q, q] in 32-bit words, [B q, words]."""
    B, q, _ = see.shape
    words = (q + 31) // 32
    bits = torch.zeros(B, q, words * 32, dtype=torch.int64)
    bits[:, :, :q] = see
    w = (bits.view(B, q, words, 32) << torch.arange(32)).sum(-1)
    return (w - ((w >> 31) << 32)).to(torch.int32).view(B * q, words)


def _key_spread(D):
    """Keys of a head: one element in sixteen is four times the others, as
    the channels of trained projections are."""
    s = torch.ones(D, device="cuda")
    s[5::16] = 4.0
    return s


def _fill(codes, scale, g, group, spread):
    """Quantised random rows all over a cache, some pages at a time."""
    n, heads, page, half = codes.shape
    step = max(1, (1 << 25) // (heads * page * half * 2))
    for lo in range(0, n, step):
        m = min(step, n - lo)
        x = torch.randn((m, heads, page, half * 2), generator=g,
                        device="cuda")
        if spread is not None:
            x *= spread
        code, ab = _quantise(x, group)
        codes[lo:lo + m], scale[lo:lo + m] = _pack(code), ab


def prepare(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    B, Hq, Hkv, D, page, group = (
        case[x] for x in ("B", "Hq", "Hkv", "D", "page", "group"))
    ql, kl = _lengths(case)
    per = [-(-n // page) for n in kl]
    num = sum(per) + 3
    ids = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
    start = [0]
    for n in ql:
        start.append(start[-1] + n)
    total = start[-1]
    s = {"case": case, "table": table, "total": total, "max_q": max(ql),
         "max_kv": max(kl),
         "q_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(kl, dtype=torch.int32, device="cuda")}
    for x in ("k", "v"):
        s[x] = torch.zeros((num, Hkv, page, D // 2), dtype=torch.uint8,
                           device="cuda")
        s[x + "_scale"] = torch.zeros((num, Hkv, page, D // group, 2),
                                      dtype=torch.float16, device="cuda")
    if case["op"] == "store":
        # one projection's output: queries, keys and values of a token
        s["qkv"] = _randn(g, total, Hq + 2 * Hkv, D)
        s["qkv"][:, Hq:Hq + Hkv] *= _key_spread(D)
        s["qkv"] = s["qkv"].to(dt)
        s["cos_sin"] = None
        rot = case["rot"]
        if rot:
            f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2
                            / rot)
            a = torch.arange(case["kv"], dtype=torch.float64)[:, None] * f
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    else:
        _fill(s["k"], s["k_scale"], g, group, _key_spread(D))
        _fill(s["v"], s["v_scale"], g, group, None)
    if case["op"] == "attend":
        # scores of about N(0, 2.5^2): a softmax with a few large terms
        s["q"] = _randn(g, total, Hq, D, dtype=dt, by=1.8)
        s["mask"] = None
        if case["tree"]:
            s["mask"] = _pack_mask(_ancestors(B, case["q"], seed)).cuda()
    if own:  # the handle that a program keeps beside its cache
        s["cache"] = _api().PagedKV4(s["k"], s["v"], s["k_scale"],
                                     s["v_scale"], table, dt)
        s["workspace"] = _api().Workspace()
    return s


# ---------------------------------------------------------- the plain forms
def _quantise(x, group):
    """x [..., D] in 32 bits: codes [..., D] and pairs [..., D / group, 2]."""
    x = torch.where(torch.isfinite(x), x.clamp(-MOST, MOST), math.nan)
    x = x.unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    a = ((hi - lo) * torch.tensor(1 / 15, dtype=torch.float32)).half()
    b = (lo - a.float() * 64).half()
    n = ((x - b.float()) * a.float().reciprocal()).round() - 64
    n = torch.where(a > 0, n.clamp(0, 15), torch.zeros_like(n))
    return n.to(torch.uint8).flatten(-2), torch.cat([a, b], -1)


def _pack(code):
    w = code.unflatten(-1, (-1, 8))[..., ORDER]
    return (w[..., 0::2] | w[..., 1::2] << 4).flatten(-2)


def _values(codes, scale, group):
    """What packed codes [..., D / 2] stand for: fp16 [..., D]."""
    w = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    n = torch.empty_like(w).unflatten(-1, (-1, 8))
    n[..., ORDER] = w.unflatten(-1, (-1, 8))
    n = n.flatten(-2).unflatten(-1, (-1, group)).float()
    a, b = scale.float().split(1, -1)
    return (b + (n + 64) * a).half().flatten(-2)


def _rotate(x, cos, sin, rot, interleaved):
    """x [n, H, D] in 32 bits; cos, sin [n, rot / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    h = rot // 2
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _tokens(s):
    """The sequence of each token and its index in it."""
    t = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["q_start"], t, right=True) - 1
    i = t.long() - s["q_start"].long()[b]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    return b, i, s["kv_len"].long()[b] - n[b] + i


def _plain_read(s):
    c = s["case"]
    b, _, at = _tokens(s)
    page, slot = s["table"][b, at // c["page"]].long(), at % c["page"]
    return {x: _values(s[x][page, :, slot], s[x + "_scale"][page, :, slot],
                       c["group"]).to(DTYPES[c["dtype"]])
            for x in ("k", "v")}


def _plain_store(s):
    c = s["case"]
    Hq, Hkv, rot, group = c["Hq"], c["Hkv"], c["rot"], c["group"]
    b, _, at = _tokens(s)
    x = s["qkv"].float()
    qk = x[:, :Hq + Hkv]
    if rot:
        cs = s["cos_sin"][at]
        qk = _rotate(qk, cs[:, :rot // 2], cs[:, rot // 2:], rot,
                     c["interleaved"])
    page, slot = s["table"][b, at // c["page"]].long(), at % c["page"]
    for name, y in (("k", qk[:, Hq:]), ("v", x[:, Hq + Hkv:])):
        code, ab = _quantise(y, group)
        s[name][page, :, slot] = _pack(code)
        s[name + "_scale"][page, :, slot] = ab
    return {"q": qk[:, :Hq].to(s["qkv"].dtype), **_plain_read(s)}


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G, mq, S = Hq // Hkv, s["max_q"], s["max_kv"]
    pages = s["table"].long().clamp(min=0)

    def cached(x):  # [B, Hkv, S, D]
        y = _values(s[x][pages], s[x + "_scale"][pages], c["group"])
        return y.transpose(1, 2).flatten(2, 3)[:, :, :S].float()

    total = s["total"]
    row = torch.arange(mq, device="cuda")
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    at = (s["q_start"][:-1, None].long() + row).clamp(max=total - 1)
    q = s["q"][at].float().view(B, mq, Hkv, G, D).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.reshape(B, Hkv, G * mq, D),
                         cached("k").transpose(2, 3)) * D ** -0.5
    j = torch.arange(S, device="cuda")
    kv, ctx = s["kv_len"].long(), s["kv_len"].long() - n
    if s["mask"] is None:
        see = j <= (ctx[:, None] + row)[..., None]
    else:
        new = (j - ctx[:, None]).clamp(0, mq - 1)[:, None].expand(B, mq, S)
        word = s["mask"].view(B, mq, -1).long().gather(2, new >> 5)
        see = (((word >> (new & 31)) & 1) == 1) | (j < ctx[:, None])[:, None]
    see = see & (j < kv[:, None])[:, None]
    score = score.view(B, Hkv, G, mq, S).masked_fill(~see[:, None, None],
                                                     -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (score - top).exp()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hkv, G * mq, S), cached("v"))
    o = o.view(B, Hkv, G, mq, D) / l
    b, i, _ = _tokens(s)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, mq, Hq, D)
    r = {"out": o[b, i].to(s["q"].dtype)}
    if c["lse"]:
        lse = (top + l.log()).permute(0, 3, 1, 2, 4).reshape(B, mq, Hq)
        r["lse"] = lse[b, i]
    return r


def _own_read(s):
    return _api().kv4_read(s["cache"], s["q_start"], s["kv_len"], s["total"])


def _own_store(s):
    c = s["case"]
    Hq, Hkv, x = c["Hq"], c["Hkv"], s["qkv"]
    q = _api().kv4_append(s["cache"], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:],
                          s["q_start"], s["kv_len"], q=x[:, :Hq],
                          cos_sin=s["cos_sin"], interleaved=c["interleaved"])
    return {"q": q, **_own_read(s)}


def _own_attend(s):
    return _api().kv4_attention(
        s["q"], s["cache"], s["q_start"], s["kv_len"], max_q=s["max_q"],
        tree_mask=s["mask"], want_lse=s["case"]["lse"],
        workspace=s["workspace"])


PLAIN = {"store": _plain_store, "read": _plain_read, "attend": _plain_attend}
OWN = {"store": _own_store, "read": _own_read, "attend": _own_attend}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------- what it needs
def work(case):
    Hq, Hkv, D, rot, group = (case[x] for x in ("Hq", "Hkv", "D", "rot",
                                                "group"))
    ql, kl = _lengths(case)
    total = sum(ql)
    held = 2 * Hkv * (D // 2 + 4 * (D // group))  # bytes a token
    if case["op"] == "read":
        return {"bytes": total * (held + 2 * Hkv * D * 2),
                "flops": total * Hkv * D * 4}
    if case["op"] == "store":
        # in: the projection's output; out: queries, codes, values read back
        return {"bytes": total * ((Hq + 2 * Hkv) * D * 2 + Hq * D * 2 +
                                  2 * held + 2 * Hkv * D * 2 + rot * 4),
                "flops": total * ((Hq + Hkv) * rot * 3 + Hkv * D * 2 * 7)}
    seen = 0
    for n, kv in zip(ql, kl):
        # a chunk sees itself causally; of a tree, whose nodes see a few
        # ancestors each, the nodes alone are counted
        seen += n * (kv - n) + (n if case["tree"] else n * (n + 1) // 2)
    return {"bytes": 2 * total * Hq * D * 2 + sum(kl) * held,
            "flops": 4 * D * Hq * seen}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read,
            "attend": _exact_attend}[case["op"]](case, s, seed)


def _to32(x):
    return x.float().double()


def _to16(x):
    return x.float().half().double()


def _held(s, name, b, lo, hi):
    """Keys (or values) lo .. hi - 1 of sequence b: [n, heads, D]."""
    case = s["case"]
    page = s["table"][b].long()[torch.arange(lo, hi, device="cuda")
                                // case["page"]]
    slot = torch.arange(lo, hi, device="cuda") % case["page"]
    word = s[name].view(torch.int32)[page, :, slot].long()
    out = torch.empty(hi - lo, case["Hkv"], case["D"], dtype=torch.float64,
                      device="cuda")
    pair = s[name + "_scale"][page, :, slot].double()
    for nibble in range(8):
        e = 2 * nibble if nibble < 4 else 2 * nibble - 7
        at = torch.arange(e, case["D"], 8, device="cuda")
        a, b_ = (pair[..., at // case["group"], i] for i in (0, 1))
        out[..., e::8] = _to16(b_ + (64 + (word >> 4 * nibble & 15)) * a)
    return out


def _exact_read(case, s, seed):
    ql, kl = _lengths(case)
    return {x: torch.cat([_held(s, x, b, kv - n, kv)
                          for b, (n, kv) in enumerate(zip(ql, kl))])
            for x in ("k", "v")}


def _exact_store(case, s, seed):
    """The stored numbers are defined by 32-bit steps, so each is rounded."""
    ql, kl = _lengths(case)
    Hq, Hkv, D, rot, group = (case[x] for x in ("Hq", "Hkv", "D", "rot",
                                                "group"))
    x = s["qkv"].double()
    pos = torch.cat([torch.arange(kv - n, kv, device="cuda")
                     for n, kv in zip(ql, kl)])
    out = {}
    turned = x[:, :Hq + Hkv].clone()
    if rot:
        c, t = (y[:, None] for y in s["cos_sin"].double()[pos].split(
            rot // 2, 1))
        at = torch.arange(rot // 2, device="cuda")
        i, j = (2 * at, 2 * at + 1) if case["interleaved"] else \
            (at, at + rot // 2)
        xi, xj = turned[..., i], turned[..., j]
        out["q"] = x[:, :Hq].clone()
        out["q"][..., i] = (xi * c - xj * t)[:, :Hq]
        out["q"][..., j] = (xi * t + xj * c)[:, :Hq]
        turned[..., i] = _to32(_to32(xi * c) - _to32(xj * t))
        turned[..., j] = _to32(_to32(xi * t) + _to32(xj * c))
    else:
        out["q"] = x[:, :Hq]
    third = torch.tensor(1 / 15, dtype=torch.float32).double()
    for name, y in (("k", turned[:, Hq:]), ("v", x[:, Hq + Hkv:])):
        held = torch.empty_like(y)
        for lo in range(0, D, group):
            z = y[..., lo:lo + group].clamp(-MOST, MOST)
            low = z.min(-1, keepdim=True).values
            high = z.max(-1, keepdim=True).values
            a = _to16(_to32(_to32(high - low) * third))
            b = _to16(_to32(low - 64 * a))
            step = torch.where(a > 0, a, torch.ones_like(a))
            n = torch.round(_to32(_to32(z - b) * _to32(1 / step))) - 64
            n = torch.where(a > 0, n.clamp(0, 15), torch.zeros_like(n))
            held[..., lo:lo + group] = _to16(b + (64 + n) * a)
        out[name] = held
    return out


def _exact_attend(case, s, seed):
    ql, kl = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G, lo = Hq // Hkv, 0
    out = torch.zeros(sum(ql), Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(ql), Hq, dtype=torch.float64, device="cuda")
    trees = _ancestors(case["B"], case["q"], seed).cuda() if case["tree"] \
        else None
    for b, (n, kv) in enumerate(zip(ql, kl)):
        see = torch.ones(n, kv, dtype=torch.bool, device="cuda")
        see[:, kv - n:] = trees[b] if case["tree"] else \
            torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        k, v = _held(s, "k", b, 0, kv), _held(s, "v", b, 0, kv)
        for h in range(Hq):
            w = torch.einsum("id,jd->ij", s["q"][lo:lo + n, h].double(),
                             k[:, h // G]) / math.sqrt(D)
            w.masked_fill_(~see, -math.inf)
            lse[lo:lo + n, h] = torch.logsumexp(w, 1)
            out[lo:lo + n, h] = torch.einsum("ij,jd->id",
                                             torch.softmax(w, 1), v[:, h // G])
        lo += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
