"""Cases of the operators around the verify step: what a speculative round does
before it (the new tokens' keys and values are rotated and appended to a paged
cache, and the chunk of new tokens attends over it) and after it (the drafter
is distilled from the target's top logits).

    append   keys and values of new tokens into the paged cache, keys and
             queries rotated by position on the way
    attend   attention of a chunk of new tokens (one token, gamma + 1 drafts,
             a token tree, part of a prompt) over the paged cache
    distill  KL from the target's top-K logits to the drafter's softmax:
             the loss ("forward"), its gradient ("backward"), both ("step")

`run` computes an operator in its plain form (elementary torch operations in
32 bits) or, where `own` is true, through the library's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _api():
    from speculative_decoding_verification_temperature_gb300 import api
    return api


# ---------------------------------------------------------------- the cases
def _paged(name, op, dtype, B, q, kv, Hq, Hkv, D, page, *, ragged=True,
           tree=False, rot=0, interleaved=False, lse=False):
    """q: new tokens of the longest sequence; kv: keys of the longest one,
    the new tokens among them.  ragged: the other sequences are shorter."""
    return {"name": name, "op": op, "dtype": dtype, "B": B, "q": q, "kv": kv,
            "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "ragged": ragged,
            "tree": tree, "rot": rot, "interleaved": interleaved, "lse": lse}


def _distill(name, part, dtype, N, V, K, T, *, full=False):
    """full: the target's log-sum-exp over its whole vocabulary is given, so
    the top-K probabilities are the target's own; otherwise they are
    normalised among themselves."""
    return {"name": name, "op": "distill", "part": part, "dtype": dtype,
            "N": N, "V": V, "K": K, "T": T, "full": full}


def listed():
    return [
        # one sequence takes one more token: the smallest call there is
        _paged("append-one", "append", "bf16", 1, 1, 300, 32, 8, 128, 16,
               rot=128),
        # a verify round: gamma = 8 drafts and the root of 32 sequences
        _paged("append-round", "append", "bf16", 32, 9, 1024, 64, 8, 128, 64,
               ragged=False, rot=128),
        # ragged prompts, half of each head rotated, neighbours as pairs
        _paged("append-prompts", "append", "f16", 8, 4000, 4000, 32, 8, 128,
               48, rot=64, interleaved=True),
        # a short chat of a small model without shared heads: gamma = 4
        _paged("attend-small", "attend", "bf16", 1, 5, 100, 8, 8, 64, 16),
        # plain decoding of a ragged batch, one token a sequence
        _paged("attend-single", "attend", "bf16", 64, 1, 8192, 32, 8, 128,
               16),
        # a verify round over long prefixes; the log-sum-exp too, for a
        # caller that joins this with attention over a shared prefix
        _paged("attend-round", "attend", "bf16", 32, 9, 8192, 64, 8, 128, 64,
               lse=True),
        # token trees of 64 nodes, each node sees its ancestors
        _paged("attend-tree", "attend", "f16", 16, 64, 4096, 32, 8, 128, 32,
               tree=True),
        # one sequence with a very long prefix, gamma = 8
        _paged("attend-long", "attend", "bf16", 1, 9, 131072, 32, 8, 128,
               128),
        # parts of two prompts over what is cached of them
        _paged("attend-prompt", "attend", "bf16", 2, 4096, 12288, 32, 8, 128,
               64),
        # loss alone, as an evaluation reads it: one round's rows
        _distill("distill-loss", "forward", "f32", 288, 32000, 16, 0.7),
        # gradient from a saved log-sum-exp; an odd number of rows
        _distill("distill-grad", "backward", "bf16", 1021, 152064, 50, 1.0),
        # training on the rows of 256 sequences of gamma = 8 drafts
        _distill("distill-step", "step", "bf16", 2048, 128256, 64, 1.0,
                 full=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


#: A drawn case has no more bytes and operations than the largest listed ones,
#: and no more values in a plain form's score matrix or padded cache.
MOST_BYTES, MOST_FLOPS, MOST_SCORES, MOST_CACHE = 1.0e9, 1.2e12, 3.0e9, 2.0e9


def draw(rng):
    while True:
        op = rng.choice(["append", "attend", "attend", "distill"])
        if op == "distill":
            c = _distill("", rng.choice(["forward", "backward", "step"]),
                         rng.choice(["bf16", "bf16", "f32"]),
                         _log_int(rng, 1, 2048), _log_int(rng, 1000, 160000),
                         _log_int(rng, 1, 128), rng.choice([0.7, 1.0, 2.0]),
                         full=rng.random() < 0.5)
            c["K"] = min(c["K"], c["V"])
        else:
            D, group = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 8, 16])
            Hkv = rng.choice([1, 2, 4, 8])
            kind = rng.choice(["one", "round", "tree", "prompt"])
            if op == "append" and kind == "tree":
                kind = "round"
            q = {"one": 1, "round": rng.randint(2, 17),
                 "tree": rng.randint(3, 130),
                 "prompt": _log_int(rng, 18, 4096)}[kind]
            B = _log_int(rng, 1, 8 if kind == "prompt" else 64)
            kv = _log_int(rng, q, 4096 if op == "append" else 65536)
            c = _paged("", op, rng.choice(["bf16", "f16"]), B, q, kv,
                       group * Hkv, Hkv, D,
                       rng.choice([8, 16, 24, 32, 64, 128]),
                       ragged=rng.random() < 0.7, tree=kind == "tree",
                       rot=rng.choice([D, D // 2]) if op == "append" else 0,
                       interleaved=op == "append" and rng.random() < 0.4,
                       lse=op == "attend" and rng.random() < 0.4)
            if B * c["Hq"] * q * kv > MOST_SCORES or \
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
            if case["op"] == "append" and q == kv:
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


def _pack(see):
    """Bits of [B, q, q] in 32-bit words, [B q, words]."""
    B, q, _ = see.shape
    words = (q + 31) // 32
    bits = torch.zeros(B, q, words * 32, dtype=torch.int64)
    bits[:, :, :q] = see
    w = (bits.view(B, q, words, 32) << torch.arange(32)).sum(-1)
    return (w - ((w >> 31) << 32)).to(torch.int32).view(B * q, words)


def _prepare_paged(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    B, Hq, Hkv, D, page = (case[x] for x in ("B", "Hq", "Hkv", "D", "page"))
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
    s = {"case": case, "table": table, "max_q": max(ql), "max_kv": max(kl),
         "q_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(kl, dtype=torch.int32, device="cuda"),
         "k_cache": _randn(g, num, page, Hkv, D, dtype=dt),
         "v_cache": _randn(g, num, page, Hkv, D, dtype=dt)}
    total = start[-1]
    if case["op"] == "append":
        # one projection's output: queries, keys and values of a token
        s["qkv"] = _randn(g, total, Hq + 2 * Hkv, D, dtype=dt)
        rot = case["rot"]
        f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
        a = torch.arange(case["kv"], dtype=torch.float64)[:, None] * f
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    else:
        # scores of about N(0, 2.5^2): a softmax with a few large terms
        s["q"] = _randn(g, total, Hq, D, dtype=dt, by=2.5)
        s["mask"] = None
        if case["tree"]:
            s["mask"] = _pack(_ancestors(B, case["q"], seed)).cuda()
    if own:  # the handle that a program keeps beside its cache
        s["cache"] = _api().PagedKV(s["k_cache"], s["v_cache"], table)
        s["workspace"] = _api().Workspace()
    return s


def _prepare_distill(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    N, V, K, T = (case[x] for x in ("N", "V", "K", "T"))
    target = _randn(g, N, V, by=3.0)
    student = (target + _randn(g, N, V)).to(dt)
    top = target.topk(K, dim=1)
    s = {"case": case, "student": student, "logit": top.values.contiguous(),
         "id": top.indices.to(torch.int32),
         "teacher_lse": (target / T).logsumexp(1) if case["full"] else None,
         # weights of the rows in the training loss; some are padding
         "weight": (torch.rand(N, generator=g, device="cuda") + 0.5) / N *
         (torch.rand(N, generator=g, device="cuda") > 0.05)}
    if case["part"] == "backward":
        s["lse"] = (student.float() / T).logsumexp(1)
    return s


def prepare(case, seed):
    return (_prepare_distill if case["op"] == "distill" else
            _prepare_paged)(case, seed)


# ---------------------------------------------------------- the plain forms
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


def _tokens(s, total):
    """The sequence of each new token and its number in it."""
    t = torch.arange(total, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["q_start"], t, right=True) - 1
    return b, t.long() - s["q_start"].long()[b]


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, rot, page = c["Hq"], c["Hkv"], c["rot"], c["page"]
    dt = s["qkv"].dtype
    b, i = _tokens(s, s["qkv"].shape[0])
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    at = s["kv_len"].long()[b] - n[b] + i
    cs = s["cos_sin"][at]
    cos, sin = cs[:, :rot // 2], cs[:, rot // 2:]
    x = s["qkv"].float()
    q = _rotate(x[:, :Hq], cos, sin, rot, c["interleaved"]).to(dt)
    k = _rotate(x[:, Hq:Hq + Hkv], cos, sin, rot, c["interleaved"]).to(dt)
    where = (s["table"][b, at // page].long(), at % page)
    s["k_cache"][where] = k
    s["v_cache"][where] = s["qkv"][:, Hq + Hkv:]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G, mq, S = Hq // Hkv, s["max_q"], s["max_kv"]
    pages = s["table"].long().clamp(min=0)
    k = s["k_cache"][pages].flatten(1, 2)[:, :S].float().permute(0, 2, 3, 1)
    v = s["v_cache"][pages].flatten(1, 2)[:, :S].float().transpose(1, 2)
    total = s["q"].shape[0]
    row = torch.arange(mq, device="cuda")
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    at = (s["q_start"][:-1, None].long() + row).clamp(max=total - 1)
    q = s["q"][at].float().view(B, mq, Hkv, G, D).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.reshape(B, Hkv, G * mq, D), k) * D ** -0.5
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
    o = torch.matmul(e.view(B, Hkv, G * mq, S), v).view(B, Hkv, G, mq, D) / l
    b, i = _tokens(s, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, mq, Hq, D)
    r = {"out": o[b, i].to(s["q"].dtype)}
    if c["lse"]:
        lse = (top + l.log()).permute(0, 3, 1, 2, 4).reshape(B, mq, Hq)
        r["lse"] = lse[b, i]
    return r


def _plain_distill(s):
    c = s["case"]
    T = c["T"]
    ids = s["id"].long()
    z, t = s["student"].float() / T, s["logit"] / T
    if s["teacher_lse"] is None:
        top = t.amax(1, keepdim=True)
        logp = t - top - (t - top).exp().sum(1, keepdim=True).log()
    else:
        logp = t - s["teacher_lse"][:, None]
    p = logp.exp()
    r = {}
    if c["part"] == "backward":
        lse = s["lse"]
    else:
        top = z.amax(1, keepdim=True)
        lse = ((z - top).exp().sum(1, keepdim=True).log() + top)[:, 0]
        logq = z.gather(1, ids) - lse[:, None]
        r["loss"], r["lse"] = (p * (logp - logq)).sum(1), lse
    if c["part"] != "forward":
        d = (z - lse[:, None]).exp() * p.sum(1, keepdim=True)
        d.scatter_add_(1, ids, -p)
        r["grad"] = (d * (s["weight"] / T)[:, None]).to(s["student"].dtype)
    return r


def _own_append(s):
    c = s["case"]
    Hq, Hkv, x = c["Hq"], c["Hkv"], s["qkv"]
    q = _api().kv_append(s["cache"], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:],
                         s["q_start"], s["kv_len"], q=x[:, :Hq],
                         cos_sin=s["cos_sin"], interleaved=c["interleaved"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    return _api().paged_attention(
        s["q"], s["cache"], s["q_start"], s["kv_len"], max_q=s["max_q"],
        tree_mask=s["mask"], want_lse=s["case"]["lse"],
        workspace=s["workspace"])


def _own_distill(s):
    api, c = _api(), s["case"]
    t = (s["logit"], s["id"])
    kw = {"teacher_lse": s["teacher_lse"]}
    if c["part"] == "forward":
        return api.distill_topk(s["student"], *t, c["T"], **kw)
    if c["part"] == "backward":
        return {"grad": api.distill_topk_backward(
            s["student"], s["lse"], *t, s["weight"], c["T"], **kw)}
    return api.distill_topk_step(s["student"], *t, s["weight"], c["T"], **kw)


PLAIN = {"append": _plain_append, "attend": _plain_attend,
         "distill": _plain_distill}
OWN = {"append": _own_append, "attend": _own_attend, "distill": _own_distill}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------- what it needs
def work(case):
    if case["op"] == "distill":
        N, V, K = case["N"], case["V"], case["K"]
        elt = 4 if case["dtype"] == "f32" else 2
        part = case["part"]
        moved = N * V * elt * (1 if part == "forward" else 2)
        return {"bytes": moved + N * K * 8 + N * 12,
                "flops": N * V * {"forward": 3, "backward": 4, "step": 6}[part]}
    Hq, Hkv, D, rot = (case[x] for x in ("Hq", "Hkv", "D", "rot"))
    ql, kl = _lengths(case)
    total = sum(ql)
    if case["op"] == "append":
        return {"bytes": total * (2 * (Hq + 2 * Hkv) * D * 2 + rot * 4),
                "flops": total * (Hq + Hkv) * rot * 3}
    seen = 0
    for n, kv in zip(ql, kl):
        # a chunk sees itself causally; of a tree, whose nodes see a few
        # ancestors each, the nodes alone are counted
        seen += n * (kv - n) + (n if case["tree"] else n * (n + 1) // 2)
    return {"bytes": 2 * total * Hq * D * 2 + sum(kl) * Hkv * D * 2 * 2,
            "flops": 4 * D * Hq * seen}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend,
            "distill": _exact_distill}[case["op"]](case, seed)


def _exact_append(case, seed):
    s = prepare(case, seed)
    ql, kl = _lengths(case)
    Hq, Hkv, rot, page = (case[x] for x in ("Hq", "Hkv", "rot", "page"))
    K, V = s["k_cache"].double(), s["v_cache"].double()
    x = s["qkv"].double()
    table = s["cos_sin"].double()
    for b, (n, kv) in enumerate(zip(ql, kl)):
        lo = sum(ql[:b])
        pos = torch.arange(kv - n, kv, device="cuda")
        # a pair (a, b) is the complex number a + ib, turned by its angle
        turn = torch.complex(table[pos, :rot // 2], table[pos, rot // 2:])
        part = x[lo:lo + n, :Hq + Hkv, :rot]
        if case["interleaved"]:
            pair = torch.complex(part[..., 0::2].contiguous(),
                                 part[..., 1::2].contiguous())
            pair = pair * turn[:, None]
            new = torch.view_as_real(pair).reshape(part.shape)
        else:
            pair = torch.complex(part[..., :rot // 2].contiguous(),
                                 part[..., rot // 2:].contiguous())
            pair = pair * turn[:, None]
            new = torch.cat([pair.real, pair.imag], -1)
        x[lo:lo + n, :Hq + Hkv, :rot] = new
        slot = s["table"][b].long()[pos // page] * page + pos % page
        K.view(-1, Hkv, case["D"])[slot] = x[lo:lo + n, Hq:Hq + Hkv]
        V.view(-1, Hkv, case["D"])[slot] = x[lo:lo + n, Hq + Hkv:]
    return {"q": x[:, :Hq], "k_cache": K, "v_cache": V}


def _exact_attend(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
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
        page = s["table"][b, :-(-kv // case["page"])].long()
        k = s["k_cache"][page].flatten(0, 1)[:kv]
        v = s["v_cache"][page].flatten(0, 1)[:kv]
        for h in range(Hq):
            w = torch.einsum("id,jd->ij", s["q"][lo:lo + n, h].double(),
                             k[:, h // G].double()) / math.sqrt(D)
            w.masked_fill_(~see, -math.inf)
            lse[lo:lo + n, h] = torch.logsumexp(w, 1)
            out[lo:lo + n, h] = torch.einsum(
                "ij,jd->id", torch.softmax(w, 1), v[:, h // G].double())
        lo += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_distill(case, seed):
    s = prepare(case, seed)
    T, part = case["T"], case["part"]
    out = {}
    loss, lses, grads = [], [], []
    for lo in range(0, case["N"], 256):
        z = s["student"][lo:lo + 256].double() / T
        ids = s["id"][lo:lo + 256].long()
        if s["teacher_lse"] is None:
            logp = torch.log_softmax(s["logit"][lo:lo + 256].double() / T, 1)
        else:
            logp = s["logit"][lo:lo + 256].double() / T \
                - s["teacher_lse"][lo:lo + 256, None].double()
        lse = torch.logsumexp(z, 1) if part != "backward" \
            else s["lse"][lo:lo + 256].double()
        logq = z - lse[:, None]
        loss.append((logp.exp() * (logp - logq.gather(1, ids))).sum(1))
        lses.append(lse)
        if part != "forward":
            target = torch.zeros_like(z).scatter_add_(1, ids, logp.exp())
            d = logp.exp().sum(1, keepdim=True) * logq.exp() - target
            grads.append(d * s["weight"][lo:lo + 256, None].double() / T)
    if part != "backward":
        out["loss"], out["lse"] = torch.cat(loss), torch.cat(lses)
    if part != "forward":
        out["grad"] = torch.cat(grads)
    return out
