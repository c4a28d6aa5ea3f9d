"""sd_distill_topk, _backward and _step against the 64-bit formula, under
bounds derived from the roundings (tests/operators_ref.py), and the gradient
against differences of the library's own loss."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_temperature_gb300 import api
from tests import operators_ref as ref
from tests.test_gpu_canaries import GuardedTorch

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


def make(N, V, K, dtype, T, seed, full=False, stride=None):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(N, V, generator=g) * 3
    z = torch.empty(N, stride or V, dtype=dtype)
    z[:, :V] = (t + torch.randn(N, V, generator=g)).to(dtype)
    if stride:
        z[:, V:] = float("nan")
    top = t.topk(K, 1)
    tl = (t / T).double().logsumexp(1).float() if full else None
    w = torch.rand(N, generator=g) * 2 - 0.5
    return z, top.values.contiguous(), top.indices.to(torch.int32), tl, w


def check(z, V, logit, ids, tl, w, T, *, status=0, out=None):
    """All three calls on the same rows; returns the step's results."""
    zc = z.cuda()[:, :V]
    a = (logit.cuda(), ids.cuda())
    kw = dict(teacher_lse=None if tl is None else tl.cuda())
    st = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3)]
    f = api.distill_topk(zc, *a, T, status=st[0], **kw)
    g = api.distill_topk_backward(zc, f["lse"], *a, w.cuda(), T,
                                  status=st[1], **kw)
    s = api.distill_topk_step(zc, *a, w.cuda(), T, status=st[2], **kw)
    torch.cuda.synchronize()
    assert [int(x.item()) for x in st] == [status] * 3
    r = ref.distill(ref.f64(z)[:, :V], ref.f64(logit), ids.numpy(), T,
                    None if tl is None else ref.f64(tl), ref.f64(w))
    u = ref.U[z.dtype]
    gtol = r["grad_tol"] * (1 + u) + u * np.abs(r["grad"]) * 1.01 + 1e-38
    for loss, lse, grad in ((f["loss"], f["lse"], g),
                            (s["loss"], s["lse"], s["grad"])):
        for got, name in ((loss, "loss"), (lse, "lse")):
            x, y = ref.f64(got), r[name]
            fine = np.isfinite(y)
            assert (x[~fine] == y[~fine]).all(), name
            assert (np.abs(x - y)[fine] <= r[name + "_tol"][fine]).all(), \
                (name, np.abs(x - y)[fine].max())
        assert grad.dtype == z.dtype
        assert (np.abs(ref.f64(grad) - r["grad"]) <= gtol).all()
    return s


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("N,V,K,T", [
    (1, 1, 1, 1.0), (1, 7, 7, 0.7), (3, 1000, 5, 1.0), (5, 1001, 16, 0.7),
    (2, 32000, 64, 2.0), (33, 4096, 50, 1.0), (2, 152064, 32, 1.0),
    (200, 515, 3, 0.5), (1, 128256, 256, 1.0), (700, 2048, 8, 1.0),
    (90, 128256, 20, 1.0), (170, 75001, 7, 0.7), (160, 9, 9, 1.0)])
def test_sizes(dtype, full, N, V, K, T):
    z, lg, ids, tl, w = make(N, V, K, dtype, T, seed=N + V, full=full)
    check(z, V, lg, ids, tl, w, T)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V,stride", [(1000, 1008), (1000, 1001),
                                      (999, 1024), (4096, 4097)])
def test_strided_rows(dtype, V, stride):
    """Padded rows (NaN past V) and rows that start off 16 bytes."""
    z, lg, ids, tl, w = make(9, V, 8, dtype, 1.0, seed=V, stride=stride)
    check(z, V, lg, ids, tl, w, 1.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,V", [(4, 2000), (3, 152064), (2, 1003)])
def test_entries_that_count_for_nothing_and_repeats(dtype, N, V):
    """Padding, logits of -inf (also where the student has -inf), ids past
    the vocabulary, the same id several times, a row without entries."""
    z, lg, ids, tl, w = make(N, V, 12, dtype, 1.0, seed=V)
    ids[:, 1] = -1
    ids[:, 2] = -7
    ids[:, 5] = ids[:, 4]
    ids[:, 9] = ids[:, 4]
    lg[:, 6] = -float("inf")
    z[torch.arange(N), ids[:, 6].long()] = -float("inf")
    lg[0, 1] = float("nan")  # padding: not looked at
    ids[-1] = -1
    check(z, V, lg, ids, None, w, 1.0)
    ids[0, 3] = V
    check(z, V, lg, ids, None, w, 1.0, status=api.DEV_BAD_TOKEN)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [1000, 1001, 64128])
def test_masked_students(dtype, V):
    """Student logits of -inf and of the type's lowest value; a teacher's
    token the student masks makes the loss infinite and the gradient
    finite."""
    z, lg, ids, tl, w = make(4, V, 6, dtype, 1.0, seed=V)
    z[0, : V // 2] = -float("inf")
    z[1, ::3] = torch.finfo(dtype).min
    z[2] = -float("inf")
    z[2, V - 1] = 0.5
    ids[0] = torch.arange(V - 6, V, dtype=torch.int32)
    ids[1] = torch.tensor([1, 2, 4, 5, 7, 8], dtype=torch.int32)
    ids[2] = V - 1
    check(z, V, lg, ids, None, w, 1.0)
    ids[3, 0] = 5
    z[3, 5] = -float("inf")
    s = check(z, V, lg, ids, None, w, 1.0)
    assert s["loss"][3].item() == float("inf")
    assert bool(torch.isfinite(s["grad"][3]).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [1000, 1001, 64128])
def test_unusable_rows(dtype, V):
    """NaN, +inf or only -inf in the student, NaN in the teacher: that row is
    NaN and the bit is set; the others are as ever; a row of weight 0 has a
    gradient of 0 all the same."""
    z, lg, ids, tl, w = make(7, V, 6, dtype, 1.0, seed=V)
    w[:] = 0.5
    clean = {k: v.clone() for k, v in check(z, V, lg, ids, None, w,
                                            1.0).items()}
    z[0, 3] = float("nan")
    z[1, V - 1] = float("inf")
    z[2] = -float("inf")
    lg[3, 2] = float("nan")
    z[5, 7] = float("nan")
    w[5] = 0.0
    a = (lg.cuda(), ids.cuda())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = api.distill_topk(z.cuda(), *a, 1.0, status=st)
    s = api.distill_topk_step(z.cuda(), *a, w.cuda(), 1.0)
    g = api.distill_topk_backward(z.cuda(), f["lse"], *a, w.cuda(), 1.0)
    torch.cuda.synchronize()
    assert int(st.item()) == api.DEV_NONFINITE
    bad, good = [0, 1, 2, 3, 5], [4, 6]
    for r in (f, s):
        assert bool(torch.isnan(r["loss"][bad]).all())
        assert bool(torch.isnan(r["lse"][bad]).all())
        for k in ("loss", "lse"):
            assert torch.equal(r[k][good], clean[k][good])
    for grad in (g, s["grad"]):
        assert bool(torch.isnan(grad[:4]).all())
        assert bool((grad[5] == 0).all())
    assert torch.equal(s["grad"][good], clean["grad"][good])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [1000, 1001, 152064])
def test_in_place(dtype, V):
    z, lg, ids, tl, w = make(5, V, 9, dtype, 1.0, seed=V)
    want = check(z, V, lg, ids, tl, w, 1.0)["grad"]
    a = (lg.cuda(), ids.cuda())
    zc = z.cuda()
    got = api.distill_topk_step(zc, *a, w.cuda(), 1.0, out=zc)
    assert torch.equal(zc, want) and got["grad"] is zc
    zc = z.cuda()
    lse = api.distill_topk(zc, *a, 1.0)["lse"]
    b = api.distill_topk_backward(zc, lse, *a, w.cuda(), 1.0)
    api.distill_topk_backward(zc, lse, *a, w.cuda(), 1.0, out=zc)
    assert torch.equal(zc, b)


def test_gradient_against_differences_of_the_loss():
    """Central differences of the GPU's own loss.  With step h the formula's
    error is at most h^2 / 6 |L'''| <= h^2 / 6 (T = 1, P = 1), the loss's own
    bound counts 1 / h."""
    V, K, h = 24, 4, 2.0 ** -4
    z, lg, ids, tl, w = make(1, V, K, F32, 1.0, seed=2)
    # one row per shifted column, both ways
    zz = z.repeat(2 * V, 1)
    for j in range(V):
        zz[j, j] += h
        zz[V + j, j] -= h
    a = lambda m: (lg.repeat(m, 1).cuda(), ids.repeat(m, 1).cuda())
    loss = ref.f64(api.distill_topk(zz.cuda(), *a(2 * V), 1.0)["loss"])
    s = api.distill_topk_step(z.cuda(), *a(1),
                              torch.ones(1, device="cuda"), 1.0)
    r = ref.distill(ref.f64(zz), ref.f64(lg.repeat(2 * V, 1)),
                    ids.repeat(2 * V, 1).numpy(), 1.0)
    d = (loss[:V] - loss[V:]) / (2 * h)
    tol = h * h / 6 + r["loss_tol"].max() / h
    assert (np.abs(ref.f64(s["grad"])[0] - d) <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V,stride", [(1000, 1000), (999, 1001),
                                      (152064, 152064)])
def test_no_write_outside_the_buffers(monkeypatch, dtype, V, stride):
    guard = GuardedTorch()
    monkeypatch.setattr(api, "torch", guard)
    z, lg, ids, tl, w = make(3, V, 9, dtype, 1.0, seed=V, stride=stride)
    a = (lg.cuda(), ids.cuda())
    zc = z.cuda()[:, :V]
    f = api.distill_topk(zc, *a, 1.0)
    api.distill_topk_backward(zc, f["lse"], *a, w.cuda(), 1.0)
    api.distill_topk_step(zc, *a, w.cuda(), 1.0)
    assert guard.check() == 6


def test_from_the_fan_out():
    """The teacher's entries as sd_fanout_topk returns them."""
    N, V, F = 6, 5000, 16
    g = torch.Generator().manual_seed(4)
    target = torch.randn(N, 1, V, generator=g).cuda() * 3
    student = torch.randn(N, V, generator=g).cuda()
    fan = api.fanout_topk(target, [F], want_logit=True)
    s = api.distill_topk_step(student, fan["logit"].contiguous(),
                              fan["tokens"].contiguous(),
                              torch.full((N,), 1 / N, device="cuda"))
    r = ref.distill(ref.f64(student), ref.f64(fan["logit"]),
                    fan["tokens"].cpu().numpy(), 1.0, None,
                    np.full(N, 1 / N))
    assert (np.abs(ref.f64(s["loss"]) - r["loss"]) <= r["loss_tol"]).all()
    tol = r["grad_tol"] + 2 * ref.U32 * np.abs(r["grad"]) + 1e-38
    assert (np.abs(ref.f64(s["grad"]) - r["grad"]) <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V,stride", [(20000, 20000), (90001, 90001),
                                      (74000, 74008)])
def test_step_over_many_rows(dtype, V, stride):
    """Rows enough that every SM takes several, weights of 0 and unusable rows
    among them: the step's gradient is the backward call's with the step's own
    log-sum-exp, and in place it is the same bits."""
    N, K = 400, 12
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(N, stride, generator=g, device="cuda").to(dtype)[:, :V]
    top = torch.randn(N, V, generator=g, device="cuda").topk(K, 1)
    a = (top.values.contiguous(), top.indices.to(torch.int32))
    w = torch.rand(N, generator=g, device="cuda")
    w[::7] = 0
    z[5, 3] = float("nan")
    z[14, 9] = float("inf")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = api.distill_topk_step(z, *a, w, 0.9, status=st)
    f = api.distill_topk(z, *a, 0.9)
    b = api.distill_topk_backward(z, s["lse"], *a, w, 0.9)
    torch.cuda.synchronize()
    assert int(st.item()) == api.DEV_NONFINITE
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[[5, 14]] = True
    for k in ("loss", "lse"):
        assert bool((torch.isnan(s[k]) == bad).all())
        x, y = s[k][~bad], f[k][~bad]
        # the two sum in another order
        assert bool(((x - y).abs() <= 1e-4 * (1 + y.abs())).all()), k
    assert bool((s["grad"][w == 0] == 0).all())
    assert bool(torch.isnan(s["grad"][5]).all())
    rows = (~bad) & (w != 0)
    x, y = s["grad"][rows].float(), b[rows].float()
    tol = 2 * ref.U[dtype] + 1e-5
    assert bool(((x - y).abs() <= tol * y.abs() + 1e-12).all())
    again = api.distill_topk_step(z, *a, w, 0.9, out=z)["grad"]
    assert again is z
    assert torch.equal(torch.nan_to_num(z), torch.nan_to_num(s["grad"]))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,V", [(4, 1000), (4, 64129), (200, 5000)])
@pytest.mark.parametrize("mask,T", [(-2e38, 0.7), (-2e38, 2.0), (-1e38, 0.3),
                                    (-2.9e38, 1.0), (-1e37, 0.7),
                                    (-1e30, 1.0), (-1e10, 0.7), (-9e8, 0.7),
                                    (-1e4, 0.7)])
def test_finite_masks(dtype, N, V, mask, T):
    """A mask far below every logit, finite or -inf, gives the same bits: the
    first half of a row, all but its end, every other column."""
    z, lg, ids, tl, w = make(N, V, 6, dtype, T, seed=V)
    hide = torch.zeros(N, V, dtype=torch.bool)
    hide[0, :V // 2] = True
    hide[1, :V - 6] = True
    hide[2, ::2] = True
    ids[:] = torch.arange(V - 11, V + 1, 2, dtype=torch.int32)
    ids[1] = torch.arange(V - 6, V, dtype=torch.int32)
    ids[2] = torch.arange(1, 12, 2, dtype=torch.int32)
    ids[ids >= V] = -1
    a = (lg.cuda(), ids.cuda())
    got = []
    for m in (mask, -float("inf")):
        zm = z.masked_fill(hide, m).cuda()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        f = api.distill_topk(zm, *a, T, status=st)
        s = api.distill_topk_step(zm, *a, w.cuda(), T, status=st)
        g = api.distill_topk_backward(zm, f["lse"], *a, w.cuda(), T,
                                      status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        got.append((f["loss"], f["lse"], s["loss"], s["lse"], s["grad"], g))
    for x, y in zip(*got):
        assert bool(torch.isfinite(x).all()) and torch.equal(x, y)


@pytest.mark.parametrize("N", [40, 200])
@pytest.mark.parametrize("stride", [152064, 152065])
def test_step_on_rows_longer_than_the_chip_keeps(N, stride):
    """fp32 rows of 152064 columns, too long for eight CTAs to keep: with 40
    rows clusters of four, with 200 single CTAs, each reads what it did not
    keep a second time, in place from a row that it is overwriting; aligned
    and off 16 bytes.  Against the formula in 64 bits (torch's log-softmax),
    under the bounds of tests/operators_ref.py."""
    V, K, T = 152064, 24, 0.9
    g = torch.Generator(device="cuda").manual_seed(N)
    z = torch.randn(N, stride, generator=g, device="cuda")[:, :V] * 3
    z = torch.empty(N, stride, device="cuda")[:, :V].copy_(z)
    top = torch.randn(N, V, generator=g, device="cuda").topk(K, 1)
    a = (top.values.contiguous(), top.indices.to(torch.int32))
    w = torch.rand(N, generator=g, device="cuda")
    w[::9] = 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = api.distill_topk_step(z, *a, w, T, status=st)
    f = api.distill_topk(z, *a, T, status=st)
    back = api.distill_topk_backward(z, s["lse"], *a, w, T, status=st)
    assert int(st.item()) == 0
    u = ref.U32
    for lo in range(0, N, 20):
        r = slice(lo, lo + 20)
        x = z[r].double() / T
        lse = torch.logsumexp(x, 1)
        logp = torch.log_softmax(top.values[r].double() / T, 1)
        logq = x - lse[:, None]
        p, size = logp.exp(), x.abs().amax(1)
        loss = (p * (logp - logq.gather(1, top.indices[r]))).sum(1)
        # as operators_ref.distill, with its largest terms for all
        lse_tol = (V / 256 + 64) * u + 8 * u * (1 + size + lse.abs())
        tsize = 2 * top.values[r].double().abs().amax(1) / T + 4
        rel = 16 * u * (1 + tsize) + 256 * u
        far = logq.abs().amax(1)
        loss_tol = lse_tol + rel * (1 + tsize + far) + \
            8 * u * (size + lse.abs())
        for got in (s, f):
            assert bool(((got["lse"][r] - lse).abs() <= lse_tol).all())
            assert bool(((got["loss"][r] - loss).abs() <= loss_tol).all())
        q = logq.exp()
        pk = torch.zeros_like(q).scatter_add_(1, top.indices[r], p)
        c = (w[r].double() / T)[:, None]
        tol = c * (q * (rel + lse_tol)[:, None] + q * 16 * u * (1 + logq.abs())
                   + pk * (rel[:, None] + 64 * u))
        for got in (s["grad"], back):
            d = (got[r].double() - c * (q - pk)).abs()
            assert bool((d <= tol * 1.01 + u * (c * (q - pk)).abs()
                         + 1e-38).all())
    want = s["grad"].clone()
    assert api.distill_topk_step(z, *a, w, T, out=z)["grad"] is z
    assert torch.equal(z, want)
