"""Distillation from a teacher's top logits vs the fp64 oracle.

Bounds: a thread adds at most V / 256 + 64 terms and joins of relative error 2^-23 each (the
exponential's two steps and its argument's rounding, whose share d 2^-24 of a term e^-d stays
below 2^-25), so lse is off by (V / 256 + 64) 2^-23 plus its own rounding, and q by the same
relative amount plus the rounding of its exponent. log p is rounded to fp32 (2^-24 |log p|).
"""
import math

import numpy as np
import pytest
import torch

from oracle import kronq_oracle as O

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {torch.float32: U32, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def K():
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import kronq
    kronq.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kronq.kronq_device_check()
    return kronq


def np64(t):
    return t.detach().cpu().double().numpy()


def inputs(n, v, k, dtype, seed, ragged=False, pad=0):
    """Student logits near a teacher's list; `pad` extra columns of row stride."""
    r = np.random.default_rng(seed)
    z = r.normal(0, 2, (n, v))
    ids = np.stack([r.permutation(v)[:k] if k <= v else r.integers(0, v, k) for _ in range(n)])
    t = 6.0 - 1.5 * np.log1p(np.arange(k))[None, :] + 0.3 * r.normal(0, 1, (n, k))
    for row in range(n):
        z[row, ids[row]] = t[row] + 0.5 * r.normal(0, 1, k)
    if ragged:
        keep = r.integers(0, k + 1, n)
        ids = np.where(np.arange(k)[None, :] < keep[:, None], ids, -1)
        ids[0] = -1                                    # a row without any entry
    zt = torch.zeros(n, v + pad, dtype=dtype, device="cuda")[:, :v]
    zt.copy_(torch.from_numpy(z))
    return (zt, torch.from_numpy(ids.astype(np.int32)).cuda(),
            torch.from_numpy(t).to(dtype).cuda())


def check(z, ids, t, tau, top_lse, w, loss, lse, dz, given_lse=None):
    wl, wlse, wg = O.distill(np64(z), ids.cpu().numpy(), np64(t), tau,
                             None if top_lse is None else np64(top_lse),
                             None if w is None else np64(w),
                             None if given_lse is None else np64(given_lse))
    n, v = z.shape
    weight = np.ones(n) if w is None else np64(w)
    stat = (v / 256 + 64) * 2.0 ** -23
    zm = np.abs(np64(z)[np.isfinite(np64(z))]).max(initial=0.0) / tau
    tm = np.abs(np64(t)[np.isfinite(np64(t))]).max(initial=0.0) / tau + zm + 20
    if lse is not None:
        fin = np.isfinite(wlse)
        np.testing.assert_array_equal(np64(lse)[~fin], wlse[~fin])
        assert (np.abs(np64(lse) - wlse)[fin] <= stat + 2 * U32 * np.abs(wlse[fin])).all()
    if loss is not None:
        fin = np.isfinite(wl)
        np.testing.assert_array_equal(np64(loss)[~fin], wl[~fin])
        # p's relative error (its exponent's rounding) times each term, and lse's
        tol = np.abs(weight) * tau * tau * (stat + 4 * tm * U32 * (1 + tm)) + 2 * U32 * np.abs(wl)
        assert (np.abs(np64(loss) - wl)[fin] <= tol[fin]).all()
    if dz is not None:
        got = np64(dz)
        # P q and p are each below q + |gradient / (w tau)|, P <= 1 + 2^-20
        u = np64(z) / tau
        with np.errstate(invalid="ignore", over="ignore"):
            q = np.where(np.isfinite(wlse)[:, None], np.exp(u - wlse[:, None]), 0.0)
        unit = np.where(weight == 0, 1.0, np.abs(weight) * tau)[:, None]
        part = unit * (2 * q + np.abs(wg / unit))
        tol = (stat + 6 * tm * U32) * part + HALF[dz.dtype] * np.abs(wg) + 1e-38
        bad = ~(np.abs(got - wg) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], wg[bad][:4])


def run(K, z, ids, t, tau=1.0, top_lse=None, w=None, ddtype=None, grad=True, dz=None):
    n, v = z.shape
    loss = torch.full((n,), float("nan"), device="cuda")
    lse = torch.full((n,), float("nan"), device="cuda")
    if grad and dz is None:
        dz = torch.full((n, v), float("nan"), dtype=ddtype or z.dtype, device="cuda")
    K.kronq_distill(z, ids, t, loss, lse, dlogits=dz, top_lse=top_lse, row_weight=w,
                    temperature=tau)
    torch.cuda.synchronize()
    return loss, lse, dz


SIZES = [(1, 1, 1), (2, 5, 3), (3, 31, 8), (1, 1000, 1), (5, 1025, 33), (4, 4099, 64), (2, 32000, 128),
         (3, 50001, 20), (1, 128256, 1024), (2, 300, 300), (9, 8200, 600)]


@pytest.mark.parametrize("n,v,k", SIZES)
@pytest.mark.parametrize("dtype,ddtype", [(torch.bfloat16, torch.bfloat16),
                                          (torch.float32, torch.float32),
                                          (torch.bfloat16, torch.float32),
                                          (torch.float32, torch.bfloat16)])
def test_loss_and_gradient(K, n, v, k, dtype, ddtype):
    z, ids, t = inputs(n, v, k, dtype, 11 * n + v + k)
    w = torch.rand(n, device="cuda") + 0.25
    for tau, mass in ((1.0, False), (2.5, True)):
        top_lse = torch.logsumexp(t.double() / tau, 1).float() + 0.1 if mass else None
        loss, lse, dz = run(K, z, ids, t, tau, top_lse, w, ddtype)
        check(z, ids, t, tau, top_lse, w, loss, lse, dz)
        only, lse2, _ = run(K, z, ids, t, tau, top_lse, w, grad=False)
        check(z, ids, t, tau, top_lse, w, only, lse2, None)
        back = torch.full((n, v), float("nan"), dtype=ddtype, device="cuda")
        K.kronq_distill_backward(z, ids, t, lse, w, back, top_lse=top_lse, temperature=tau)
        torch.cuda.synchronize()
        check(z, ids, t, tau, top_lse, w, None, None, back, given_lse=lse)


@pytest.mark.parametrize("n", [7, 160, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ragged_lists_and_weights(K, n, dtype):
    z, ids, t = inputs(n, 1537, 24, dtype, n, ragged=True, pad=3)
    t[ids < 0] = float("nan")                          # absent logits are not looked at
    w = torch.rand(n, device="cuda")
    w[1::3] = 0.0
    z[1::3, 5] = float("nan")                          # nor is anything of a row of weight 0
    loss, lse, dz = run(K, z, ids, t, 1.3, None, w)
    assert bool((loss[1::3] == 0).all()) and bool((dz[1::3] == 0).all())
    assert float(loss[0]) == 0.0 and bool((dz[0] == 0).all())
    keep = torch.ones(n, dtype=torch.bool)
    keep[1::3] = False
    keep = keep.cuda()
    check(z[keep], ids[keep], torch.nan_to_num(t[keep]), 1.3, None, w[keep], loss[keep], lse[keep],
          dz[keep])


def test_masked_entries(K):
    n, v, k = 6, 2000, 16
    z, ids, t = inputs(n, v, k, torch.float32, 5)
    lowest = torch.finfo(torch.float32).min
    free = torch.ones(n, v, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), False)
    z[0][free[0]] = float("-inf")                      # all but the listed entries
    z[1][free[1]] = lowest
    z[2, ids[2, 3].long()] = float("-inf")             # a listed entry: infinite loss
    z[3] = float("-inf")                               # nothing left
    z[4] = lowest                                      # the same as a uniform row
    t[5, 2:] = float("-inf")                           # listed with no probability
    loss, lse, dz = run(K, z, ids, t)
    assert math.isinf(float(loss[2])) and math.isinf(float(loss[3])) and float(loss[2]) > 0
    rows = [0, 1, 2, 5]
    check(z[rows], ids[rows], t[rows], 1.0, None, None, loss[rows], lse[rows], dz[rows])
    # row 3: q = 0, so the gradient is -p alone
    p = torch.softmax(t[3].double(), 0)
    want = torch.zeros(v, dtype=torch.float64, device="cuda").scatter_(0, ids[3].long(), -p)
    assert float((dz[3].double() - want).abs().max()) <= 64 * U32
    q = torch.full((v,), 1.0 / v, dtype=torch.float64, device="cuda")
    p = torch.softmax(t[4].double(), 0)
    assert float((dz[4].double() - q.scatter_add(0, ids[4].long(), -p)).abs().max()) <= 64 * U32
    # the same rows through the backward pass
    back = torch.empty_like(dz)
    K.kronq_distill_backward(z, ids, t, lse, torch.ones(n, device="cuda"), back)
    for r in (0, 1, 2, 3, 5):
        assert float((back[r] - dz[r]).abs().max()) <= 256 * U32


def test_bf16_mask_of_the_lowest_value(K):
    z, ids, t = inputs(3, 4096, 8, torch.bfloat16, 8)
    z[:, 1000:] = torch.finfo(torch.bfloat16).min
    ids = (ids % 1000).to(torch.int32)                 # ids may now repeat
    for tau in (0.5, 1.0):
        loss, lse, dz = run(K, z, ids, t, tau)
        check(z, ids, t, tau, None, None, loss, lse, dz)


def test_repeated_and_outside_ids(K):
    v = 900
    z, ids, t = inputs(4, v, 40, torch.float32, 21)
    ids[0] = 17                                        # one entry forty times
    ids[1, 20:] = ids[1, :20]
    ids[2, ::3] = v                                    # outside: absent
    ids[2, 1] = 2 ** 31 - 1
    ids[2, 2] = -(2 ** 31)
    ids[3, 5] = v - 1
    top_lse = torch.logsumexp(t, 1)
    for tl in (None, top_lse):
        loss, lse, dz = run(K, z, ids, t, 1.0, tl)
        check(z, ids, t, 1.0, tl, None, loss, lse, dz)


def test_in_place_and_no_list(K):
    for dtype in (torch.bfloat16, torch.float32):
        z, ids, t = inputs(5, 3001, 12, dtype, 3, pad=7)
        loss, lse, dz = run(K, z, ids, t, 0.7)
        zc = torch.empty(5, 3008, dtype=dtype, device="cuda")[:, :3001]
        zc.copy_(z)
        loss2, lse2, _ = run(K, zc, ids, t, 0.7, dz=zc)
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
        assert torch.equal(dz, zc)
        zc.copy_(z)
        back = torch.empty_like(dz)
        one = torch.ones(5, device="cuda")
        K.kronq_distill_backward(z, ids, t, lse, one, back, temperature=0.7)
        K.kronq_distill_backward(zc, ids, t, lse, one, zc, temperature=0.7)
        torch.cuda.synchronize()
        assert torch.equal(back, zc)
    loss, lse, dz = run(K, z, ids[:, :0], t[:, :0])
    assert bool((loss == 0).all()) and bool((dz == 0).all())
    K.kronq_distill(z[:0], ids[:0], t[:0], loss[:0])   # no tokens


def test_rows_do_not_depend_on_the_batch(K):
    """One row alone, in a small batch and in a large one: however rows are split over the GPU, the
    bits of a batch repeat, and rows of different batches agree to rounding."""
    z, ids, t = inputs(400, 20011, 30, torch.bfloat16, 77)
    loss, lse, dz = run(K, z, ids, t, 1.5)
    again = run(K, z, ids, t, 1.5)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1]) and torch.equal(dz, again[2])
    for rows in (slice(0, 1), slice(3, 20), slice(100, 300)):
        l1, s1, d1 = run(K, z[rows], ids[rows], t[rows], 1.5)
        check(z[rows], ids[rows], t[rows], 1.5, None, None, l1, s1, d1)


def test_gradient_against_differences(K):
    v, k, tau = 60, 7, 1.7
    z, ids, t = inputs(2, v, k, torch.float32, 99)
    ids[1, 4:] = -1
    w = torch.tensor([0.8, 1.9], device="cuda")
    _, _, dz = run(K, z, ids, t, tau, None, w)
    h = 1e-5
    base = np64(z)
    for col in list(range(0, v, 7)) + [int(ids[0, 0]), int(ids[1, 1])]:
        for row in range(2):
            up, dn = base.copy(), base.copy()
            up[row, col] += h
            dn[row, col] -= h
            lu, _, _ = O.distill(up, ids.cpu().numpy(), np64(t), tau, None, np64(w))
            ld, _, _ = O.distill(dn, ids.cpu().numpy(), np64(t), tau, None, np64(w))
            # the difference quotient is off by h^2 and 1e-16 / h; the gradient by its fp32 parts
            assert abs((lu - ld)[row] / (2 * h) - float(dz[row, col])) <= 1e-5


def test_captured_and_replayed_on_a_side_stream(K):
    z, ids, t = inputs(70, 9001, 16, torch.bfloat16, 31)
    loss, lse, dz = run(K, z, ids, t)
    z2 = z.clone()
    l2, s2, d2 = torch.zeros_like(loss), torch.zeros_like(lse), torch.zeros_like(dz)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            K.kronq_distill(z2, ids, t, l2, s2, dlogits=d2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(d2, dz) and torch.equal(l2, loss)
    z2.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(z2, ids, t, 1.0, None, None, l2, s2, d2)
    del g


def test_the_head_gradient_feeds_the_statistics(K):
    """Loss -> dlogits -> kronq_accumulate: H_G of an output head, vs fp64 from the oracle."""
    n, v, k = 256, 504, 12
    z, ids, t = inputs(n, v, k, torch.bfloat16, 123)
    w = torch.full((n,), 1.0 / n, device="cuda")
    dz = torch.empty(n, v, dtype=torch.bfloat16, device="cuda")
    loss = torch.empty(n, device="cuda")
    K.kronq_distill(z, ids, t, loss, dlogits=dz, row_weight=w)
    hg = torch.zeros(v, v, device="cuda")
    K.kronq_accumulate(g=dz, hg_sum=hg)
    torch.cuda.synchronize()
    _, _, g = O.distill(np64(z), ids.cpu().numpy(), np64(t), 1.0, None, np64(w))
    want = g.T @ g
    # each factor is a bf16 rounding (2^-8) off: twice that in a product, in the norm
    assert np.linalg.norm(np64(hg) - want) <= 2.0 * 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.parametrize("v,k,dtype", [(128256, 128, torch.bfloat16), (40001, 300, torch.bfloat16),
                                       (70000, 7, torch.float32), (300000, 64, torch.bfloat16),
                                       (20000, 1024, torch.float32)])
def test_many_long_rows(K, v, k, dtype):
    """Enough rows that every CTA takes several in turn; each row against fp64 on the device."""
    n, tau = 1400, 1.3
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    z = torch.empty(n, v, dtype=dtype, device="cuda")
    for r in range(0, n, 200):
        z[r:r + 200] = 2.0 * torch.randn(200, v, generator=g, device="cuda")
    start = torch.randint(0, v, (n, 1), generator=g, device="cuda")
    ids = ((start + torch.arange(k, device="cuda") * (v // k - 1)) % v).to(torch.int32)
    ids[5::9, k // 2:] = -1
    if k > 2:
        ids[7::11, 2] = ids[7::11, 0]                  # listed twice
    t = (9.0 - torch.arange(k, device="cuda") / k * 4).expand(n, k).to(dtype).contiguous()
    z.scatter_(1, ids.clamp(min=0).long(), t)
    w = torch.rand(n, generator=g, device="cuda")
    first = None
    for _ in range(3):
        loss, lse, dz = run(K, z, ids, t, tau, None, w)
        if first is None:
            first = (loss, lse, dz)
        else:
            assert all(torch.equal(a, b) for a, b in zip(first, (loss, lse, dz)))
    stat = (v / 256 + 64) * 2.0 ** -23
    for r in range(0, n, 50):
        rows = slice(r, r + 50)
        u = z[rows].double() / tau
        l = torch.logsumexp(u, 1)
        there = ids[rows] >= 0
        at = ids[rows].clamp(min=0).long()
        logp = torch.log_softmax((t[rows].double() / tau).masked_fill(~there, -math.inf), 1)
        p = logp.exp()
        wl = w[rows].double() * tau * tau * (p * (logp - u.gather(1, at) + l[:, None])).masked_fill(
            ~there, 0.0).sum(1)
        q = (u - l[:, None]).exp()
        unit = w[rows].double()[:, None] * tau
        wg = unit * (q - torch.zeros_like(q).scatter_add_(1, at, p))
        assert bool(((lse[rows].double() - l).abs() <= stat + 2 * U32 * l.abs()).all())
        assert bool(((loss[rows].double() - wl).abs() <= tau * tau * (stat + 4e3 * U32)
                     + 2 * U32 * wl.abs()).all())
        tol = (stat + 6 * 40 * U32) * (2 * unit * q + wg.abs()) + HALF[dtype] * wg.abs() + 1e-38
        assert bool(((dz[rows].double() - wg).abs() <= tol).all())
    assert K.kronq_device_error() == 0


@pytest.mark.parametrize("n,v,k,dtype", [(3, 700, 300, torch.float32), (5, 50000, 1024, torch.bfloat16),
                                         (320, 40000, 200, torch.bfloat16), (310, 40000, 1000, torch.float32)])
def test_lists_that_repeat_their_ids(K, n, v, k, dtype):
    """Many entries on few ids, one id for all, pads of -inf on one id: sums over the repeats."""
    z, ids, t = inputs(n, v, k, dtype, 55)
    r = np.random.default_rng(8)
    ids.copy_(torch.from_numpy(r.integers(0, 5 * k, (n, k)).astype(np.int32) % v))
    ids[0] = v - 1
    ids[1, k // 3:] = 0
    t[1, k // 3:] = float("-inf")
    ids[2] = torch.arange(k, device="cuda", dtype=torch.int32).flip(0) // 2
    w = torch.from_numpy(r.uniform(0.5, 2, n).astype(np.float32)).cuda()
    loss, lse, dz = run(K, z, ids, t, 1.1, None, w)
    again = run(K, z, ids, t, 1.1, None, w)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1]) and torch.equal(dz, again[2])
    some = torch.tensor([0, 1, 2] + list(range(3, n, 37)))
    check(z[some], ids[some], t[some], 1.1, None, w[some], loss[some], lse[some], dz[some])
    back = torch.empty_like(dz)
    K.kronq_distill_backward(z, ids, t, lse, w, back, temperature=1.1)
    torch.cuda.synchronize()
    check(z[some], ids[some], t[some], 1.1, None, w[some], None, None, back[some],
          given_lse=lse[some])
    assert K.kronq_device_error() == 0
