"""Distillation on long rows: many of them (clusters that take rows in turn, at 1, 2, 4 and 8 CTAs a
row), and few (rows read twice), vs the definition in fp64 on the device.

Bounds: a thread adds at most V / 256 + 64 terms and joins of relative error 2^-23 each, so sums, and
with them q, are off by STAT = (V / 256 + 64) 2^-23 relative. An exponent is one FMA against a rounded
reference; the reference's rounding is the same number in the sum and in q, so only the exponent's own
rounding is left, 2^-24 of its size, whatever z / tau is.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {torch.float32: U32, torch.bfloat16: 2.0 ** -8}
BF16, F32 = torch.bfloat16, torch.float32

# rows, vocabulary, type: 1, 2, 4 and 8 CTAs a row by the rule of distill.cu; every vocabulary is odd, so
# that rows begin and end beside their 16-byte vectors
RING = [(600, 20011, BF16), (300, 50257, BF16), (150, 128257, BF16), (80, 240001, BF16),
        (300, 20011, F32)]
# few rows, which registers hold, and too long for that
FEW = [(5, 20011, BF16), (5, 20011, F32), (3, 300001, BF16), (3, 140001, F32)]


@pytest.fixture(scope="module")
def K():
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import kronq
    kronq.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kronq.kronq_device_check()
    return kronq


def inputs(n, v, k, dtype, seed):
    """Student logits near a teacher's list of distinct entries (in fp32)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.empty(n, v, dtype=dtype, device="cuda")
    for r in range(0, n, 100):
        z[r:r + 100] = 2.0 * torch.randn(min(100, n - r), v, generator=g, device="cuda")
    start = torch.randint(0, v, (n, 1), generator=g, device="cuda")
    step = torch.randint(1, v // k, (n, 1), generator=g, device="cuda")
    ids = (start + torch.arange(k, device="cuda") * step) % v
    t = 9.0 - 4.0 * torch.rand(n, k, generator=g, device="cuda")
    z.scatter_(1, ids, (t + 0.5 * torch.randn(n, k, generator=g, device="cuda")).to(dtype))
    return z, ids.to(torch.int32), t


def run(K, z, ids, t, tau=1.0, w=None, dz=None):
    loss = torch.full((z.shape[0],), 7.0, device="cuda")
    lse = torch.full((z.shape[0],), 7.0, device="cuda")
    if dz is None:
        dz = torch.full(z.shape, 7.0, dtype=z.dtype, device="cuda")
    K.kronq_distill(z, ids, t, loss, lse, dlogits=dz, row_weight=w, temperature=tau)
    torch.cuda.synchronize()
    return loss, lse, dz


def exact(z, ids, t, tau, w=None):
    """(loss, lse, q, gradient) of rows with finite logits at their listed entries."""
    u = z.double() / tau
    lse = torch.logsumexp(u, 1)
    there = ids >= 0
    at = ids.clamp(min=0).long()
    logp = torch.log_softmax((t.double() / tau).masked_fill(~there, -math.inf), 1)
    logp = logp.masked_fill(~there, -math.inf)         # a row without entries too
    p = logp.exp()
    w = torch.ones(z.shape[0], dtype=torch.float64, device="cuda") if w is None else w.double()
    terms = p * (logp - u.gather(1, at) + lse[:, None])
    loss = w * tau * tau * terms.masked_fill(p == 0, 0.0).sum(1)
    q = (u - lse[:, None]).exp()
    unit = (w * tau)[:, None]
    grad = unit * (q * p.sum(1, keepdim=True) - torch.zeros_like(q).scatter_add_(1, at, p))
    return loss, lse, q, grad


@pytest.mark.parametrize("n,v,dtype", RING + FEW)
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_logits_that_are_not_finite(K, n, v, dtype, bad):
    """+inf or NaN anywhere in a row (its first and last elements lie beside the vectors) makes the row
    NaN, and no other."""
    k = 20
    z, ids, t = inputs(n, v, k, dtype, v)
    ok = run(K, z, ids, t)
    rows = list(range(0, n, max(1, n // 40)))
    for i, r in enumerate(rows):
        z[r, (0, v - 1, v // 2, 1, v - 2, int(ids[r, 3]))[i % 6]] = bad
    loss, lse, dz = run(K, z, ids, t)
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[rows] = True
    assert bool(loss[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert bool(dz[hit].isnan().all())
    assert torch.equal(loss[~hit], ok[0][~hit]) and torch.equal(lse[~hit], ok[1][~hit])
    assert torch.equal(dz[~hit], ok[2][~hit])
    assert K.kronq_device_error() == 0


@pytest.mark.parametrize("n,v,dtype", [c for c in RING + FEW if c[2] == F32])
@pytest.mark.parametrize("side", [0, -1])
def test_maximum_beside_the_vectors_at_a_small_temperature(K, n, v, dtype, side):
    """A row's first or last element far above the others: q there is 1 however large z / tau is."""
    tau = 2.0 ** -8
    z, ids, t = inputs(n, v, 4, dtype, v + 1)
    z.clamp_(max=20.0)
    z[:, side] = 90.0 + torch.rand(n, device="cuda")   # z / tau near 23000
    ids[:, 0] = v // 2
    ids[:, 1:] = -1                                    # p = 1 in the middle
    loss, lse, dz = run(K, z, ids, t, tau)
    _, _, q, grad = exact(z, ids, t, tau)
    stat = (v / 256 + 64) * 2.0 ** -23
    tol = (stat + U32) * tau
    assert float((dz[:, side].double() - grad[:, side]).abs().max()) <= tol


@pytest.mark.parametrize("n,v,dtype", [c for c in RING + FEW if c[2] == F32])
def test_close_logits_at_a_small_temperature(K, n, v, dtype):
    """A dozen entries within a few tau of the maximum, in different threads, z / tau near 23000: each
    thread's reference rounds by up to 2^-10, which has to cancel where the sums are joined.

    Tolerance: q and p are each off by STAT and 8 2^-23 (an exponent below 8 rounded by 2^-24 of its
    size, the exponential's two steps, p's rounding), the mass P by the same; a loss term log p - log q
    is below 10."""
    k, tau, top = 8, 2.0 ** -8, 12
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    z, _, _ = inputs(n, v, k, dtype, v + 2)
    z.clamp_(max=20.0)
    start = torch.randint(0, v, (n, 1), generator=g, device="cuda")
    at = (start + torch.arange(top, device="cuda") * (v // top - 1)) % v
    z.scatter_(1, at, 90.0 - 3 * tau * torch.rand(n, top, generator=g, device="cuda"))
    ids = at[:, :k].to(torch.int32)
    t = 90.0 - 3 * tau * torch.rand(n, k, generator=g, device="cuda")
    loss, lse, dz = run(K, z, ids, t, tau)
    alone = torch.empty(n, device="cuda")
    K.kronq_distill(z, ids, t, alone, temperature=tau)
    torch.cuda.synchronize()
    wl, wlse, q, wg = exact(z, ids, t, tau)
    rel = (v / 256 + 64) * 2.0 ** -23 + 8 * 2.0 ** -23
    p = torch.softmax(t.double() / tau, 1)
    size = tau * (2 * q + torch.zeros_like(q).scatter_add_(1, at[:, :k], p))
    assert bool(((dz.double() - wg).abs() <= rel * size + U32 * wg.abs() + 1e-38).all())
    assert bool(((lse.double() - wlse).abs() <= rel + U32 * wlse.abs()).all())
    for got in (loss, alone):
        assert bool(((got.double() - wl).abs() <= tau * tau * 12 * rel + U32 * wl.abs()).all())


def relative(z, ids, t, tau):
    """(loss, q, gradient) of rows however large their logits are: everything as a difference to the
    row's, or the list's, maximum."""
    u = (z.double() - z.double().amax(1, keepdim=True)) / tau
    logs = u.exp().sum(1, keepdim=True).log()
    c = t.double() - t.double().amax(1, keepdim=True)
    logp = torch.log_softmax(c / tau, 1)
    p = logp.exp()
    at = ids.long()
    q = (u - logs).exp()
    loss = tau * tau * (p * (logp - (u - logs).gather(1, at))).sum(1)
    return loss, q, tau * (q - torch.zeros_like(q).scatter_add_(1, at, p))


@pytest.mark.parametrize("n,v,dtype", RING + FEW)
@pytest.mark.parametrize("value", [-1e7, -1e12, -1e30, 1e12, -2e38, "lowest"])
def test_rows_of_one_large_value(K, n, v, dtype, value):
    """Rows, and lists, that hold nothing but one large finite value (a mask of -1e30, say): q = 1 / V,
    p = 1 / k, loss = log V - log k."""
    k, tau = 20, 0.75
    if value == "lowest":
        value = torch.finfo(dtype).min
    z, ids, t = inputs(n, v, k, dtype, v + 3)
    # a third of the rows, half of those with a list of the value too
    hit = torch.arange(n, device="cuda") % 3 == 1
    both = torch.arange(n, device="cuda") % 6 == 4
    z[hit] = value
    t[both] = value
    loss, lse, dz = run(K, z, ids, t, tau)
    alone = torch.empty(n, device="cuda")
    K.kronq_distill(z, ids, t, alone, temperature=tau)
    torch.cuda.synchronize()
    wl, q, wg = relative(z, ids, t, tau)
    stat = (v / 256 + 64) * 2.0 ** -23
    # an entry's exponent is below 32 here, log p and log q below 40, p and the mass good to stat
    rel = stat + 64 * U32
    size = tau * (2 * q + wg.abs() / tau)
    assert bool(((dz.double() - wg).abs() <= rel * size + HALF[dtype] * wg.abs() + 1e-38).all())
    for got in (loss, alone):
        assert bool(((got.double() - wl).abs() <= tau * tau * 80 * rel + U32 * wl.abs()).all())
    top = z[hit].double().amax(1) / tau
    if abs(value) / tau > torch.finfo(F32).max:        # past fp32, which rounds it to an infinity
        assert bool((lse[hit] == math.copysign(math.inf, value)).all())
    else:
        assert bool(((lse[hit].double() - top - math.log(v)).abs() <= stat + 2 * U32 * top.abs()).all())
    assert K.kronq_device_error() == 0


@pytest.mark.parametrize("n,v,dtype", [c for c in RING + FEW if c[2] == F32])
@pytest.mark.parametrize("middle", [2.0 ** 20, -2.0 ** 20, 3e6, -4e7])
def test_maxima_of_every_size(K, n, v, dtype, middle):
    """Entries within a few tau of each other whose z / tau lies around 2^20 and beyond, where the
    kernels change the form of the exponent: maxima of either form meet in a row's sum."""
    k, tau = 6, 0.75
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    z = torch.full((n, v), -3e38, device="cuda")
    at = torch.randint(0, v // 12, (n, 12), generator=g, device="cuda") + torch.arange(
        12, device="cuda") * (v // 12)
    near = middle * tau * math.log(2.0)                # z c = middle
    z.scatter_(1, at, near + torch.randint(-4, 5, (n, 12), generator=g, device="cuda").float() / 2)
    ids = at[:, :k].to(torch.int32)
    t = near + torch.randint(-4, 5, (n, k), generator=g, device="cuda").float() / 2
    loss, lse, dz = run(K, z, ids, t, tau)
    wl, q, wg = relative(z, ids, t, tau)
    # exponents below 8, a dozen terms: the sums' joins and the exponentials
    rel = 96 * 2.0 ** -23
    p = torch.softmax((t.double() - near) / tau, 1)
    size = tau * (2 * q + torch.zeros_like(q).scatter_add_(1, at[:, :k], p))
    assert bool(((dz.double() - wg).abs() <= rel * size + U32 * wg.abs() + 1e-38).all())
    assert bool(((loss.double() - wl).abs() <= tau * tau * 20 * rel + U32 * wl.abs()).all())


@pytest.mark.parametrize("n,v,dtype", RING + FEW)
def test_in_place(K, n, v, dtype):
    """dlogits = logits, with entries of every CTA's part of the row listed: the bits of a gradient of its
    own, and those near the definition's. The teacher's logits are fp32 beside either type."""
    k, tau = 64, 1.25
    z, ids, t = inputs(n, v, k, dtype, v + 4)
    ids[1::5, 3] = ids[1::5, 40]                       # listed twice
    w = 0.5 + torch.rand(n, device="cuda")
    loss, lse, dz = run(K, z, ids, t, tau, w)
    for _ in range(5):
        zc = z.clone()
        loss2, lse2, _ = run(K, zc, ids, t, tau, w, dz=zc)
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dz, zc)
    back, zc = torch.empty_like(z), z.clone()
    K.kronq_distill_backward(z, ids, t, lse, w, back, temperature=tau)
    K.kronq_distill_backward(zc, ids, t, lse, w, zc, temperature=tau)
    torch.cuda.synchronize()
    assert torch.equal(back, zc)
    stat = (v / 256 + 64) * 2.0 ** -23
    for r in range(0, n, 100):
        s = slice(r, r + 100)
        wl, wlse, q, wg = exact(z[s], ids[s], t[s], tau, w[s])
        unit = w[s].double()[:, None] * tau
        size = 2 * unit * q + wg.abs()
        tol = (stat + 100 * U32) * size + HALF[dtype] * wg.abs() + 1e-38
        assert bool(((dz[s].double() - wg).abs() <= tol).all())
        # from the rounded lse: 2^-24 of it more in the exponent
        tol = tol + 2 * U32 * wlse.abs()[:, None] * size
        assert bool(((back[s].double() - wg).abs() <= tol).all())
        assert bool(((loss[s].double() - wl).abs() <= w[s] * tau * tau * 40 * (stat + 100 * U32)
                     + U32 * wl.abs()).all())
    assert K.kronq_device_error() == 0


@pytest.mark.parametrize("n,v,dtype", RING + FEW)
def test_masked_rows(K, n, v, dtype):
    """Rows of every kind beside each other: masks of -inf and of the type's lowest value around the
    list, nothing left, an entry masked, weight 0, no entries, entries without probability."""
    k, tau = 20, 1.0
    z, ids, t = inputs(n, v, k, dtype, v + 5)
    w = 0.5 + torch.rand(n, device="cuda")
    kind = torch.arange(n, device="cuda") % 10 if n >= 10 else torch.arange(n, device="cuda") * 2 + 1
    listed = torch.zeros(n, v, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
    for at, value in ((1, -math.inf), (2, torch.finfo(dtype).min)):
        z.masked_fill_((kind == at)[:, None] & ~listed, value)
    z[kind == 3] = -math.inf
    hide = kind == 4
    z[hide, ids[hide, 7].long()] = -math.inf
    w[kind == 5] = 0.0
    z[kind == 5, 11] = math.nan
    z[kind == 5, v - 1] = math.inf
    ids[kind == 6] = -1
    t[kind == 6] = math.nan                            # absent: not looked at
    t[kind == 7, 2:] = -math.inf
    ids[kind == 8, 5:] = v                             # outside
    del listed
    loss, lse, dz = run(K, z, ids, t, tau, w)
    none = (kind == 5) | (kind == 6)
    assert bool((loss[none] == 0).all()) and bool((dz[none] == 0).all())
    assert bool((loss[(kind == 3) | hide] == math.inf).all()) and bool((lse[kind == 3] == -math.inf).all())
    stat = (v / 256 + 64) * 2.0 ** -23
    # nothing left: q = 0, the gradient is -w p alone
    rows = kind == 3
    p = torch.softmax(t[rows].double(), 1)
    want = torch.zeros_like(dz[rows], dtype=torch.float64).scatter_(1, ids[rows].long(),
                                                                     -w[rows].double()[:, None] * p)
    tol = (stat + 100 * U32 + HALF[dtype]) * want.abs()
    assert bool(((dz[rows].double() - want).abs() <= tol).all())
    ids = ids.masked_fill(ids >= v, -1)
    t = t.masked_fill((kind == 6)[:, None], 0.0)
    rows = ~(none | (kind == 3))
    z, ids, t, w, loss, lse, dz, hide = (c[rows] for c in (z, ids, t, w, loss, lse, dz, hide))
    wl, wlse, q, wg = exact(z, ids, t, tau, w)
    unit = w.double()[:, None] * tau
    tol = (stat + 100 * U32) * (2 * unit * q + wg.abs()) + HALF[dtype] * wg.abs() + 1e-38
    assert bool(((dz.double() - wg).abs() <= tol).all())
    assert bool(((lse.double() - wlse).abs() <= stat + 2 * U32 * wlse.abs()).all())
    off = (loss.double() - wl).abs() <= w * 40 * (stat + 100 * U32) + U32 * wl.abs()
    assert bool((off | hide).all())
    assert K.kronq_device_error() == 0
