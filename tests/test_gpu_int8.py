"""The quantized layer in 8-bit integers vs the fp64 oracle.

Without a rotation the token codes, scales and sums are defined exactly, so they must be equal.
With one, x' comes from log2(b) fp32 butterfly stages over values no larger than A = sum |x / s_x|
of the block, then one product with fl(1 / sqrt(b)) (itself half a step off), after one division:
|x' error| <= (log2(b) + 4) 2^-24 A / sqrt(b), and a code may be that much over s away from the
nearest. The product's integer part is exact: its output carries one rounding to fp32, one of
s_t s_o, one of their product, and y's own.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kronq_oracle as O
from post_quantization_b200 import synth

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24                       # half a step of fp32
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


def padded(rows, cols, dtype, extra=0):
    ld = (cols + 15) // 16 * 16 + 16 * extra
    return torch.full((rows, ld), 77, dtype=dtype, device="cuda")[:, :cols]


def quantize(K, x, s_x=None, sign_in=None, **kw):
    n, d = x.shape
    q = padded(n, d, torch.int8)
    scale = torch.full((n,), -1.0, device="cuda")
    total = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    flags = (K.BIIP_SCALE_IN if s_x is not None else 0) | \
        (K.BIIP_ROTATE_IN if sign_in is not None else 0)
    K.kronq_quantize_tokens(x, q, scale, total, s_x=s_x, sign_in=sign_in, flags=flags, **kw)
    torch.cuda.synchronize()
    return q, scale, total


def fp32_scaled(x, s_x):
    """x / s_x as fp32 rounds it: the value that the codes of an unrotated token are defined on."""
    return (x.detach().cpu().float().numpy() / s_x.detach().cpu().numpy()[None, :])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (2, 16), (5, 333), (64, 4096), (9, 11008),
                                 (2, 65536), (1, 28672)])
@pytest.mark.parametrize("scaled", [False, True])
def test_quantize_tokens_exact(K, dtype, n, d, scaled):
    tag = ("i8q", n, d, scaled, str(dtype))
    x = synth.activations(n, d, synth.seed_for(tag), dtype=dtype, device="cuda")
    s_x = synth.positive_scales(d, synth.seed_for(tag, "s"), device="cuda") if scaled else None
    q, scale, total = quantize(K, x, s_x)
    xin = fp32_scaled(x, s_x) if scaled else x.float().cpu().numpy()
    _, s, want, wsum = O.quantize_tokens(xin)
    np.testing.assert_array_equal(np64(scale), s)
    np.testing.assert_array_equal(q.cpu().numpy(), want)
    np.testing.assert_array_equal(total.cpu().numpy(), wsum)
    base = torch.as_strided(q, (n, q.stride(0)), (q.stride(0), 1))
    assert bool((base[:, d:] == 77).all())               # nothing written past the width


def test_quantize_tokens_ties_and_borders(K):
    # s = 1 (the largest entry is 127): halves round to even, and neighbours of a half by one ulp
    h = np.arange(-126.5, 127.0, 1.0, dtype=np.float32)
    row = np.concatenate([[127.0], h, np.nextafter(h, np.float32(1e9)),
                          np.nextafter(h, np.float32(-1e9))]).astype(np.float32)
    # and scales that are no power of two: values k s / 2 rounded to fp32, next to each border
    s = np.float32(0.0123)
    k = (np.arange(-253, 254, 2) * 0.5 * np.float64(s)).astype(np.float32)
    row2 = np.concatenate([[np.float32(127) * s], k, np.nextafter(k, np.float32(1)),
                           np.nextafter(k, np.float32(-1))]).astype(np.float32)
    width = max(row.size, row2.size)
    x = np.zeros((2, width), np.float32)
    x[0, :row.size] = row
    x[1, :row2.size] = row2
    q, scale, total = quantize(K, torch.from_numpy(x).cuda())
    _, sc, want, wsum = O.quantize_tokens(x)
    np.testing.assert_array_equal(np64(scale), sc)
    np.testing.assert_array_equal(q.cpu().numpy(), want)
    np.testing.assert_array_equal(total.cpu().numpy(), wsum)


def test_quantize_tokens_special_rows(K):
    d = 300
    x = torch.randn(7, d, device="cuda")
    x[1] = 0.0
    x[2, 5] = float("inf")
    x[3, 299] = float("nan")
    x[4] = 1e-44                                          # below the smallest scale
    x[5] *= 3e38 / x[5].abs().max()
    x[6] *= 1e-36
    q, scale, total = quantize(K, x)
    _, s, want, wsum = O.quantize_tokens(x.cpu().numpy())
    np.testing.assert_array_equal(np64(scale), s)         # NaN where not finite
    assert math.isnan(float(scale[2])) and math.isnan(float(scale[3]))
    assert float(scale[1]) == 1.0 and float(scale[4]) == 1.0
    np.testing.assert_array_equal(q.cpu().numpy(), want)
    np.testing.assert_array_equal(total.cpu().numpy(), wsum)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 1), (2, 2), (3, 24), (4, 336), (7, 1024), (2, 11008),
                                 (33, 8192), (2, 28672), (1, 53248), (3, 16384), (5, 333)])
def test_quantize_tokens_rotated(K, dtype, n, d):
    tag = ("i8r", n, d, str(dtype))
    x = synth.activations(n, d, synth.seed_for(tag), dtype=dtype, device="cuda")
    s_x = synth.positive_scales(d, synth.seed_for(tag, "s"), device="cuda")
    si = synth.rademacher(d, synth.seed_for(tag, "si"), device="cuda")
    q, scale, total = quantize(K, x, s_x, si)
    xp, s, _, _ = O.quantize_tokens(np64(x), np64(s_x), np64(si))
    b = O.hadamard_block_size(d)
    mag = np.abs(np64(x) / np64(s_x)).reshape(n, d // b, b).sum(-1) / math.sqrt(b)
    err = (math.log2(b) + 4) * U32 * mag
    got_s = np64(scale)
    assert (np.abs(got_s - s) <= err.max(1) / 127 + 2 * U32 * s).all()
    off = np.abs(q.cpu().numpy() - xp / got_s[:, None])
    room = np.repeat(err, b, axis=1) / got_s[:, None]
    assert (off <= 0.5 + room + 1e-12).all()
    np.testing.assert_array_equal(total.cpu().numpy(), q.cpu().numpy().astype(np.int64).sum(1))


def weights(d_out, d_in, signed, tag):
    r = np.random.default_rng(synth.seed_for(tag) % (1 << 32))
    lo = -128 if signed else 0
    c = r.integers(lo, lo + 256, (d_out, d_in))
    codes = padded(d_out, d_in, torch.int8 if signed else torch.uint8)
    codes.copy_(torch.from_numpy(c))
    scale, zero = synth.grid_params(d_out, 0, 8, synth.seed_for(tag, "grid"), device="cuda")
    return codes, scale, zero


def tokens(n, d_in, tag):
    r = np.random.default_rng(synth.seed_for(tag, "q") % (1 << 32))
    q = padded(n, d_in, torch.int8)
    q.copy_(torch.from_numpy(r.integers(-127, 128, (n, d_in))))
    scale = torch.from_numpy(r.lognormal(-4, 1, n).astype(np.float32)).cuda()
    return q, scale, q.to(torch.int64).sum(1).to(torch.int32)


def check_matmul(y, q, ts, codes, scale, zero):
    want = O.matmul_i8(q.cpu().numpy(), np64(ts), codes.cpu().numpy(), np64(scale),
                       None if zero is None else np64(zero))
    got = np64(y)
    tol = (3.1 * U32 + HALF[y.dtype]) * np.abs(want) + 1e-300
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5])


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 512), (2, 130, 300), (3, 1000, 4096), (16, 256, 1000),
          (17, 129, 129), (33, 1024, 2048), (64, 384, 640), (65, 77, 4112), (127, 640, 256),
          (128, 1, 8192), (200, 513, 1040), (257, 300, 144), (300, 2049, 384), (513, 1025, 16),
          (1000, 768, 11008), (1, 28672, 256), (5, 64, 28672), (40, 8192, 96), (90, 4096, 4096)]


@pytest.mark.parametrize("n,d_out,d_in", SHAPES)
@pytest.mark.parametrize("signed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matmul_i8(K, n, d_out, d_in, signed, dtype):
    tag = ("i8m", n, d_out, d_in, signed)
    codes, scale, zero = weights(d_out, d_in, signed, tag)
    if signed and (n + d_out) % 2:
        zero = None
    q, ts, total = tokens(n, d_in, tag)
    buf = torch.full((n + 2, d_out + 5), float("nan"), dtype=dtype, device="cuda")
    y = buf[1:n + 1, 2:d_out + 2]                     # rows and columns around it stay as they are
    K.kronq_matmul_i8(q, ts, total if zero is not None else None, codes, scale, zero, y)
    torch.cuda.synchronize()
    check_matmul(y, q, ts, codes, scale, zero)
    buf[1:n + 1, 2:d_out + 2] = float("nan")
    assert bool(buf.isnan().all())
    assert K.kronq_device_error() == 0


def test_matmul_i8_extreme_sums(K):
    # the largest magnitudes the int32 sums can take: all codes 255, all token codes -128 / 127
    n, d_out, d_in = 3, 130, 65536
    codes = torch.full((d_out, d_in), 255, dtype=torch.uint8, device="cuda")
    q = torch.full((n, d_in), 127, dtype=torch.int8, device="cuda")
    q[1] = -128
    q[2, ::2] = -127
    ts = torch.tensor([0.5, 0.25, 3.0], device="cuda")
    total = q.to(torch.int64).sum(1).to(torch.int32)
    scale = torch.full((d_out,), 0.125, device="cuda")
    zero = torch.zeros(d_out, device="cuda")
    zero[1::4], zero[2::4] = 255.0, 128.0
    # zeros far outside the code range, a fraction, and one that int32 could not hold
    zero[3], zero[7], zero[11], zero[15] = -2550.0, 0.5, 3.0e9, -16777216.0
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.empty(n, d_out, dtype=dtype, device="cuda")
        K.kronq_matmul_i8(q, ts, total, codes, scale, zero, y)
        torch.cuda.synchronize()
        check_matmul(y, q, ts, codes, scale, zero)


def test_matmul_i8_nan_token_and_empty(K):
    codes, scale, zero = weights(64, 96, False, ("i8n",))
    q, ts, total = tokens(4, 96, ("i8n",))
    q[2] = 0
    total[2] = 0
    ts[2] = float("nan")
    y = torch.zeros(4, 64, device="cuda")
    K.kronq_matmul_i8(q, ts, total, codes, scale, zero, y)
    assert bool(y[2].isnan().all()) and not bool(y[[0, 1, 3]].isnan().any())
    K.kronq_matmul_i8(q[:0], ts[:0], total[:0], codes, scale, zero, y[:0])
    # a single row whose tensor stride is no valid row stride
    y1 = torch.zeros(1, 64, device="cuda")
    q1 = torch.as_strided(q, (1, 96), (3, 1))
    K.kronq_matmul_i8(q1, ts[:1], total[:1], codes, scale, zero, y1)
    torch.cuda.synchronize()
    assert torch.equal(y1[0], y[0])


@pytest.mark.parametrize("budget", [1, 5, 100])
def test_matmul_i8_budget_and_token_slices_give_the_same_bits(K, budget):
    codes, scale, zero = weights(1300, 2000, False, ("i8b",))
    q, ts, total = tokens(300, 2000, ("i8b",))
    y = torch.empty(300, 1300, device="cuda")
    K.kronq_matmul_i8(q, ts, total, codes, scale, zero, y)
    parts = torch.empty_like(y)
    try:
        K.kronq_set_sm_budget(budget)
        for t0, t1 in ((0, 1), (1, 12), (12, 44), (44, 108), (108, 300)):
            K.kronq_matmul_i8(q[t0:t1], ts[t0:t1], total[t0:t1], codes, scale, zero, parts[t0:t1])
        torch.cuda.synchronize()
    finally:
        K.kronq_set_sm_budget(0)
    assert torch.equal(y, parts)


LAYERS = [(1, 256, 256), (1, 4096, 1024), (3, 300, 520), (17, 1024, 4096), (70, 768, 11008),
          (2, 8192, 512), (33, 1001, 77), (2, 16384, 64), (260, 640, 1536)]


@pytest.mark.parametrize("n,d_out,d_in", LAYERS)
@pytest.mark.parametrize("flags", [0, 1, 2, 5, 8, 10, 15])
def test_qlinear8(K, n, d_out, d_in, flags):
    tag = ("i8l", n, d_out, d_in, flags)
    codes, scale, zero = weights(d_out, d_in, False, tag)
    x = synth.activations(n, d_in, synth.seed_for(tag, "x"), dtype=torch.bfloat16, device="cuda")
    s_x = synth.positive_scales(d_in, synth.seed_for(tag, "sx"), device="cuda")
    s_g = synth.positive_scales(d_out, synth.seed_for(tag, "sg"), device="cuda")
    si = synth.rademacher(d_in, synth.seed_for(tag, "si"), device="cuda")
    so = synth.rademacher(d_out, synth.seed_for(tag, "so"), device="cuda")
    dtype = torch.float32 if (n + flags) % 2 else torch.bfloat16
    y = torch.full((n, d_out), float("nan"), dtype=dtype, device="cuda")
    K.kronq_qlinear8(x, codes, scale, zero, s_x if flags & 1 else None, s_g if flags & 2 else None,
                     si if flags & 4 else None, so if flags & 8 else None, flags, y)
    # the token codes are checked above; the rest of the layer is compared from them on
    q, ts, _ = quantize(K, x, s_x if flags & 1 else None, si if flags & 4 else None)
    yp = O.matmul_i8(q.cpu().numpy(), np64(ts), codes.cpu().numpy(), np64(scale), np64(zero))
    b = O.hadamard_block_size(d_out) if flags & 8 else 1
    want = yp
    mag = np.abs(yp).reshape(n, d_out // b, b).sum(-1, keepdims=True) / math.sqrt(b)
    mag = np.broadcast_to(mag, (n, d_out // b, b)).reshape(n, d_out)
    if flags & 8:
        want = O.hadamard_rows(yp) * np64(so)[None, :]
    if flags & 2:
        want, mag = want / np64(s_g)[None, :], mag / np64(s_g)[None, :]
    # three roundings of the product, log2(b) stages, 1 / sqrt(b) and its product, the division
    tol = (3.1 + math.log2(b) + 4) * U32 * mag + HALF[dtype] * np.abs(want)
    got = np64(y)
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
    assert K.kronq_device_error() == 0


def test_qlinear8_more_tokens_than_a_pass_strides_and_replay(K):
    n, d_out, d_in = 2100, 256, 272
    tag = ("i8p",)
    codes, scale, zero = weights(d_out, d_in, False, tag)
    xb = torch.zeros(n, d_in + 3, dtype=torch.bfloat16, device="cuda")
    xb[:, 1:d_in + 1] = synth.activations(n, d_in, synth.seed_for(tag, "x"), dtype=torch.bfloat16,
                                          device="cuda")
    x = xb[:, 1:d_in + 1]                              # rows off alignment
    so = synth.rademacher(d_out, synth.seed_for(tag, "so"), device="cuda")
    yb = torch.full((n, d_out + 1), -7.0, dtype=torch.bfloat16, device="cuda")
    y = yb[:, :d_out]
    size = K.kronq_qlinear8_workspace_size(n, d_out, d_in, K.BIIP_ROTATE_OUT)
    assert size == K.kronq_qlinear8_workspace_size(2048, d_out, d_in, K.BIIP_ROTATE_OUT)
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:size]

    def call():
        K.kronq_qlinear8(x, codes, scale, zero, None, None, None, so, K.BIIP_ROTATE_OUT, y,
                         workspace=ws)
    call()
    torch.cuda.synchronize()
    first = y.clone()
    assert bool((yb[:, d_out:] == -7.0).all())
    for rows in (slice(0, 40), slice(2040, 2100)):     # both sides of the passes' border
        part = torch.empty(rows.stop - rows.start, d_out, dtype=torch.bfloat16, device="cuda")
        K.kronq_qlinear8(x[rows], codes, scale, zero, None, None, None, so, K.BIIP_ROTATE_OUT, part)
        torch.cuda.synchronize()
        assert torch.equal(part, first[rows])
    y.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            call()
    xb.mul_(2.0)                                       # exact in bf16: y doubles
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first * 2)
    del g


def test_8bit_layer_of_a_solved_layer(K):
    """Solve at 8 bits, run it through pipeline.Linear8: near W x, and a better fit than 4 bits."""
    from post_quantization_b200 import pipeline as P
    d_out, d_in, n = 264, 500, 2048                    # a width that needs padded code rows
    tag = ("i8e",)
    xall = synth.correlated_x(n + 40, d_in, synth.seed_for(tag, "X"), device="cuda")
    g = synth.gradients(n, d_out, synth.seed_for(tag, "G"), device="cuda")
    xc = torch.zeros(n, 504, dtype=torch.bfloat16, device="cuda")[:, :d_in]
    xc.copy_(xall[:n])
    w = synth.weight(d_out, d_in, synth.seed_for(tag, "W"), dtype=torch.float32, device="cuda")
    si = synth.rademacher(d_in, synth.seed_for(tag, "si"), device="cuda")
    so = synth.rademacher(d_out, synth.seed_for(tag, "so"), device="cuda")
    hx = torch.zeros(d_in, d_in, device="cuda")
    hg = torch.zeros(d_out, d_out, device="cuda")
    K.kronq_accumulate(xc, None, g, hx, hg, None)
    errs = {}
    x = xall[n:]
    full = np64(x) @ np64(w).T
    for bits in (4, 8):
        r = P.biip(w, hx, hg, None, 1.0 / n, si, so)
        P.cholinv(r)
        P.quantize(r, bits)
        layer = P.Linear8.of(r, si, so)
        y = layer(x, dtype=torch.float32)
        torch.cuda.synchronize()
        dense = O.qlinear_dense(np64(r.w_hat), np64(x), np64(r.s_x), np64(r.s_g), np64(si), np64(so))
        # what 8-bit activations add to the dequantized layer: a rounding of half a step of
        # max |x'| / 127 per entry, independent over the 500 entries, so near 127^-1 / sqrt(12)
        # of max |x'| / rms(x') (below 6) relative: 1.4e-2; three times that here
        e = np.linalg.norm(np64(y) - dense) / np.linalg.norm(dense)
        assert e <= 4.2e-2, e
        errs[bits] = np.einsum("ti,ij,tj->", np64(y) - full, np64(hg), np64(y) - full)
    assert errs[8] < errs[4]


@pytest.mark.parametrize("n,d_out,d_in,signed", [(2100, 2561, 400, False), (4096, 2560, 144, True),
                                                 (700, 9000, 1000, False), (16384, 300, 272, False)])
def test_matmul_i8_prompts(K, n, d_out, d_in, signed):
    """Large calls: every output against the exact integer product (fp64 on the device)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n + d_out)
    lo = -128 if signed else 0
    codes = padded(d_out, d_in, torch.int8 if signed else torch.uint8)
    codes.copy_(torch.randint(lo, lo + 256, (d_out, d_in), generator=g, device="cuda"))
    q = padded(n, d_in, torch.int8)
    q.copy_(torch.randint(-127, 128, (n, d_in), generator=g, device="cuda"))
    ts = torch.rand(n, generator=g, device="cuda") + 0.1
    total = q.to(torch.int64).sum(1).to(torch.int32)
    scale, zero = synth.grid_params(d_out, 0, 8, synth.seed_for("i8pp", n), device="cuda")
    want = (q.double() @ (codes.double() - zero.double()[:, None]).t()) * ts.double()[:, None] * \
        scale.double()[None, :]
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((n, d_out + 3), float("nan"), dtype=dtype, device="cuda")[:, :d_out]
        K.kronq_matmul_i8(q, ts, total, codes, scale, zero, y)
        torch.cuda.synchronize()
        tol = (3.1 * U32 + HALF[dtype]) * want.abs() + 1e-300
        assert bool(((y.double() - want).abs() <= tol).all())
    assert K.kronq_device_error() == 0


@pytest.mark.parametrize("d", [16, 48, 96, 192, 384, 1536, 2048, 6144, 32768, 49152])
def test_rotations_of_every_block_size(K, d):
    """Blocks of 16 .. 32768 on both sides, on aligned rows and on others: the same bits."""
    n, d2 = 3, min(d, 16384)
    tag = ("i8b", d)
    x = synth.activations(n, d, synth.seed_for(tag), dtype=torch.bfloat16, device="cuda")
    si = synth.rademacher(d, synth.seed_for(tag, "si"), device="cuda")
    s_x = synth.positive_scales(d, synth.seed_for(tag, "s"), device="cuda")
    q, scale, total = quantize(K, x, s_x, si)
    xp, s, _, _ = O.quantize_tokens(np64(x), np64(s_x), np64(si))
    b = O.hadamard_block_size(d)
    mag = np.abs(np64(x) / np64(s_x)).reshape(n, d // b, b).sum(-1) / math.sqrt(b)
    err = (math.log2(b) + 4) * U32 * mag
    assert (np.abs(np64(scale) - s) <= err.max(1) / 127 + 2 * U32 * s).all()
    off = np.abs(q.cpu().numpy() - xp / np64(scale)[:, None])
    assert (off <= 0.5 + np.repeat(err, b, axis=1) / np64(scale)[:, None] + 1e-12).all()
    np.testing.assert_array_equal(total.cpu().numpy(), q.cpu().numpy().astype(np.int64).sum(1))
    for dtype in (torch.bfloat16, torch.float32):      # rows off alignment; fp32 holds the same x
        xo = torch.zeros(n, d + 3, dtype=dtype, device="cuda")[:, 1:d + 1]
        xo.copy_(x)
        qo, so, to = quantize(K, xo, s_x, si)
        assert torch.equal(q, qo) and torch.equal(scale, so) and torch.equal(total, to)

    codes, ws, zero = weights(d2, 64, False, tag)
    x2 = synth.activations(n, 64, synth.seed_for(tag, "x"), dtype=torch.bfloat16, device="cuda")
    s_g = synth.positive_scales(d2, synth.seed_for(tag, "sg"), device="cuda")
    sgn = synth.rademacher(d2, synth.seed_for(tag, "so"), device="cuda")
    flags = K.BIIP_SCALE_OUT | K.BIIP_ROTATE_OUT
    q, ts, _ = quantize(K, x2)
    yp = O.matmul_i8(q.cpu().numpy(), np64(ts), codes.cpu().numpy(), np64(ws), np64(zero))
    want = O.hadamard_rows(yp) * np64(sgn)[None, :] / np64(s_g)[None, :]
    b = O.hadamard_block_size(d2)
    mag = np.repeat(np.abs(yp).reshape(n, d2 // b, b).sum(-1) / math.sqrt(b), b, axis=1) / np64(s_g)
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.empty(n, d2, dtype=dtype, device="cuda")
        yo = torch.full((n, d2 + 3), -7.0, dtype=dtype, device="cuda")
        K.kronq_qlinear8(x2, codes, ws, zero, None, s_g, None, sgn, flags, y)
        K.kronq_qlinear8(x2, codes, ws, zero, None, s_g, None, sgn, flags, yo[:, 1:d2 + 1])
        torch.cuda.synchronize()
        tol = (3.1 + math.log2(b) + 4) * U32 * mag + HALF[dtype] * np.abs(want)
        assert (np.abs(np64(y) - want) <= tol).all()
        assert torch.equal(y, yo[:, 1:d2 + 1])
        assert bool((yo[:, 0] == -7.0).all()) and bool((yo[:, d2 + 1:] == -7.0).all())


def test_rotated_tokens_that_are_not_finite(K):
    """Infinities, NaN and sums past fp32 anywhere in a block: the token has no codes and scale NaN."""
    d = 512
    x = torch.randn(9, d, device="cuda")
    si = torch.ones(d, dtype=torch.int8, device="cuda")
    x[1] = 0.0
    x[2, 77] = float("inf")
    x[3, 300] = float("-inf")
    x[3, 301] = float("inf")
    x[4, 511] = float("nan")
    x[5] = 0.0                                         # sums of 6e38, some of which cancel
    x[5, [8, 9, 12]] = 3e38
    x[5, [13]] = 3e38
    x[6] = 0.0
    x[6, [8, 9, 12, 13]] = torch.tensor([3e38, 3e38, -3e38, -3e38], device="cuda")
    x[7] *= 1e-41
    q, scale, total = quantize(K, x, None, si)
    bad = torch.isnan(scale).tolist()
    assert bad == [False, False, True, True, True, True, True, False, False]
    rows = [1, 2, 3, 4, 5, 6, 7]
    assert float(scale[1]) == 1.0 and float(scale[7]) == 1.0
    assert int(q[rows].abs().max()) == 0 and int(total[rows].abs().max()) == 0
    # the other rows do not feel them
    ok, s_ok, _ = quantize(K, x[[0, 8]].contiguous(), None, si)
    assert torch.equal(q[[0, 8]], ok) and torch.equal(scale[[0, 8]], s_ok)


def test_two_streams_at_once(K):
    """Tokens quantized and multiplied on two streams side by side, and codes that the call before
    has just written: the bits of one call after the other."""
    n, d_out, d_in = 200, 640, 1040
    a = [weights(d_out, d_in, False, ("i8t", i)) for i in range(2)]
    xs = [synth.activations(n, d_in, synth.seed_for(("i8t", "x"), i), dtype=torch.bfloat16,
                            device="cuda") for i in range(2)]
    si = synth.rademacher(d_in, 5, device="cuda")
    so = synth.rademacher(d_out, 6, device="cuda")
    want = []
    for (c, s, z), x in zip(a, xs):
        y = torch.empty(n, d_out, device="cuda")
        K.kronq_qlinear8(x, c, s, z, None, None, si, so, K.BIIP_ROTATE_IN | K.BIIP_ROTATE_OUT, y)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty(n, d_out, device="cuda") for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for r in range(6):
        for i, s in enumerate(streams):
            c, sc, z = a[i]
            K.kronq_qlinear8(xs[i], c, sc, z, None, None, si, so,
                             K.BIIP_ROTATE_IN | K.BIIP_ROTATE_OUT, got[i][r], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(w, g) for w, gs in zip(want, got) for g in gs)

    # the codes themselves come from kronq_quantize_tokens (symmetric, one grid per row)
    w = torch.randn(d_out, d_in, device="cuda")
    codes = padded(d_out, d_in, torch.int8)
    grid = torch.empty(d_out, device="cuda")
    sums = torch.empty(d_out, dtype=torch.int32, device="cuda")
    q, ts, total = quantize(K, xs[0])
    y = torch.empty(n, d_out, device="cuda")
    for k in range(4):
        w.mul_(-1.25)
        K.kronq_quantize_tokens(w, codes, grid, sums)
        K.kronq_matmul_i8(q, ts, total, codes, grid, None, y)
    torch.cuda.synchronize()
    _, s, c, _ = O.quantize_tokens(w.cpu().numpy())
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    ref = O.matmul_i8(q.cpu().numpy(), np64(ts), c, s, None)
    assert (np.abs(np64(y) - ref) <= 3.1 * 2 * U32 * np.abs(ref) + 1e-300).all()
