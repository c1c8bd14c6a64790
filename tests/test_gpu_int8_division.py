"""Channel scales of the 8-bit layer: x / s_x and y' / s_g are fp32 quotients to 2 ulp on rotated sides
(blocks above 8 on the input), subnormal numbers included.

With one nonzero entry per Hadamard block every entry of the block's transform is plus or minus that
entry, so that each rounding can be followed. Relative to the exact value, 2 ulp are at most
4 x 2^-24 and a rounding 2^-24; below 2^-126 an ulp is 2^-149 whatever the value.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kronq_oracle as O
from post_quantization_b200 import synth

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def K():
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import kronq
    kronq.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kronq.kronq_device_check()
    return kronq


def quantize(K, x, s_x, sign_in):
    n, d = x.shape
    q = torch.zeros(n, (d + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :d]
    scale, total = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    K.kronq_quantize_tokens(x, q, scale, total, s_x=s_x, sign_in=sign_in,
                            flags=K.BIIP_SCALE_IN | K.BIIP_ROTATE_IN)
    torch.cuda.synchronize()
    return q, scale, total


@pytest.mark.parametrize("d", [8, 16, 48, 512, 2048, 8192])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("exponents", [(-3.0, 3.0), (-30.0, 30.0)])
def test_quotients_of_rotated_tokens(K, d, dtype, exponents):
    n = 500
    r = np.random.default_rng(d)
    x = torch.zeros(n, d, dtype=dtype, device="cuda")
    at = torch.from_numpy(r.integers(0, d, n)).cuda()
    x[torch.arange(n, device="cuda"), at] = torch.from_numpy(
        r.normal(size=n) * 10.0 ** r.uniform(*exponents, n)).to(dtype).cuda()
    s_x = torch.from_numpy((10.0 ** r.uniform(-3, 3, d)).astype(np.float32)).cuda()
    q, scale, total = quantize(K, x, s_x, synth.rademacher(d, 1, device="cuda"))
    b = O.hadamard_block_size(d)
    rows = np.arange(n)
    at = at.cpu().numpy()
    want = np.abs(x.double().cpu().numpy()[rows, at] / s_x.double().cpu().numpy()[at]) / math.sqrt(b) / 127
    # the quotient, 1 / sqrt(b), its product, the scale: 4 + 1 + 1 + 1 half steps
    assert (np.abs(scale.double().cpu().numpy() - want) <= 7.01 * U32 * want).all()
    assert bool((q.abs().amax(1) == 127).all())


@pytest.mark.parametrize("d", [16, 333 * 16, 4096])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_subnormal_tokens_with_small_scales(K, d, dtype):
    """Entries near 1e-39 (subnormal) over scales near 1e-6: tokens like any other, to rounding."""
    n = 5
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    x = (torch.randn(n, d, generator=g, device="cuda", dtype=torch.float64) * 3e-39).to(dtype)
    s_x = synth.positive_scales(d, 3, device="cuda") * 1e-6
    si = synth.rademacher(d, 4, device="cuda")
    q, scale, total = quantize(K, x, s_x, si)
    f64 = lambda v: v.cpu().double().numpy()  # noqa: E731
    xp, s, _, _ = O.quantize_tokens(f64(x), f64(s_x), f64(si))
    b = O.hadamard_block_size(d)
    # as in the tests of rotated tokens: log2(b) stages, quotient, 1 / sqrt(b), its product
    mag = np.abs(f64(x) / f64(s_x)).reshape(n, d // b, b).sum(-1) / math.sqrt(b)
    err = (math.log2(b) + 4) * U32 * mag
    got = f64(scale)
    assert (np.abs(got - s) <= err.max(1) / 127 + 2 * U32 * s).all()
    off = np.abs(q.cpu().numpy() - xp / got[:, None])
    assert (off <= 0.5 + np.repeat(err, b, axis=1) / got[:, None] + 1e-12).all()


@pytest.mark.parametrize("d_out", [1, 8, 16, 1024, 48, 2048, 4096, 16384])
@pytest.mark.parametrize("size", [1.0, 1e-36])
def test_quotients_of_rotated_outputs(K, d_out, size):
    """One nonzero channel: y = +- y' / sqrt(b) / s_g (size 1e-36: y is subnormal for the larger s_g)."""
    n, d_in = 40, 64
    r = np.random.default_rng(d_out)
    codes = torch.zeros(d_out, d_in, dtype=torch.int8, device="cuda")
    codes[d_out // 2] = torch.from_numpy(r.integers(-100, 100, d_in)).cuda()
    scale = torch.from_numpy((size * r.uniform(0.5, 2, d_out)).astype(np.float32)).cuda()
    x = synth.activations(n, d_in, 7, dtype=torch.bfloat16, device="cuda")
    s_g = torch.from_numpy((10.0 ** r.uniform(-3, 4, d_out)).astype(np.float32)).cuda()
    so = synth.rademacher(d_out, 9, device="cuda")
    y = torch.zeros(n, d_out, device="cuda")
    K.kronq_qlinear8(x, codes, scale, None, None, s_g, None, so,
                     K.BIIP_SCALE_OUT | K.BIIP_ROTATE_OUT, y)
    plain = torch.zeros(n, d_out, device="cuda")
    K.kronq_qlinear8(x, codes, scale, None, None, None, None, None, 0, plain)
    torch.cuda.synchronize()
    b = O.hadamard_block_size(d_out)
    first = d_out // 2 // b * b                        # the block of the nonzero channel
    v = np.abs(plain.double().cpu().numpy()[:, d_out // 2:d_out // 2 + 1]) / math.sqrt(b)
    want = v / s_g.double().cpu().numpy()[None, first:first + b]
    got = y.double().cpu().numpy()
    # fl(1 / sqrt(b)) and its product are a half step each, the quotient 2 ulp
    off = np.abs(np.abs(got[:, first:first + b]) - want)
    assert (off <= 6.01 * U32 * want + 2.5 * 2.0 ** -149).all()
    got[:, first:first + b] = 0.0
    assert not got.any()
