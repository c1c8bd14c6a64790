"""A prompt through a wide 8-bit layer with all transforms: the bits repeat whatever runs in between, and
every step follows from the one before in fp64 on the device.

Bounds as for the single steps: |x' error| <= (log2(b) + 4) 2^-24 A / sqrt(b) with A the block's sum of
|x / s_x| (the quotient's 2 ulp take the place of one rounding: + 3), a code is that much over s away from
the nearest, and three roundings of the product, log2(b) stages, 1 / sqrt(b), its product and the quotient
follow for y.
"""
import math

import pytest
import torch

from post_quantization_b200 import synth

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def hadamard(x, b):
    """Orthonormal Hadamard transform of every aligned block of b."""
    n, d = x.shape
    h = 1
    while h < b:
        v = x.reshape(n, d // (2 * h), 2, h)
        x = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).reshape(n, d)
        h *= 2
    return x / math.sqrt(b)


@pytest.mark.parametrize("n,d_out,d_in", [(2048, 8192, 8192), (333, 11008, 4096), (2500, 1536, 28672)])
def test_a_prompt_repeats_and_follows_its_codes(n, d_out, d_in):
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import kronq as K
    from post_quantization_b200 import pipeline as P
    layers, xs = [], []
    for i in range(2):
        tag = ("prompt", d_out, d_in, i)
        scale, zero = synth.grid_params(d_out, 0, 8, synth.seed_for(tag, "g"), device="cuda")
        layers.append(P.Linear8(
            synth.codes(d_out, d_in, 8, synth.seed_for(tag, "c"), device="cuda"), scale, zero,
            synth.positive_scales(d_in, synth.seed_for(tag, "sx"), device="cuda"),
            synth.positive_scales(d_out, synth.seed_for(tag, "sg"), device="cuda"),
            synth.rademacher(d_in, synth.seed_for(tag, "si"), device="cuda"),
            synth.rademacher(d_out, synth.seed_for(tag, "so"), device="cuda")))
        xs.append(synth.activations(n, d_in, synth.seed_for(tag, "x"), dtype=torch.bfloat16,
                                    device="cuda"))
    ws = P.Workspace("cuda")
    first = [layer(x, ws=ws) for layer, x in zip(layers, xs)]
    for _ in range(5):
        for layer, x, want in zip(layers, xs, first):
            assert torch.equal(layer(x, ws=ws), want)

    a, x = layers[0], xs[0].double() / layers[0].s_x.double()
    b = d_in & -d_in
    q = torch.zeros(n, d_in, dtype=torch.int8, device="cuda")
    scale, total = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    K.kronq_quantize_tokens(xs[0], q, scale, total, s_x=a.s_x, sign_in=a.sign_in,
                            flags=K.BIIP_SCALE_IN | K.BIIP_ROTATE_IN)
    s = scale.double()[:, None]
    xp = hadamard(x * a.sign_in.double(), b)
    err = (math.log2(b) + 7) * U32 * x.abs().reshape(n, d_in // b, b).sum(2) / math.sqrt(b)
    assert bool(((s[:, 0] - xp.abs().amax(1) / 127).abs() <= err.amax(1) / 127 + 2 * U32 * s[:, 0]).all())
    room = err.repeat_interleave(b, 1) / s
    assert bool(((q.double() - xp / s).abs() <= 0.5 + room + 1e-12).all())

    w = a.codes.double() - a.zero.double()[:, None]
    y = (q.double() @ w.t()) * s * a.scale.double()
    b = d_out & -d_out
    mag = y.abs().reshape(n, d_out // b, b).sum(2).repeat_interleave(b, 1) / math.sqrt(b)
    s_g = a.s_g.double()
    y = hadamard(y, b) * a.sign_out.double() / s_g
    tol = (3.1 + math.log2(b) + 7) * U32 * mag / s_g + 2.0 ** -8 * y.abs()
    assert bool(((first[0].double() - y).abs() <= tol).all())
    assert K.kronq_device_error() == 0
