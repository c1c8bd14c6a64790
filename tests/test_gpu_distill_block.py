"""The calibration block's backward from a distillation loss, vs autograd in fp64.

The whole chain is restated in fp64 with a plain loss: block with full-precision weights -> top
logits; block with rounded weights -> loss -> gradients of every linear's output. The generator runs
in fp32 (dtype float32, so that nothing is rounded to bf16): products over at most 512 terms, a
softmax over 64 positions and one over the vocabulary, each good to about 2^-20 of its size; 1e-3
of a gradient's norm leaves room for the cancellation between the student's and the teacher's
probabilities, which differ by a few per cent.
"""
import pytest
import torch

from post_quantization_b200 import synth

pytestmark = pytest.mark.gpu


def block64(x, w, nb, seq, heads, kv, hd, outs=None):
    def lin(name, inp):
        out = inp @ w[name].t()
        if outs is not None:
            out.retain_grad()
            outs[name] = out
        return out

    def norm(v):
        return v * torch.rsqrt(v.pow(2).mean(-1, keepdim=True) + 1e-5)
    n1 = norm(x)
    q = lin("q_proj", n1).view(nb, seq, heads, hd).transpose(1, 2)
    k = lin("k_proj", n1).view(nb, seq, kv, hd).transpose(1, 2).repeat_interleave(heads // kv, 1)
    v = lin("v_proj", n1).view(nb, seq, kv, hd).transpose(1, 2).repeat_interleave(heads // kv, 1)
    s = (q @ k.transpose(-1, -2)) / hd ** 0.5
    s = s.masked_fill(torch.ones(seq, seq, dtype=torch.bool, device=x.device).triu(1), -1e300)
    u = x + lin("o_proj", (s.softmax(-1) @ v).transpose(1, 2).reshape(x.shape[0], -1))
    n2 = norm(u)
    y = u + lin("down_proj", torch.nn.functional.silu(lin("gate_proj", n2)) * lin("up_proj", n2))
    return norm(y)


@pytest.mark.parametrize("temperature", [1.0, 2.0])
def test_distilled_block_gradients(temperature):
    from post_quantization_b200 import build
    build.build()
    wl = synth.Workload("tiny", synth._block(256, 128, 512), 256, 2, "none")
    n, seq, hd, seed = 256, 64, 64, 5
    d = synth.Distillation(vocab=1003, top_k=20, temperature=temperature, bits=4)
    losses = torch.empty(n, device="cuda")
    xs, gs = synth.block_calibration(wl, n, seed, device="cuda", seq_len=seq, head_dim=hd,
                                     seqs_per_chunk=2, dtype=torch.float32, distill=d,
                                     losses=losses)
    f32 = torch.float32
    w = {s.name: synth.weight(s.d_out, s.d_in, synth.seed_for(seed, s.name, "W"), dtype=f32,
                              device="cuda") for s in wl.sublayers}
    student = {k: synth.rounded(v, 4).double() for k, v in w.items()}
    w = {k: v.double() for k, v in w.items()}
    head = synth.weight(1003, 256, synth.seed_for(seed, "head"), dtype=f32, device="cuda").double()
    x = synth.correlated_x(n, 256, synth.seed_for(seed, "x"), dtype=f32, device="cuda").double()
    x.requires_grad_(True)
    nb = n // seq
    with torch.no_grad():
        top, ids = (block64(x, w, nb, seq, 4, 2, hd) @ head.t()).topk(20, dim=1)
        logp = torch.log_softmax(top / temperature, 1)
    outs = {}
    u = block64(x, student, nb, seq, 4, 2, hd, outs) @ head.t() / temperature
    kl = (logp.exp() * (logp - torch.log_softmax(u, 1).gather(1, ids))).sum(1)
    loss = temperature ** 2 * kl
    loss.sum().backward()
    assert float((losses.double() - loss).norm() / loss.norm()) <= 1e-3
    for name, out in outs.items():
        assert float((gs[name].double() - out.grad).norm() / out.grad.norm()) <= 1e-3, name
    assert torch.isfinite(xs["down_in"]).all()


def test_distillation_needs_the_gpu():
    wl = synth.Workload("tiny", synth._block(256, 128, 512), 256, 2, "none")
    with pytest.raises(ValueError):
        synth.block_calibration(wl, 256, 1, device="cpu", seq_len=64, head_dim=64,
                                distill=synth.Distillation())
