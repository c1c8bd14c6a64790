"""Performance cases of the 8-bit layer and distillation operators.

The operators are the integer path of a quantized layer (token quantization, the 8-bit matrix
product, the whole layer with its incoherence transforms) and the distillation loss from a
teacher's top logits with its gradient. `run` computes a case either in elementary torch
operations (`own` false) or through the library's public calls (`own` true); `exact` computes the
same outputs in 64 bits, written apart from both.
"""
import math

import torch

own = False

# transform flags of the library's layer calls
SCALE_IN, SCALE_OUT, ROTATE_IN, ROTATE_OUT = 1, 2, 4, 8
FULL = 15


def listed():
    return [
        # one token through a square attention projection: the weights' read is all there is
        dict(name="matmul_1x8192x8192", op="matmul", n=1, d_out=8192, d_in=8192, signed=False,
             y="f32"),
        # a decode batch through a narrow key/value projection: latency
        dict(name="matmul_16x1024x8192", op="matmul", n=16, d_out=1024, d_in=8192, signed=False,
             y="bf16"),
        # a short ragged prompt, symmetric weights, odd sizes on every side
        dict(name="matmul_333x1001x11008", op="matmul", n=333, d_out=1001, d_in=11008,
             signed=True, y="f32"),
        # a prompt chunk through the widest layer of the largest block
        dict(name="matmul_4096x28672x8192", op="matmul", n=4096, d_out=28672, d_in=8192,
             signed=False, y="bf16"),
        # a decode batch's activations into an 8192-wide layer, with its input transforms
        dict(name="quantize_32x8192_rotated", op="quantize", n=32, d=8192, flags=SCALE_IN |
             ROTATE_IN, x="bf16"),
        # a prompt's activations into a layer without transforms, ragged width
        dict(name="quantize_4096x11000", op="quantize", n=4096, d=11000, flags=0, x="bf16"),
        # the whole layer for one token: three launches' latency beside the weights' read
        dict(name="layer_1x4096x11008", op="layer", n=1, d_out=4096, d_in=11008, flags=FULL,
             x="bf16"),
        # the whole layer for a prompt chunk
        dict(name="layer_2048x8192x8192", op="layer", n=2048, d_out=8192, d_in=8192, flags=FULL,
             x="bf16"),
        # evaluation of a quantized model against its teacher: the loss alone
        dict(name="distill_2048x32000_loss", op="distill", mode="loss", n=2048, v=32000, k=64,
             dtype="bf16", tau=1.0, ragged=False, mass=False),
        # a small calibration batch, a vocabulary of odd size (rows off alignment), ragged lists
        dict(name="distill_96x50001_grad", op="distill", mode="grad", n=96, v=50001, k=20,
             dtype="bf16", tau=2.0, ragged=True, mass=True),
        # a calibration batch over a large vocabulary: loss and gradient of the logits
        dict(name="distill_4096x128256_grad", op="distill", mode="grad", n=4096, v=128256, k=128,
             dtype="bf16", tau=1.0, ragged=False, mass=False),
        # the backward pass on its own, in fp32, upstream gradient per row
        dict(name="distill_1024x32000_backward", op="distill", mode="backward", n=1024, v=32000,
             k=64, dtype="f32", tau=1.5, ragged=True, mass=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer width: any number, or one with a power-of-two factor as layers have."""
    d = _log(rng, lo, hi)
    if rng.random() < 0.6:
        p = 1 << rng.randint(4, 10)
        d = max(p, d // p * p)
    return d


def draw(rng):
    op = rng.choice(["matmul", "matmul", "quantize", "layer", "distill", "distill"])
    if op == "matmul":
        d_out, d_in = _width(rng, 64, 28672), _width(rng, 64, 28672)
        most = max(1, min(4096, 4096 * 28672 * 8192 // (d_out * d_in)))
        return dict(op=op, n=_log(rng, 1, most), d_out=d_out, d_in=d_in,
                    signed=rng.random() < 0.5, y=rng.choice(["f32", "bf16"]))
    if op == "quantize":
        d = _width(rng, 64, 28672)
        return dict(op=op, n=_log(rng, 1, min(16384, (1 << 27) // d)), d=d,
                    flags=rng.choice([0, SCALE_IN, SCALE_IN | ROTATE_IN]),
                    x=rng.choice(["bf16", "f32"]))
    if op == "layer":
        d_out, d_in = _width(rng, 64, 16384), _width(rng, 64, 16384)
        return dict(op=op, n=_log(rng, 1, 2048), d_out=d_out, d_in=d_in,
                    flags=rng.choice([FULL, SCALE_IN | ROTATE_IN, SCALE_OUT]), x="bf16")
    v = _log(rng, 1000, 131072)
    return dict(op=op, mode=rng.choice(["loss", "grad", "backward"]),
                n=_log(rng, 1, min(4096, (1 << 28) // v)), v=v, k=_log(rng, 1, 256),
                dtype=rng.choice(["bf16", "f32"]), tau=rng.choice([1.0, 1.5, 2.0, 4.0]),
                ragged=rng.random() < 0.5, mass=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "matmul":
        n, do, di = case["n"], case["d_out"], case["d_in"]
        return {"bytes": n * di + do * di + n * do * _size(case["y"]) + 8 * (n + do),
                "flops": 2.0 * n * do * di}
    if op == "quantize":
        n, d = case["n"], case["d"]
        extra = (4 * d if case["flags"] & SCALE_IN else 0) + (d if case["flags"] & ROTATE_IN else 0)
        b = d & -d if case["flags"] & ROTATE_IN else 1
        return {"bytes": n * d * (_size(case["x"]) + 1) + 8 * n + extra,
                "flops": n * d * (3.0 + math.log2(b))}
    if op == "layer":
        n, do, di = case["n"], case["d_out"], case["d_in"]
        return {"bytes": n * di * 2 + do * di + n * do * 2 + 8 * do + 5 * (di + do),
                "flops": 2.0 * n * do * di}
    n, v, k, b = case["n"], case["v"], case["k"], _size(case["dtype"])
    reads = n * v * b + n * k * (4 + b) + 12 * n
    return {"bytes": reads if case["mode"] == "loss" else reads + n * v * b, "flops": 5.0 * n * v}


# ------------------------------------------------------------------------------------ inputs

def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _dtype(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(n, d, g, dtype):
    """Normal activations with a few outlier channels, as layer inputs have."""
    x = torch.randn(n, d, generator=g, device="cuda")
    x[:, torch.randint(0, d, (4,), generator=g, device="cuda")] *= 20.0
    return x.to(dtype)


def _padded(rows, cols, dtype):
    """rows x cols with a row stride of a multiple of 16 bytes, as the 8-bit calls want it."""
    return torch.zeros(rows, (cols + 15) // 16 * 16, dtype=dtype, device="cuda")[:, :cols]


def _weights(d_out, d_in, signed, g):
    """8-bit codes of normal weights, one grid per output row."""
    codes = _padded(d_out, d_in, torch.int8 if signed else torch.uint8)
    w = torch.randn(d_out, d_in, generator=g, device="cuda") * 0.02
    if signed:
        scale = w.abs().amax(1) / 127
        zero = None
        codes.copy_((w / scale[:, None]).round_())
    else:
        lo, hi = w.amin(1), w.amax(1)
        scale = (hi - lo) / 255
        zero = (-lo / scale).round()
        codes.copy_(((w / scale[:, None]).round_() + zero[:, None]).clamp_(0, 255))
    return codes, scale, zero


def _positive(d, g):
    return torch.exp(torch.rand(d, generator=g, device="cuda") * 2.0 - 1.0)


def _signs(d, g):
    return (torch.randint(0, 2, (d,), generator=g, device="cuda") * 2 - 1).to(torch.int8)


def _hadamard(d, dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _factors(d, dtype):
    """Hadamard matrices H_a, H_b with a b = the largest power of two in d."""
    b = d & -d
    b1 = 1 << ((b.bit_length() - 1) // 2)
    return _hadamard(b1, dtype), _hadamard(b // b1, dtype)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "quantize":
        n, d = case["n"], case["d"]
        s["x"] = _activations(n, d, g, _dtype(case["x"]))
        s["s_x"] = _positive(d, g) if case["flags"] & SCALE_IN else None
        s["sign_in"] = _signs(d, g) if case["flags"] & ROTATE_IN else None
        s["h_in"] = _factors(d, torch.float64)
        s["q"] = _padded(n, d, torch.int8)
        s["tok_scale"] = torch.empty(n, device="cuda")
        s["tok_sum"] = torch.empty(n, dtype=torch.int32, device="cuda")
    elif op == "matmul":
        n, do, di = case["n"], case["d_out"], case["d_in"]
        x = _activations(n, di, g, torch.float32)
        s["codes"], s["scale"], s["zero"] = _weights(do, di, case["signed"], g)
        s["tok_scale"] = x.abs().amax(1) / 127
        q = (x / s["tok_scale"][:, None]).round_().clamp_(-127, 127)
        s["q"] = _padded(n, di, torch.int8)
        s["q"].copy_(q)
        s["tok_sum"] = q.sum(1, dtype=torch.float64).to(torch.int32)
        s["y"] = torch.empty(n, do, dtype=_dtype(case["y"]), device="cuda")
    elif op == "layer":
        n, do, di, fl = case["n"], case["d_out"], case["d_in"], case["flags"]
        s["x"] = _activations(n, di, g, torch.bfloat16)
        s["codes"], s["scale"], s["zero"] = _weights(do, di, False, g)
        s["s_x"] = _positive(di, g) if fl & SCALE_IN else None
        s["s_g"] = _positive(do, g) if fl & SCALE_OUT else None
        s["sign_in"] = _signs(di, g) if fl & ROTATE_IN else None
        s["sign_out"] = _signs(do, g) if fl & ROTATE_OUT else None
        s["h_in"], s["h_out"] = _factors(di, torch.float64), _factors(do, torch.float32)
        s["y"] = torch.empty(n, do, dtype=torch.bfloat16, device="cuda")
        s["ws"] = {}                       # the program's workspace, made at its first pass
    else:
        n, v, k, dt = case["n"], case["v"], case["k"], _dtype(case["dtype"])
        tau = case["tau"]
        z = torch.empty(n, v, dtype=dt, device="cuda")
        for r0 in range(0, n, 1024):
            z[r0:r0 + 1024] = torch.randn(min(1024, n - r0), v, generator=g, device="cuda") * 2.0
        z[:, v - max(1, v // 100):] = float("-inf")      # the vocabulary's padding
        # k distinct entries of a row: an arithmetic progression modulo the unpadded vocabulary
        u = v - max(1, v // 100)
        start = torch.randint(0, u, (n, 1), generator=g, device="cuda")
        step = torch.randint(1, max(2, u // k), (n, 1), generator=g, device="cuda")
        j = torch.arange(k, device="cuda")[None, :]
        ids = (start + j * step) % u
        # the teacher's logits fall off from the top; the student is near them
        t = 12.0 - 2.0 * torch.log1p(j.float()) + 0.5 * torch.randn(n, k, generator=g, device="cuda")
        z.scatter_(1, ids, (t + 0.7 * torch.randn(n, k, generator=g, device="cuda")).to(dt))
        t = t.to(dt)
        ids = ids.to(torch.int32)
        if case["ragged"]:                 # lists of different lengths; some rows have none
            length = torch.randint(0, k + 1, (n, 1), generator=g, device="cuda")
            ids = torch.where(j < length, ids, -1).to(torch.int32)
        s["z"], s["ids"], s["t"] = z, ids.contiguous(), t.contiguous()
        # the teacher's full log-sum: a little more than its top logits'
        s["top_lse"] = (torch.logsumexp(t.double() / tau, 1) + 0.05).float() if case["mass"] else None
        w = torch.rand(n, generator=g, device="cuda") + 0.5
        w[torch.rand(n, generator=g, device="cuda") < 0.1] = 0.0       # prompt tokens count nothing
        s["weight"] = w
        s["loss"] = torch.empty(n, device="cuda")
        s["lse"] = torch.empty(n, device="cuda")
        if case["mode"] != "loss":
            s["dz"] = torch.empty(n, v, dtype=dt, device="cuda")
        if case["mode"] == "backward":
            for r0 in range(0, n, 1024):
                s["lse"][r0:r0 + 1024] = torch.logsumexp(z[r0:r0 + 1024].double() / tau, 1).float()
    return s


# -------------------------------------------------------------------------------- plain forms

def _transform(x, factors):
    """Orthonormal Walsh-Hadamard transform of every aligned block of the largest power of two
    in the width, as two matrix products: H_ab = H_a (x) H_b."""
    h1, h2 = factors
    v = x.reshape(x.shape[0], -1, h1.shape[0], h2.shape[0])
    v = h1 @ (v @ h2)
    return v.reshape(x.shape) / math.sqrt(h1.shape[0] * h2.shape[0])


def _input_side(x, s_x, sign_in, factors):
    """V S_X^-1 x; in 64 bits where it is rotated, as its results are rounded to whole codes."""
    x = x.float() if sign_in is None else x.double()
    if s_x is not None:
        x = x / s_x.to(x.dtype)
    if sign_in is not None:
        x = _transform(x * sign_in.to(x.dtype), factors)
    return x


def _plain_quantize(x):
    """(codes, scale, sum): the codes are whole numbers, taken in 64 bits next to a border."""
    scale = (x.abs().amax(1).double() / 127).float()
    scale = torch.where(scale < 2.0 ** -126, 1.0, scale)
    q = (x.double() / scale.double()[:, None]).round_()
    return q, scale, q.sum(1).to(torch.int32)


def _plain_matmul(q, tok_scale, codes, scale, zero):
    c = codes.float()
    if zero is not None:
        c = c - zero[:, None]
    return (q.float() @ c.t()) * (tok_scale[:, None] * scale[None, :])


def _plain_distill(s, c, want_loss, want_grad):
    tau = c["tau"]
    ids, mode = s["ids"], c["mode"]
    there = ids >= 0
    at = ids.clamp(min=0).long()
    z = s["z"].float() / tau
    t = torch.where(there, s["t"].float() / tau, -math.inf)
    if mode == "backward":
        lse = s["lse"]
    else:
        m = z.amax(1, keepdim=True)
        lse = (m + (z - m).exp_().sum(1, keepdim=True).log())[:, 0]
    if s["top_lse"] is None:
        m = t.amax(1, keepdim=True).clamp(min=-1e30)
        e = (t - m).exp()
        p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        p = (t - s["top_lse"][:, None]).exp()
    out = []
    if want_loss:
        zk = z.gather(1, at).double()
        terms = torch.where(p > 0, p.double() * (p.double().log() - zk + lse.double()[:, None]), 0.0)
        out += [(s["weight"].double() * tau * tau * terms.sum(1)).float(), lse]
    if want_grad:
        w = (s["weight"] * tau)[:, None]
        mass = p.sum(1, keepdim=True)
        d = (z - lse[:, None]).exp_() * (w * mass)
        d.scatter_add_(1, at, -w * p)
        out.append(d.to(s["z"].dtype))
    return out


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        q, scale, total = _plain_quantize(_input_side(s["x"], s["s_x"], s["sign_in"], s["h_in"]))
        return {"values": (q * scale.double()[:, None]).to(torch.bfloat16), "scale": scale}
    if op == "matmul":
        y = _plain_matmul(s["q"], s["tok_scale"], s["codes"], s["scale"], s["zero"])
        return y.to(s["y"].dtype)
    if op == "layer":
        q, scale, _ = _plain_quantize(_input_side(s["x"], s["s_x"], s["sign_in"], s["h_in"]))
        y = _plain_matmul(q, scale, s["codes"], s["scale"], s["zero"])
        if s["sign_out"] is not None:
            y = _transform(y, s["h_out"]) * s["sign_out"].float()
        if s["s_g"] is not None:
            y = y / s["s_g"]
        return y.to(torch.bfloat16)
    return _plain_distill(s, c, c["mode"] != "backward", c["mode"] != "loss")


# ------------------------------------------------------------------------- the library's calls

def _library(s):
    from post_quantization_b200 import kronq as K
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        K.kronq_quantize_tokens(s["x"], s["q"], s["tok_scale"], s["tok_sum"], s_x=s["s_x"],
                                sign_in=s["sign_in"], flags=c["flags"])
        # 8-bit codes are returned as the values they stand for
        return {"values": (s["q"] * s["tok_scale"][:, None]).to(torch.bfloat16),
                "scale": s["tok_scale"]}
    if op == "matmul":
        K.kronq_matmul_i8(s["q"], s["tok_scale"], s["tok_sum"], s["codes"], s["scale"], s["zero"],
                          s["y"])
        return s["y"]
    if op == "layer":
        if "buf" not in s["ws"]:
            size = K.kronq_qlinear8_workspace_size(c["n"], c["d_out"], c["d_in"], c["flags"])
            buf = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
            off = -buf.data_ptr() % 256
            s["ws"]["buf"] = buf[off:off + size]
        K.kronq_qlinear8(s["x"], s["codes"], s["scale"], s["zero"], s["s_x"], s["s_g"],
                         s["sign_in"], s["sign_out"], c["flags"], s["y"],
                         workspace=s["ws"]["buf"])
        return s["y"]
    if c["mode"] == "backward":
        K.kronq_distill_backward(s["z"], s["ids"], s["t"], s["lse"], s["weight"], s["dz"],
                                 top_lse=s["top_lse"], temperature=c["tau"])
        return [s["dz"]]
    dz = s["dz"] if c["mode"] == "grad" else None
    K.kronq_distill(s["z"], s["ids"], s["t"], s["loss"], s["lse"], dlogits=dz,
                    top_lse=s["top_lse"], row_weight=s["weight"], temperature=c["tau"])
    return [s["loss"], s["lse"]] + ([dz] if dz is not None else [])


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------------------------------- 64-bit definition

def _butterfly(x):
    """Walsh-Hadamard transform of the last axis by butterflies, orthonormal."""
    b = x.shape[-1]
    h = 1
    while h < b:
        v = x.reshape(*x.shape[:-1], b // (2 * h), 2, h)
        x = torch.stack([v[..., 0, :] + v[..., 1, :], v[..., 0, :] - v[..., 1, :]], -2)
        x = x.reshape(*x.shape[:-3], b)
        h *= 2
    return x / math.sqrt(b)


def _exact_quantize(x, s_x, sign_in):
    x = x.double()
    if s_x is not None:
        # without a rotation the quotient is an fp32 value of the definition
        x = x / s_x.double() if sign_in is not None else (x / s_x.double()).float().double()
    if sign_in is not None:
        d = x.shape[1]
        x = _butterfly((x * sign_in.double()).reshape(x.shape[0], d // (d & -d), d & -d))
        x = x.reshape(-1, d)
    step = (x.abs().max(dim=1).values / 127).float().double()
    step[step < 2.0 ** -126] = 1.0
    return torch.round(x / step.unsqueeze(1)), step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, step = _exact_quantize(s["x"], s["s_x"], s["sign_in"])
        return {"values": q * step.unsqueeze(1), "scale": step}
    if op in ("matmul", "layer"):
        if op == "matmul":
            q, step = s["q"].double(), s["tok_scale"].double()
        else:
            q, step = _exact_quantize(s["x"], s["s_x"], s["sign_in"])
        w = s["codes"].double()
        if s["zero"] is not None:
            w -= s["zero"].double().unsqueeze(1)
        w *= s["scale"].double().unsqueeze(1)
        y = torch.mm(q * step.unsqueeze(1), w.t())
        if op == "layer":
            if s["sign_out"] is not None:
                d = y.shape[1]
                y = _butterfly(y.reshape(-1, d // (d & -d), d & -d)).reshape(-1, d)
                y = y * s["sign_out"].double()
            if s["s_g"] is not None:
                y = y / s["s_g"].double()
        return y
    tau, n = case["tau"], case["n"]
    loss = torch.empty(n, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, dtype=torch.float64, device="cuda")
    grad = None if case["mode"] == "loss" else torch.empty(n, case["v"], dtype=torch.float64,
                                                           device="cuda")
    for r0 in range(0, n, 512):
        rows = slice(r0, min(n, r0 + 512))
        z = s["z"][rows].double() / tau
        there = s["ids"][rows] >= 0
        at = s["ids"][rows].long().clamp(min=0)
        lz = s["lse"][rows].double() if case["mode"] == "backward" else torch.logsumexp(z, 1)
        t = (s["t"][rows].double() / tau).masked_fill(~there, -math.inf)
        lt = torch.logsumexp(t, 1) if s["top_lse"] is None else s["top_lse"][rows].double()
        logp = (t - lt.unsqueeze(1)).masked_fill(~there, -math.inf)
        p = torch.exp(logp)
        logq = torch.gather(z, 1, at) - lz.unsqueeze(1)
        w = s["weight"][rows].double()
        lse[rows] = lz
        loss[rows] = tau ** 2 * w * (p * (logp - logq)).masked_fill(~there, 0.0).sum(1)
        if grad is not None:
            q = torch.exp(z - lz.unsqueeze(1)) * p.sum(1).unsqueeze(1)
            target = torch.zeros_like(q).scatter_add_(1, at, p)
            grad[rows] = tau * w.unsqueeze(1) * (q - target)
    if case["mode"] == "backward":
        return [grad]
    return [loss, lse] + ([grad] if grad is not None else [])
