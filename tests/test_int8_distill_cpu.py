"""Host checks of the 8-bit layer and distillation calls, and pins of their oracle (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import kronq_oracle as O


@pytest.fixture(scope="module")
def K():
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import kronq
    kronq.load_library()
    return kronq


def caller(fn, names, ok):
    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return fn(*a)
    return call


def test_quantize_tokens_refusals(K):
    call = caller(K.load_library().kronq_quantize_tokens,
                  ["x", "dtype", "ld_x", "n", "d", "s_x", "si", "flags", "q", "ld_q", "ts", "sum",
                   "stream"],
                  [256, K.DTYPE_BF16, 64, 2, 64, 512, 768, K.BIIP_SCALE_IN | K.BIIP_ROTATE_IN,
                   1024, 64, 2048, 4096, None])
    assert call(n=0) == K.OK
    assert call(n=-1) == K.ERR_SHAPE and call(d=0) == K.ERR_SHAPE
    assert call(flags=K.BIIP_SCALE_OUT) == K.ERR_INVALID_ARG
    assert call(x=None) == K.ERR_INVALID_ARG and call(x=257) == K.ERR_INVALID_ARG
    assert call(dtype=K.DTYPE_U8) == K.ERR_INVALID_ARG
    assert call(ld_x=63) == K.ERR_SHAPE
    assert call(s_x=None) == K.ERR_INVALID_ARG and call(si=None) == K.ERR_INVALID_ARG
    assert call(d=65537, ld_x=65552, ld_q=65552, flags=0) == K.ERR_UNSUPPORTED
    assert call(d=53249, ld_x=65552, ld_q=65552) == K.ERR_UNSUPPORTED
    assert call(q=1032) == K.ERR_INVALID_ARG and call(q=None) == K.ERR_INVALID_ARG
    assert call(ld_q=72) == K.ERR_INVALID_ARG and call(ld_q=48) == K.ERR_SHAPE
    assert call(ts=None) == K.ERR_INVALID_ARG and call(sum=None) == K.ERR_INVALID_ARG


def test_matmul_i8_refusals(K):
    call = caller(K.load_library().kronq_matmul_i8,
                  ["q", "ld_q", "ts", "sum", "n", "codes", "cd", "ld_c", "scale", "zero", "d_out",
                   "d_in", "y", "yd", "ld_y", "stream"],
                  [256, 64, 512, 768, 2, 1024, K.DTYPE_U8, 64, 2048, 4096, 32, 64, 8192,
                   K.DTYPE_F32, 32, None])
    assert call(n=0) == K.OK
    assert call(n=-1) == K.ERR_SHAPE and call(d_out=0) == K.ERR_SHAPE
    assert call(cd=K.DTYPE_BF16) == K.ERR_INVALID_ARG
    assert call(codes=1032) == K.ERR_INVALID_ARG and call(codes=None) == K.ERR_INVALID_ARG
    assert call(ld_c=72) == K.ERR_INVALID_ARG and call(ld_c=48) == K.ERR_SHAPE
    assert call(ld_q=80, q=264) == K.ERR_INVALID_ARG
    assert call(scale=None) == K.ERR_INVALID_ARG and call(ts=None) == K.ERR_INVALID_ARG
    assert call(sum=None) == K.ERR_INVALID_ARG                 # zero needs the sums
    assert call(d_in=65552, ld_q=65552, ld_c=65552) == K.ERR_UNSUPPORTED
    assert call(y=None) == K.ERR_INVALID_ARG and call(y=8194) == K.ERR_INVALID_ARG
    assert call(yd=K.DTYPE_S8) == K.ERR_INVALID_ARG and call(ld_y=31) == K.ERR_SHAPE


def test_qlinear8_refusals_and_workspace(K):
    size = K.kronq_qlinear8_workspace_size
    assert size(0, 64, 64, 15) == 0 and size(4, 0, 64, 15) == 0
    assert size(1, 64, 60, 0) == 3 * 256                       # q (64 bytes), scales, sums
    assert size(5000, 64, 64, K.BIIP_ROTATE_OUT) == 2048 * 64 + 2 * 8192 + 2048 * 64 * 4
    assert size(1 << 20, 64, 64, 0) == 16384 * 64 + 2 * 65536
    call = caller(K.load_library().kronq_qlinear8,
                  ["x", "xd", "ld_x", "n", "codes", "cd", "ld_c", "scale", "zero", "s_x", "s_g",
                   "si", "so", "flags", "d_out", "d_in", "y", "yd", "ld_y", "ws", "wsb", "stream"],
                  [256, K.DTYPE_BF16, 64, 2, 1024, K.DTYPE_U8, 64, 2048, 4096, 512, 768, 1280, 1536,
                   15, 32, 64, 8192, K.DTYPE_F32, 32, 16384, 1 << 20, None])
    assert call(n=0) == K.OK
    assert call(flags=16) == K.ERR_INVALID_ARG
    for name in ("x", "codes", "scale", "s_x", "s_g", "si", "so", "y"):
        assert call(**{name: None}) == K.ERR_INVALID_ARG, name
    assert call(ws=None) == K.ERR_WORKSPACE and call(wsb=256) == K.ERR_WORKSPACE
    assert call(ws=16385) == K.ERR_WORKSPACE
    assert call(d_out=32768, ld_y=32768) == K.ERR_UNSUPPORTED  # Hadamard block 32768


def distill_call(K):
    return caller(K.load_library().kronq_distill,
                  ["z", "zd", "ld_z", "ids", "ld_i", "top", "td", "ld_t", "n", "v", "k", "tl", "w",
                   "tau", "loss", "lse", "dz", "dd", "ld_d", "stream"],
                  [1 << 20, K.DTYPE_BF16, 100, 256, 8, 512, K.DTYPE_F32, 8, 4, 100, 8, None, None,
                   1.0, 1024, 2048, 1 << 21, K.DTYPE_BF16, 100, None])


def test_distill_refusals(K):
    call = distill_call(K)
    assert call(n=0) == K.OK
    assert call(n=-1) == K.ERR_SHAPE and call(v=0) == K.ERR_SHAPE and call(k=-1) == K.ERR_SHAPE
    assert call(k=1025, ld_i=1025, ld_t=1025) == K.ERR_UNSUPPORTED
    assert call(z=None) == K.ERR_INVALID_ARG and call(z=(1 << 20) + 1) == K.ERR_INVALID_ARG
    assert call(zd=K.DTYPE_U8) == K.ERR_INVALID_ARG and call(ld_z=99) == K.ERR_SHAPE
    assert call(ids=None) == K.ERR_INVALID_ARG and call(top=None) == K.ERR_INVALID_ARG
    assert call(ld_i=7) == K.ERR_SHAPE and call(ld_t=7) == K.ERR_SHAPE
    for tau in (0.0, -1.0, 1e5, float("nan"), float("inf")):
        assert call(tau=tau) == K.ERR_INVALID_ARG
    assert call(loss=None) == K.ERR_INVALID_ARG
    assert call(dd=K.DTYPE_S8) == K.ERR_INVALID_ARG and call(ld_d=99) == K.ERR_SHAPE
    # dlogits may be logits itself, and nothing in between
    assert call(dz=1 << 20, dd=K.DTYPE_F32) == K.ERR_INVALID_ARG
    assert call(dz=1 << 20, ld_d=108) == K.ERR_INVALID_ARG
    assert call(dz=(1 << 20) + 2) == K.ERR_INVALID_ARG
    assert call(dz=(1 << 20) - 798) == K.ERR_INVALID_ARG
    back = K.load_library().kronq_distill_backward
    base = [1 << 20, K.DTYPE_BF16, 100, 256, 8, 512, K.DTYPE_F32, 8, 4, 100, 8, None, 1024, 2048,
            1.0, 1 << 21, K.DTYPE_BF16, 100, None]
    for i in (12, 13, 15):                                     # lse, dloss, dlogits
        a = list(base)
        a[i] = None
        assert back(*a) == K.ERR_INVALID_ARG
    base[8] = 0
    assert back(*base) == K.OK


def test_binding_checks(K):
    f = torch.zeros
    with pytest.raises(ValueError):                            # wrong code type
        K.kronq_quantize_tokens(f(2, 16), f(2, 16), f(2), f(2, dtype=torch.int32))
    with pytest.raises(ValueError):                            # wrong scale length
        K.kronq_quantize_tokens(f(2, 16), f(2, 16, dtype=torch.int8), f(3), f(2, dtype=torch.int32))
    with pytest.raises(ValueError):                            # fp16 input
        K.kronq_quantize_tokens(f(2, 16).half(), f(2, 16, dtype=torch.int8), f(2),
                                f(2, dtype=torch.int32))
    c = f(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):                            # widths differ
        K.kronq_matmul_i8(f(2, 32, dtype=torch.int8), f(2), f(2, dtype=torch.int32), c, f(4), f(4),
                          f(2, 4))
    with pytest.raises(ValueError):                            # transposed output
        K.kronq_matmul_i8(f(2, 16, dtype=torch.int8), f(2), f(2, dtype=torch.int32), c, f(4), f(4),
                          f(4, 2).t())
    with pytest.raises(ValueError):                            # 64-bit ids
        K.kronq_distill(f(2, 9), f(2, 3, dtype=torch.int64), f(2, 3), f(2))
    with pytest.raises(ValueError):                            # ids and logits of different k
        K.kronq_distill(f(2, 9), f(2, 3, dtype=torch.int32), f(2, 4), f(2))


def test_linear8_lays_codes_out_once():
    from post_quantization_b200 import pipeline as P
    c = torch.randint(0, 256, (5, 37), dtype=torch.uint8)
    rows = P.byte_rows(c)
    assert torch.equal(rows, c) and rows.stride(0) == 48 and rows.data_ptr() % 16 == 0
    c16 = torch.zeros(5, 64, dtype=torch.uint8)
    assert P.byte_rows(c16) is c16
    with pytest.raises(ValueError):                            # a grid per group of columns
        P.Linear8(c, torch.ones(5, 1), torch.zeros(5, 1))


# --------------------------------------------------------------------------- oracle pins

def test_oracle_quantize_tokens_by_hand():
    x = np.array([[127.0, 0.5, 1.5, -2.5], [0.0, 0.0, 0.0, 0.0], [1.0, np.inf, 0.0, 0.0]])
    _, s, q, total = O.quantize_tokens(x)
    assert s[0] == 1.0 and q[0].tolist() == [127, 0, 2, -2] and total[0] == 127
    assert s[1] == 1.0 and not q[1].any() and math.isnan(s[2]) and not q[2].any()


def test_oracle_hadamard_rows_is_the_matrix():
    import scipy.linalg as sla
    r = np.random.default_rng(2)
    x = r.normal(size=(3, 24))
    h = np.kron(np.eye(3), sla.hadamard(8) / math.sqrt(8))
    np.testing.assert_allclose(O.hadamard_rows(x), x @ h.T, atol=1e-14)


def test_oracle_distill_closed_forms():
    # uniform student over v, teacher certain of one entry: loss = log v; gradient 1/v - [v = id]
    z = np.zeros((1, 10))
    loss, lse, g = O.distill(z, np.array([[3, -1]]), np.array([[5.0, 1.0]]))
    assert abs(loss[0] - math.log(10)) < 1e-15 and abs(lse[0] - math.log(10)) < 1e-15
    want = np.full(10, 0.1)
    want[3] -= 1
    np.testing.assert_allclose(g[0], want, atol=1e-15)
    # the student equal to the teacher over the whole vocabulary: loss 0 and gradient 0
    t = np.array([[0.3, -1.0, 2.0]])
    loss, _, g = O.distill(t, np.array([[0, 1, 2]]), t, tau=2.0)
    assert abs(loss[0]) < 1e-15 and np.abs(g).max() < 1e-15
    # an entry listed twice: the gradient is that of the loss
    r = np.random.default_rng(4)
    z, ids, t = r.normal(size=(1, 6)), np.array([[2, 2, 5]]), r.normal(size=(1, 3))
    _, _, g = O.distill(z, ids, t, 1.5, weight=[0.7])
    for v in range(6):
        e = np.zeros((1, 6))
        e[0, v] = 1e-6
        up, dn = O.distill(z + e, ids, t, 1.5, weight=[0.7]), O.distill(z - e, ids, t, 1.5,
                                                                        weight=[0.7])
        assert abs((up[0][0] - dn[0][0]) / 2e-6 - g[0, v]) < 1e-8
