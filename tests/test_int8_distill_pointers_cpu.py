"""Pointers and sizes that the kernels of the 8-bit layer and of distillation could not take are refused on
the host (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def K():
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import kronq
    kronq.load_library()
    return kronq


def calls(K):
    """(function, argument names, arguments that only a missing GPU would refuse, its 4-byte vectors)"""
    lib = K.load_library()
    return {
        "quantize_tokens": (
            lib.kronq_quantize_tokens,
            ["x", "dtype", "ld_x", "n", "d", "s_x", "si", "flags", "q", "ld_q", "ts", "sum", "stream"],
            [256, K.DTYPE_BF16, 64, 2, 64, 512, 768, K.BIIP_SCALE_IN | K.BIIP_ROTATE_IN, 1024, 64, 2048,
             4096, None], ["s_x", "ts", "sum"]),
        "matmul_i8": (
            lib.kronq_matmul_i8,
            ["q", "ld_q", "ts", "sum", "n", "codes", "cd", "ld_c", "scale", "zero", "d_out", "d_in", "y",
             "yd", "ld_y", "stream"],
            [256, 64, 512, 768, 2, 1024, K.DTYPE_U8, 64, 2048, 4096, 32, 64, 8192, K.DTYPE_F32, 32, None],
            ["ts", "sum", "scale", "zero"]),
        "qlinear8": (
            lib.kronq_qlinear8,
            ["x", "xd", "ld_x", "n", "codes", "cd", "ld_c", "scale", "zero", "s_x", "s_g", "si", "so",
             "flags", "d_out", "d_in", "y", "yd", "ld_y", "ws", "wsb", "stream"],
            [256, K.DTYPE_BF16, 64, 2, 1024, K.DTYPE_U8, 64, 2048, 4096, 512, 768, 1280, 1536, 15, 32, 64,
             8192, K.DTYPE_F32, 32, 16384, 1 << 20, None], ["scale", "zero", "s_x", "s_g"]),
        "distill": (
            lib.kronq_distill,
            ["z", "zd", "ld_z", "ids", "ld_i", "top", "td", "ld_t", "n", "v", "k", "tl", "w", "tau",
             "loss", "lse", "dz", "dd", "ld_d", "stream"],
            [1 << 20, K.DTYPE_BF16, 100, 256, 8, 512, K.DTYPE_BF16, 8, 4, 100, 8, 4096, 8192, 1.0, 1024,
             2048, 1 << 21, K.DTYPE_BF16, 100, None], ["ids", "tl", "w", "loss", "lse"]),
        "distill_backward": (
            lib.kronq_distill_backward,
            ["z", "zd", "ld_z", "ids", "ld_i", "top", "td", "ld_t", "n", "v", "k", "tl", "lse", "dloss",
             "tau", "dz", "dd", "ld_d", "stream"],
            [1 << 20, K.DTYPE_BF16, 100, 256, 8, 512, K.DTYPE_BF16, 8, 4, 100, 8, 4096, 1024, 2048, 1.0,
             1 << 21, K.DTYPE_BF16, 100, None], ["ids", "tl", "lse", "dloss"]),
    }


def status(call, **changed):
    fn, names, ok, _ = call
    return fn(*(changed.get(n, a) for n, a in zip(names, ok)))


@pytest.mark.parametrize("name", ["quantize_tokens", "matmul_i8", "qlinear8", "distill",
                                  "distill_backward"])
def test_vectors_off_alignment(K, name):
    call = calls(K)[name]
    for vector in call[3]:
        at = call[2][call[1].index(vector)]
        for off in (1, 2, 3):
            assert status(call, **{vector: at + off}) == K.ERR_INVALID_ARG, (vector, off)


@pytest.mark.parametrize("name", ["matmul_i8", "qlinear8"])
def test_sizes_whose_last_tile_passes_32_bits(K, name):
    """A tile of 256 channels or tokens from there on would end past 2^31 - 1."""
    call = calls(K)[name]
    most = 2 ** 31 - 256
    wide = {"ld_y": 2 ** 31, "wsb": 2 ** 62, "flags": 0}
    tokens = [] if name == "qlinear8" else [(32, most + 1), (32, 2 ** 31 - 1)]   # that takes passes
    for d_out, n in [(most + 1, 2), (2 ** 31 - 1, 2)] + tokens:
        changed = {k: v for k, v in {**wide, "d_out": d_out, "n": n}.items() if k in call[1]}
        assert status(call, **changed) == K.ERR_UNSUPPORTED, (d_out, n)
