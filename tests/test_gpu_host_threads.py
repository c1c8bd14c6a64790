"""Calls of the 8-bit layer and of distillation from several host threads at once, each on a stream of its
own: the results of one call after the other, whatever sizes the other threads' calls have."""
import threading

import pytest
import torch

from post_quantization_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import kronq
    kronq.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kronq.kronq_device_check()
    return kronq


def side_by_side(K, jobs, rounds):
    """Makes every job's C call `rounds` times in a thread of its own. job: (function, its arguments
    with the stream last). The arguments are ready, so that the threads spend their time in the calls."""
    failed = []
    start = threading.Barrier(len(jobs))
    streams = [torch.cuda.Stream() for _ in jobs]

    def loop(fn, args, stream):
        args = args + (stream.cuda_stream,)
        start.wait()
        for i in range(rounds):
            if fn(*args) != K.OK:
                failed.append((i, K.load_library().kronq_last_error_detail().decode()))
                break
            if i % 64 == 63:
                stream.synchronize()

    threads = [threading.Thread(target=loop, args=(*j, s)) for j, s in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_tokens_of_several_widths(K):
    """Widths whose rows take different amounts of shared memory of one kernel."""
    fn = K.load_library().kronq_quantize_tokens
    got, want, jobs, keep = [], [], [], []
    for d in (28672, 20480, 45056, 53248):
        x = synth.activations(2, d, synth.seed_for("threads", d), dtype=torch.bfloat16, device="cuda")
        si = synth.rademacher(d, synth.seed_for("threads", d, "si"), device="cuda")
        outs = [(torch.zeros(2, d, dtype=torch.int8, device="cuda"), torch.zeros(2, device="cuda"),
                 torch.zeros(2, dtype=torch.int32, device="cuda")) for _ in range(2)]
        K.kronq_quantize_tokens(x, *outs[0], sign_in=si, flags=K.BIIP_ROTATE_IN)
        want.append(outs[0])
        got.append(outs[1])
        q, scale, total = outs[1]
        keep.append((x, si))
        jobs.append((fn, (x.data_ptr(), K.DTYPE_BF16, d, 2, d, None, si.data_ptr(), K.BIIP_ROTATE_IN,
                          q.data_ptr(), d, scale.data_ptr(), total.data_ptr())))
    torch.cuda.synchronize()
    side_by_side(K, jobs, 20000)
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


def test_lists_of_several_lengths(K):
    """List lengths whose tables take different amounts of shared memory beside the rows."""
    fn = K.load_library().kronq_distill
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n, v = 600, 20011
    z = torch.randn(n, v, generator=g, device="cuda").to(torch.bfloat16)
    got, want, jobs, keep = [], [], [], []
    for k in (4, 60, 120, 200):
        ids = torch.randint(0, v, (n, k), generator=g, device="cuda").to(torch.int32)
        t = torch.randn(n, k, generator=g, device="cuda")
        outs = [(torch.zeros(n, device="cuda"), torch.zeros_like(z)) for _ in range(2)]
        K.kronq_distill(z, ids, t, outs[0][0], dlogits=outs[0][1])
        want.append(outs[0])
        got.append(outs[1])
        loss, dz = outs[1]
        keep.append((ids, t))
        jobs.append((fn, (z.data_ptr(), K.DTYPE_BF16, v, ids.data_ptr(), k, t.data_ptr(), K.DTYPE_F32,
                          k, n, v, k, None, None, 1.0, loss.data_ptr(), None, dz.data_ptr(),
                          K.DTYPE_BF16, v)))
    torch.cuda.synchronize()
    side_by_side(K, jobs, 4000)
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


def test_packed_layers_of_several_widths(K):
    """kronq_qlinear: its kernels' shared memory goes by the layer's width and the token count."""
    fn = K.load_library().kronq_qlinear
    got, want, jobs, keep = [], [], [], []
    for d_in, n in ((1024, 1), (4096, 4), (8192, 2), (11008, 3), (2048, 8), (28672, 1)):
        d_out, tag = 256, ("threads", d_in)
        packed = K.kronq_pack_codes(synth.codes(d_out, d_in, 2, synth.seed_for(tag, "c"), device="cuda"), 2)
        scale, zero = synth.grid_params(d_out, 0, 2, synth.seed_for(tag, "g"), device="cuda")
        grid = K.kronq_pack_grid(scale, zero, d_out, d_in, 0)
        s_x = synth.positive_scales(d_in, synth.seed_for(tag, "sx"), device="cuda")
        s_g = synth.positive_scales(d_out, synth.seed_for(tag, "sg"), device="cuda")
        si = synth.rademacher(d_in, synth.seed_for(tag, "si"), device="cuda")
        so = synth.rademacher(d_out, synth.seed_for(tag, "so"), device="cuda")
        x = synth.activations(n, d_in, synth.seed_for(tag, "x"), dtype=torch.bfloat16, device="cuda")
        ys = [torch.zeros(n, d_out, device="cuda") for _ in range(2)]
        K.kronq_qlinear(x, packed, grid, s_x, s_g, si, so, K.BIIP_FULL, d_out, 2, ys[0])
        want.append(ys[0])
        got.append(ys[1])
        size = K.kronq_qlinear_workspace_size(d_out, d_in, n)
        ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
        ws = ws[-ws.data_ptr() % 256:][:size]
        keep.append((packed, grid, s_x, s_g, si, so, x, ws))
        jobs.append((fn, (x.data_ptr(), K.DTYPE_BF16, d_in, n, packed.data_ptr(), grid.data_ptr(), 0,
                          s_x.data_ptr(), s_g.data_ptr(), si.data_ptr(), so.data_ptr(), K.BIIP_FULL,
                          d_out, d_in, 2, ys[1].data_ptr(), d_out, ws.data_ptr(), size)))
    torch.cuda.synchronize()
    side_by_side(K, jobs, 4000)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
