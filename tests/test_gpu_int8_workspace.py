"""A captured 8-bit layer whose workspace grows afterwards: replays give the same bits and touch nothing
that was allocated since."""
import pytest
import torch

from post_quantization_b200 import synth

pytestmark = pytest.mark.gpu


def test_replay_after_the_workspace_has_grown():
    from post_quantization_b200 import build
    build.build()
    from post_quantization_b200 import pipeline as P
    d, n = 512, 40
    codes = synth.codes(d, d, 8, 1, device="cuda")
    scale, zero = synth.grid_params(d, 0, 8, 2, device="cuda")
    layer = P.Linear8(codes, scale, zero, sign_in=synth.rademacher(d, 3, device="cuda"),
                      sign_out=synth.rademacher(d, 4, device="cuda"))
    x = synth.activations(n, d, 5, dtype=torch.bfloat16, device="cuda")
    large = synth.activations(50 * n, d, 6, dtype=torch.bfloat16, device="cuda")
    ws = P.Workspace("cuda")
    y = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    layer(x, y=y, ws=ws)
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, y=y, ws=ws)
    layer(large, ws=ws)
    torch.cuda.synchronize()
    after = [torch.full((1 << k,), 7, dtype=torch.uint8, device="cuda") for k in range(9, 24)]
    y.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert all(bool((a == 7).all()) for a in after)
    del graph
