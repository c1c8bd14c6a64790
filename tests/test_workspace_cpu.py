"""pipeline.Workspace: what a captured graph was given stays allocated when the workspace grows (no GPU)."""
import weakref

from post_quantization_b200 import pipeline as P


def test_a_captured_buffer_outlives_a_larger_request(monkeypatch):
    capturing = [False]
    monkeypatch.setattr(P, "_capturing", lambda buf: capturing[0])
    ws = P.Workspace("cpu")
    capturing[0] = True
    first = ws.get(1000)                               # the graph now holds its address
    capturing[0] = False
    held = weakref.ref(ws.buf)
    assert held() is not None
    del first
    large = ws.get(100000)
    assert held() is not None                          # a replay still writes there
    assert large.numel() == 100000 and large.data_ptr() % 256 == 0
    held = weakref.ref(ws.buf)
    del large
    ws.get(1000000)                                    # no graph has the second one
    assert held() is None


def test_requests_reuse_the_buffer():
    ws = P.Workspace("cpu")
    a = ws.get(5000)
    assert ws.get(0) is None
    assert ws.get(300).data_ptr() == a.data_ptr()
