"""The error words of matmul_i8 calls that bring no workspace: one a stream, so
that a checked call neither raises for another stream's timeout nor clears it."""
import pytest
import torch

import frequency_ranked_drafter_gb300 as vt
from gpu_util import need_cuda
from test_gpu_matmul_i8_timeout import inputs, right, short_call

pytestmark = pytest.mark.gpu

VT_ERR_TIMEOUT = 5


def word_of(stream):
    return vt._i8_words[stream.device.index, stream.cuda_stream]


def test_a_checked_call_sees_its_own_stream_only(monkeypatch):
    dev = need_cuda()
    monkeypatch.setattr(vt, "_i8_words", {})
    ins, want, tol = inputs(dev, 40, 12000, 1024)
    lost = torch.empty(40, 12000, device=dev)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
    for s in (a, b):
        with torch.cuda.stream(s):
            assert right(vt.matmul_i8(*ins), want, tol)
    assert right(vt.matmul_i8(*ins, check=True), want, tol)  # the default stream's
    words = [word_of(s) for s in (a, b, torch.cuda.current_stream(dev))]
    assert len({w.data_ptr() for w in words}) == 3
    # a call on stream a that gives up, seen by nobody yet
    with torch.cuda.stream(a):
        assert short_call(*ins, lost, words[0], 1) == 0
    a.synchronize()
    with torch.cuda.stream(b):
        assert right(vt.matmul_i8(*ins, check=True), want, tol)
    assert right(vt.matmul_i8(*ins, check=True), want, tol)
    with torch.cuda.stream(a):
        vt.matmul_i8(*ins)
        with pytest.raises(vt.VTError) as e:
            vt.matmul_i8(*ins, check=True)
        assert e.value.status == VT_ERR_TIMEOUT
        assert right(vt.matmul_i8(*ins, check=True), want, tol)
    # a workspace of the call's own leaves the stream's word alone
    own = torch.zeros(256, dtype=torch.uint8, device=dev)
    assert short_call(*ins, lost, own, 1) == 0
    assert right(vt.matmul_i8(*ins, check=True), want, tol)
    with pytest.raises(vt.VTError):
        vt.check_error_word("vt_matmul_i8", own)


def test_a_captured_call_keeps_its_word(monkeypatch):
    """First use of the product under capture: its word outlives the call, is no
    memory of the graph's, and no replay clears it."""
    dev = need_cuda()
    monkeypatch.setattr(vt, "_i8_words", {})
    ins, want, tol = inputs(dev, 40, 12000, 1024)
    torch.cuda.synchronize()
    graphs, outs, others = [], [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(vt.matmul_i8(*ins))
            # the sizes of a word, where a freed one would be given out again
            others.append([torch.full((256,), 7, dtype=torch.uint8, device=dev)
                           for _ in range(20)])
        graphs.append(g)
    assert len(vt._i8_words) == 1  # both graphs' calls
    word, = vt._i8_words.values()
    assert word.shape == (256,) and word.device == dev and not bool(word.any())
    lo, hi = word.data_ptr(), word.data_ptr() + 256
    for t in [t for ts in others for t in ts] + outs:
        assert t.data_ptr() >= hi or t.data_ptr() + t.numel() * t.element_size() <= lo
    word[128] = VT_ERR_TIMEOUT  # as a wait that gave up in an earlier replay
    for g, y, ts in zip(graphs, outs, others):
        y.fill_(-7.0)
        g.replay()
        torch.cuda.synchronize()
        assert right(y, want, tol)
        assert all(bool((t == 7).all()) for t in ts)
        assert int(word[128].item()) == VT_ERR_TIMEOUT
    with pytest.raises(vt.VTError):
        vt.check_error_word("vt_matmul_i8", word)
    # graphs gone, the word is still good for the next capture, and eager calls
    # on the stream of the caller have another
    del graphs, outs, others
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = vt.matmul_i8(*ins)
    g.replay()
    assert right(y, want, tol) and right(vt.matmul_i8(*ins, check=True), want, tol)
    assert len(vt._i8_words) == 2 and not bool(word.any())
