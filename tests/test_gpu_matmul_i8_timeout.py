"""The failure path of vt_matmul_i8's bounded waits: with waits that give up at
once, or somewhere on the way, the call reports VT_ERR_TIMEOUT, ends by itself
with nothing left under way, and the next call is right."""
import numpy as np
import pytest
import torch

import frequency_ranked_drafter_gb300 as vt
import serving_ref as ref
from gpu_util import need_cuda
from test_gpu_serving import int8_rows

pytestmark = pytest.mark.gpu

VT_ERR_TIMEOUT, VT_ERR_UNSUPPORTED = 5, 3


def inputs(dev, M, N, d):
    X, W = int8_rows(M, d, M + 1), int8_rows(N, d, N + 2)
    xs, ws = torch.rand(M) * 0.02 + 1e-4, torch.rand(N) * 1e-3 + 1e-5
    want, tol = ref.matmul(X.numpy(), xs.numpy(), W.numpy(), ws.numpy())
    return [t.to(dev) for t in (X, xs, W, ws)], want, tol


def short_call(X, xs, W, ws, out, word, budget):
    lib = vt.load()
    return lib.vt_selftest_matmul_i8(
        X.data_ptr(), xs.data_ptr(), X.shape[0], W.data_ptr(), ws.data_ptr(), W.shape[0],
        X.shape[1], None, out.data_ptr(), 2, out.stride(0), word.data_ptr(), word.numel(), budget,
        torch.cuda.current_stream().cuda_stream)


def right(y, want, tol):
    return bool((np.abs(y.cpu().double().numpy() - want) <= tol).all())


# One tile a CTA and many, one MMA a tile and two, shared k, blocks of X in turn
# and side by side, fewer stages than places and more.
@pytest.mark.parametrize("M,N,d", [(5, 40000, 1024), (17, 20000, 2048), (60, 1000, 4096),
                                   (64, 9000, 4096), (128, 4000, 4096), (300, 30000, 512),
                                   (256, 4096, 2048), (40, 300, 16384), (20, 129, 64)])
def test_waits_that_run_out(M, N, d):
    dev = need_cuda()
    ins, want, tol = inputs(dev, M, N, d)
    word = torch.zeros(256, dtype=torch.uint8, device=dev)
    out = torch.empty(M, N, device=dev)
    for budget in (1, 200, 1000, 1, 4000, 20000, 1):
        out.fill_(-7.0)
        assert short_call(*ins, out, word, budget) == 0, vt.load().vt_last_error()
        torch.cuda.synchronize()
        e = int(word[128:132].view(torch.int32).item())
        assert e in (0, VT_ERR_TIMEOUT)
        if budget == 1:  # a stage's conversion takes hundreds of clocks
            assert e == VT_ERR_TIMEOUT
        if e == 0:
            assert right(out, want, tol)
        assert int(word.sum(dtype=torch.int64).item()) == e  # nothing else is written
        word.zero_()
        assert right(vt.matmul_i8(*ins, ws=word, check=True), want, tol)


def test_a_checked_call_reports_and_clears_the_word():
    dev = need_cuda()
    ins, want, tol = inputs(dev, 33, 3000, 512)
    word = torch.zeros(256, dtype=torch.uint8, device=dev)
    out = torch.empty(33, 3000, device=dev)
    assert short_call(*ins, out, word, 1) == 0
    with pytest.raises(vt.VTError) as e:
        vt.matmul_i8(*ins, ws=word, check=True)
    assert e.value.status == VT_ERR_TIMEOUT
    assert not bool(word.any())
    assert right(vt.matmul_i8(*ins, ws=word, check=True), want, tol)
    # the kernels without waits leave the word alone, and it is read all the same
    few, want, tol = inputs(dev, 3, 3000, 512)
    assert short_call(*few, torch.empty(3, 3000, device=dev), word, 1) == VT_ERR_UNSUPPORTED
    word[128] = VT_ERR_TIMEOUT
    with pytest.raises(vt.VTError):
        vt.matmul_i8(*few, ws=word, check=True)
    assert right(vt.matmul_i8(*few, ws=word, check=True), want, tol)


def test_two_timeouts_at_once_and_while_captured():
    """Calls that give up on two streams, and in a replayed graph."""
    dev = need_cuda()
    ins, want, tol = inputs(dev, 40, 12000, 1024)
    words = [torch.zeros(256, dtype=torch.uint8, device=dev) for _ in range(3)]
    outs = [torch.empty(40, 12000, device=dev) for _ in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(5):
        for s, w, o in zip(streams, words, outs):
            with torch.cuda.stream(s):
                assert short_call(*ins, o, w, 1) == 0
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        assert short_call(*ins, outs[2], words[2], 1) == 0
        y = vt.matmul_i8(*ins)
    g.replay()
    torch.cuda.synchronize()
    assert all(int(w[128].item()) == VT_ERR_TIMEOUT for w in words)
    assert right(y, want, tol)
