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
