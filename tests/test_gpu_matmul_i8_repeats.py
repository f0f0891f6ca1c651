"""vt_matmul_i8 many times over on inputs that are not in L2: exact every time.
Short rows of X and W leave the tensor-core kernel's stages in any order of
landing, tile after tile and block after block."""
import pytest
import torch

import frequency_ranked_drafter_gb300 as vt
from gpu_util import need_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,d", [(256, 38290, 144), (128, 40000, 272), (100, 60000, 400),
                                   (300, 39000, 144), (80, 78000, 640), (1024, 20000, 144),
                                   (60, 80000, 144), (33, 80000, 400), (17, 120000, 272),
                                   (128, 2000, 2048), (256, 3000, 1040)])
def test_the_same_sums_every_time(M, N, d):
    """Whole sums below 2^24 and scales of 1: bit for bit."""
    dev = need_cuda()
    g = torch.Generator(device=dev).manual_seed(M + N + d)
    one = torch.ones(max(M, N), device=dev)
    spoil = torch.empty(2 ** 28, dtype=torch.uint8, device=dev)  # twice L2
    for turn in range(40):
        X = torch.randint(-128, 128, (M, d), generator=g, dtype=torch.int8, device=dev)
        W = torch.randint(-128, 128, (N, d), generator=g, dtype=torch.int8, device=dev)
        # sums of up to 640 products of at most 2^14 are whole numbers below 2^24
        # (2048: of random signs, far below); each product and sum is exact in fp64
        want = (X.double() @ W.double().T).float()
        if turn % 2:
            spoil.fill_(turn)
        out = torch.full((M, N), -7.0, device=dev)
        vt.matmul_i8(X, one[:M], W, one[:N], out=out)
        same = out == want
        assert bool(same.all()), (turn, int((~same).sum()), (~same).nonzero()[0].tolist())
