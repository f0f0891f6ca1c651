"""Top-p borders that fall exactly on the fp32 sums by which vt_sample_logits
places its search: the nucleus has to reach top_p of the mass all the same."""
import numpy as np
import pytest
import torch

import frequency_ranked_drafter_gb300 as vt
from gpu_util import need_cuda

pytestmark = pytest.mark.gpu

F = np.float32
BINS, PER, WARP = 1024, 4, 32


def bin_sums(x):
    """For a row of 128 logits: the sums of the bins' lower bounds as a thread
    of the kernel has them (its own four bins', and with all before it), and
    the logits that are counted (those down to the tenth largest, shortened to
    16 bits of its pattern)."""
    least = (np.sort(x)[-10].view(np.uint32) & np.uint32(0xffff0000)).view(F)
    xs = x[x >= least]
    scale = F(BINS - 1) / (x.max() - least)
    b = ((x.max() - xs) * scale).astype(int)
    count = np.bincount(b[b < BINS], minlength=BINS).reshape(-1, PER).astype(F)
    step = F(1.44269504) / scale
    e = np.exp2(-step * np.arange(0, BINS, PER, dtype=F), dtype=F)
    ratio = np.exp2(-step, dtype=F)
    own = np.zeros(BINS // PER, F)
    for i in range(PER):
        e = e * ratio
        own = own + count[:, i] * e
    v = own.reshape(-1, WARP).copy()
    for o in (1, 2, 4, 8, 16):
        v = np.concatenate([v[:, :o], v[:, o:] + v[:, :-o]], 1)
    before = np.concatenate([[F(0)], np.cumsum(v[:-1, -1], dtype=F)])
    return own, (v + before[:, None]).reshape(-1), xs


def border_cases(rows, around, seed):
    """Rows with a thread whose sum is off by a rounding once its own part has
    been taken away and added again, and top_p around the value for which that
    sum is the very bound that is asked for."""
    rng = np.random.default_rng(seed)
    X, P = [], []
    while len(P) < rows:
        x = np.maximum(F(8) + rng.standard_normal(128) * 2, 0.01).astype(F)
        own, upto, xs = bin_sums(x)
        mass = np.exp(x.astype(np.float64) - x.max()).sum()
        listed = np.exp(xs.astype(np.float64) - x.max()).sum()
        for t in np.nonzero((own > 0) & ((upto - own) + own < upto))[0]:
            p = F(upto[t] / 1.001 / mass)
            if 0.02 < p < 0.99 * listed / mass:
                near = (p.view(np.int32) + np.arange(-around, around + 1, dtype=np.int32)).view(F)
                X += [x] * len(near)
                P += list(near)
    return torch.from_numpy(np.stack(X[:rows])), torch.from_numpy(np.array(P[:rows], dtype=F))


def test_nucleus_reaches_top_p_at_the_bins_borders():
    """60000 rows: the kept logits are the shortest prefix, in the order of the
    logits, whose mass is at least top_p of the row's, to the 2^-27 of the mass
    (and 2^-43 for each logit) that fixed-point weights may be off; and the
    distribution is their share of it."""
    dev = need_cuda()
    x, p = (t.to(dev) for t in border_cases(60000, 24, 1))
    dist = vt.sample_logits(x, None, top_p=p)
    w = torch.exp(x.double() - x.double().max(1, keepdim=True).values)
    share = w / w.sum(1, keepdim=True)
    tol = 2.0 ** -27 + 128 * 2.0 ** -43
    order = torch.argsort(x, dim=1, descending=True, stable=True)
    kept = (dist > 0).gather(1, order)
    assert bool((kept[:, 1:] <= kept[:, :-1]).all()), "what is kept is a prefix"
    mass = (share.gather(1, order) * kept).cumsum(1)[:, -1]
    last = (share * (dist > 0) + 2.0 * (dist == 0)).min(1).values
    short = mass < p.double() - tol
    long = mass - last >= p.double() + tol
    assert not bool(short.any()), (int(short.sum()), x[short][0], p[short][0], mass[short][0])
    assert not bool(long.any()), (int(long.sum()), x[long][0], p[long][0], mass[long][0])
    # four roundings of a probability and the weights' own errors, below
    # 4.1 * 2^-24 in all
    want = share * (dist > 0) / mass[:, None]
    assert bool(((dist.double() - want).abs() <= (4.1 * 2.0 ** -24 + tol) * want).all())
