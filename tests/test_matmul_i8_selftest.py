"""vt_selftest_matmul_i8's refusals, on the host (nothing here makes a CUDA
call): its own argument and vt_matmul_i8's."""
import frequency_ranked_drafter_gb300 as vt

OK, INVALID, WORKSPACE = 0, 1, 4
FAKE, FAR = 1 << 20, 1 << 40  # non-null addresses never dereferenced


def test_refusals():
    lib = vt.load()
    good = dict(X=FAKE, M=20, d=64, od=2, ldo=100, ws=FAKE, n=256, budget=1000)

    def call(**kw):
        a = dict(good, **kw)
        return lib.vt_selftest_matmul_i8(a["X"], FAKE, a["M"], FAKE, FAKE, 100, a["d"], None, FAR,
                                         a["od"], a["ldo"], a["ws"], a["n"], a["budget"], None)

    for kw in (dict(budget=0), dict(budget=-1), dict(budget=(1 << 31) + 1), dict(X=None),
               dict(d=24), dict(od=1), dict(ldo=99), dict(M=65536)):
        assert call(**kw) == INVALID, kw
    assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE
    assert call(M=0) == OK
