"""The hand-over of stages in the product's tensor-core kernel (one loading role,
two sets of converting warps that take turns at stages, one multiplying role), as
a model on the CPU: every warp reads the stage that it waited for and overwrites
no operand that is still multiplied, whatever order loads land in and roles run
in.  A parity wait passes when the barrier's running phase has the other parity,
so it may pass too early for a warp that is two phases ahead of the barrier; the
order in which a warp makes its two waits is the kernel's (read from its source).
"""
import os
import random
import re

import pytest

import frequency_ranked_drafter_gb300 as vt

CSRC = os.path.join(os.path.dirname(vt.__file__), "csrc")


def wait_orders():
    """For each converting role: the barriers it waits for at a stage, in order."""
    text = open(os.path.join(CSRC, "matmul_i8_tc.cu")).read()
    pairs = re.findall(r"await\(&(\w+)\[\w+\.i\], [^)]*\) &&\s*await\(&(\w+)\[\w+\.i\], [^)]*\)\)\) \{",
                       text)
    return [p for p in pairs if set(p) == {"raw_full", "cv_empty"}]


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, parity):
        return self.done % 2 != parity


class Stale(Exception):
    pass


def run(stages, conv, total, order, rng, warps=2):
    """One CTA's work over `total` stages, `warps` in each converting set."""
    raw_full = [Barrier(1) for _ in range(stages)]
    raw_empty = [Barrier(warps) for _ in range(stages)]
    cv_full = [Barrier(warps) for _ in range(conv)]
    cv_empty = [Barrier(1) for _ in range(conv)]
    raw = [None] * stages                 # the stage whose bytes lie there
    operand = [[None] * warps for _ in range(conv)]
    landing, multiplied = [], []          # loads and products under way
    used = [None] * conv                  # the stage whose product reads the operand

    def loader():
        for i in range(total):
            s, ph = i % stages, i // stages % 2
            yield lambda: raw_empty[s].passes(ph ^ 1)
            landing.append(i)

    def converter(u, w):
        for i in range(u, total, 2):
            s, ph = i % stages, i // stages % 2
            c, cph = i % conv, i // conv % 2
            waits = {"raw_full": lambda: raw_full[s].passes(ph),
                     "cv_empty": lambda: cv_empty[c].passes(cph ^ 1)}
            for name in order:
                yield waits[name]
            for _ in range(2):            # reads go on for a while
                if raw[s] != i:
                    raise Stale(f"stage {i} read where {raw[s]} lies")
                yield lambda: True
            if used[c] is not None:
                raise Stale(f"operand of {used[c]} overwritten by {i}")
            operand[c][w] = i
            cv_full[c].arrive()
            raw_empty[s].arrive()

    def multiplier():
        for i in range(total):
            c, cph = i % conv, i // conv % 2
            yield lambda: cv_full[c].passes(cph)
            if operand[c] != [i] * warps:
                raise Stale(f"product of {i} reads {operand[c]}")
            used[c] = i
            multiplied.append(i)

    roles = [loader(), multiplier()] + [converter(u, w) for u in (0, 1) for w in range(warps)]
    weight = [rng.choice([0.1, 1.0, 10.0]) for _ in roles]
    slow = rng.choice([0.02, 0.3, 1.0])   # how fast loads land
    state = [(r, next(r, None)) for r in roles]
    while any(want is not None for _, want in state) or landing or multiplied:
        moves = [k for k, (_, want) in enumerate(state) if want is not None and want()]
        events = (["land"] if landing else []) + (["product"] if multiplied else [])
        assert moves or events, "no role can go on"
        pick = rng.choices(moves + events,
                           [weight[k] for k in moves] + [slow if e == "land" else 0.5
                                                         for e in events])[0]
        if pick == "land":                # in any order
            i = landing.pop(rng.randrange(len(landing)))
            raw[i % stages] = i
            raw_full[i % stages].arrive()
        elif pick == "product":           # in the order of their issue
            c = multiplied.pop(0) % conv
            used[c] = None
            cv_empty[c].arrive()
        else:
            r = state[pick][0]
            state[pick] = (r, next(r, None))


def test_both_converting_roles_wait_in_one_order():
    orders = wait_orders()
    assert len(orders) == 2 and orders[0] == orders[1], orders


@pytest.mark.parametrize("stages", [2, 3, 4, 5, 6, 7, 8])
def test_every_stage_is_the_one_waited_for(stages):
    order = wait_orders()[0]
    for seed in range(150):
        rng = random.Random(1000 * stages + seed)
        run(stages, 3, rng.choice([1, 2, 3, 5, 16, 40]), order, rng)


def test_the_other_order_reads_stale_stages():
    """What the model is for: with the raw stage waited for first, an odd number
    of stages is read too early."""
    with pytest.raises(Stale):
        for seed in range(300):
            rng = random.Random(seed)
            run(3, 3, 40, ("raw_full", "cv_empty"), rng)
