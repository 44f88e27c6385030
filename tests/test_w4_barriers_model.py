"""A model of the barriers of the products on 4-bit weights (``grouped_matmul_w4.cu``),
without a GPU: who waits for what, under random delays.

An mbarrier's wait tells its rounds apart by parity alone, so a warp that runs two
rounds ahead of a barrier goes on with a stage's old bytes.  Two warps issue the MMAs
of alternate blocks of k.  With an even number of stages the same warp has waited for
a stage's round before; with an odd number the other one has, and only the accumulators'
barriers keep this warp close enough.  The model runs the kernel's rule for the number
of stages and the order of the two waits, and, to show that it would see the fault,
two rules that break it."""
import random

import pytest

MOST_STAGES = 8


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def over(self, parity):  # a fresh barrier counts as having ended the round before its first
        return (self.phase & 1) != parity


class Stale(AssertionError):
    """Something was read that is not what was waited for."""


def run(stages, per, operands_first, tiles, rng):
    """One launch's warps of a block, tiles of `tiles` blocks of k, stepped in random order."""
    kept = 16 if per == 1 else 32
    full = [Barrier(2) for _ in range(stages)]  # the operands' and the scales' landing
    empty = [Barrier(1) for _ in range(stages)]
    acc_full, acc_empty = [Barrier(per) for _ in range(2)], [Barrier(2) for _ in range(2)]
    stage, scales_of = [[None, None] for _ in range(stages)], [None] * kept
    acc = [[None] * per for _ in range(2)]  # block of k in each place of an accumulator
    read = [[2] * per for _ in range(2)]    # adding warps that have read it
    landing = [[], []]                      # copies on their way
    pipe = []                               # MMAs in order of issue
    total = sum(tiles)

    def load(which):
        st = phase = 0
        for it in range(total):
            if it >= stages:
                while not empty[st].over(phase ^ 1):
                    yield
            landing[which].append((it, st))
            yield
            st += 1
            if st == stages:
                st, phase = 0, phase ^ 1

    def land(which):
        while True:
            if landing[which]:
                # in any order, the oldest last as often as not
                it, st = landing[which].pop(rng.choice([-1, rng.randrange(len(landing[which]))]))
                stage[st][which] = it
                if which == 1:
                    scales_of[it % kept] = it
                full[st].arrive()
            yield

    def issue(odd):
        it = st = phase = group = 0
        for blocks in tiles:
            slot = 0
            for kb in range(blocks):
                at, turn, ac, last = st, phase, group & 1, kb + 1 == blocks
                here, round_of_acc = slot, (group >> 1) & 1
                st += 1
                if st == stages:
                    st, phase = 0, phase ^ 1
                slot += 1
                if slot == per or last:
                    slot, group = 0, group + 1
                if (it & 1) == odd:
                    waits = [(full[at], turn), (acc_empty[ac], round_of_acc ^ 1)]
                    for bar, parity in waits if operands_first else waits[::-1]:
                        while not bar.over(parity):
                            yield
                    pipe.append((it, at, ac, here))
                    if last:
                        for _ in range(here + 1, per):
                            acc_full[ac].arrive()
                    yield
                it += 1

    def tensor_core():
        while True:
            if pipe:
                it, at, ac, here = pipe.pop(0)
                if stage[at] != [it, it]:
                    raise Stale(f"block {it} read {stage[at]}")
                if read[ac][here] != 2:
                    raise Stale(f"block {it} overwrote block {acc[ac][here]}")
                acc[ac][here], read[ac][here] = it, 0
                acc_full[ac].arrive()
                empty[at].arrive()
            yield

    def add():
        it = group = 0
        for blocks in tiles:
            kb = 0
            while kb < blocks:
                ac, n = group & 1, min(per, blocks - kb)
                while not acc_full[ac].over((group >> 1) & 1):
                    yield
                for i in range(n):
                    if acc[ac][i] != it + i or scales_of[(it + i) % kept] != it + i:
                        raise Stale(f"sums of block {it + i} took {acc[ac][i]}, scales {scales_of[(it + i) % kept]}")
                    read[ac][i] += 1
                    yield
                acc_empty[ac].arrive()
                kb, it, group = kb + n, it + n, group + 1
                yield

    todo = [load(0), load(1), issue(0), issue(1), add(), add()]
    ever = [land(0), land(1), tensor_core()]
    speed = {id(a): 4.0 ** rng.uniform(-2, 2) for a in todo + ever}
    for _ in range(60 * total * 30):
        if not todo:
            return
        actors = todo + ever
        one = rng.choices(actors, [speed[id(a)] for a in actors])[0]
        for _ in range(1 if one in ever else rng.choice([1, 2, 8])):
            try:
                next(one)
            except StopIteration:
                todo.remove(one)
                break
    assert not todo, "no end"


def stages_of(fit, per):
    """The kernel's rule: stages that fit -> stages used."""
    return fit - 1 if fit & 1 and (per == 4 or fit < 5) else fit


def launches(rng):
    return [rng.choice([1, 2, 3, 5, 11, 16]) for _ in range(6)] + [rng.randint(1, 30)]


@pytest.mark.parametrize("per", [1, 2, 4])
@pytest.mark.parametrize("fit", range(2, MOST_STAGES + 1))
def test_every_block_reads_its_own_bytes(fit, per):
    rng = random.Random(100 * fit + per)
    for _ in range(25):
        run(stages_of(fit, per), per, per == 1, launches(rng), rng)


@pytest.mark.parametrize("stages,per,operands_first", [(5, 2, True), (5, 4, False), (3, 1, True)])
def test_the_model_sees_rules_that_do_not_hold(stages, per, operands_first):
    rng = random.Random(7)
    with pytest.raises(Stale):
        for _ in range(400):
            run(stages, per, operands_first, launches(rng), rng)
