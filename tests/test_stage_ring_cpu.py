"""Without a GPU: the ring of block stages of the 4-bit decode (csrc/stage_ring.h), copies landing in any order.

A model of one CTA: the producer issues blocks in order as stages become free, copies land in any order, readers
wait for a phase by its parity as the hardware does (a phase counts as complete when the barrier's count of
completed phases has the other parity). A reader may only ever pass a wait with its own block in the stage."""
import ctypes
import random
import subprocess

import pytest

from hybrid_sliding_window_swa_b200 import _build

STAGES = [4, 7, 9, 10, 22]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src = '#include "stage_ring.h"\nextern "C" {\n'
    for ns in STAGES:
        src += (f"int stage_{ns}(unsigned b) {{ return hswa::StageRing<{ns}>::stage(b); }}\n"
                f"int parity_{ns}(unsigned b) {{ return (int)hswa::StageRing<{ns}>::parity(b); }}\n"
                f"int may_wait_{ns}(unsigned i, unsigned b) {{ return hswa::StageRing<{ns}>::may_wait(i, b); }}\n")
    (d / "ring.cpp").write_text(src + "}\n")
    so = str(d / "ring.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", _build.CSRC, "-o", so, str(d / "ring.cpp")], check=True)
    return ctypes.CDLL(so)


def early(lib, ns, readers, n_blocks, seed, who, guarded=True):
    """The first block that a reader took before it had landed, or None. who(block) -> reader; without `guarded`
    readers wait by parity alone."""
    stage, parity, may_wait = (getattr(lib, f"{f}_{ns}") for f in ("stage", "parity", "may_wait"))
    rng = random.Random(seed)
    landed, freed, holds = [0] * ns, [0] * ns, [None] * ns
    mine = [[b for b in range(n_blocks) if who(b) == r] for r in range(readers)]
    done = lambda phases, par: (phases & 1) != par  # a barrier that has completed `phases` phases
    issued, flying, at = 0, [], [0] * readers
    slow = rng.randrange(readers)  # copies of one reader's blocks tend to be late
    while any(at[r] < len(mine[r]) for r in range(readers)):
        moves = []
        if issued < n_blocks and done(freed[stage(issued)], parity(issued) ^ 1):
            moves.append(("issue", issued))
        late = [b for b in flying if who(b) != slow]
        moves += [("land", b) for b in (late if late and rng.random() < 0.9 else flying)]
        for r in range(readers):
            if at[r] < len(mine[r]):
                b = mine[r][at[r]]
                if (not guarded or may_wait(issued, b)) and done(landed[stage(b)], parity(b)):
                    moves.append(("read", b))
        assert moves, "stuck"
        what, b = rng.choice(moves)
        st = stage(b)
        if what == "issue":
            assert holds[st] is None  # nobody still reads the stage
            flying.append(b)
            issued += 1
        elif what == "land":
            holds[st] = b
            landed[st] += 1
            flying.remove(b)
        else:
            if holds[st] != b:
                return b
            holds[st] = None
            freed[st] += 1
            at[who(b)] += 1
    return None


def deals(readers, seed):
    """Blocks to readers in turn, and in uneven turns, as items of a few blocks each give."""
    r = random.Random(seed + 99)
    deal = [r.randrange(readers) for _ in range(400)]
    return [lambda b: b % readers, lambda b: deal[b], lambda b: (b // 3) % readers]


@pytest.mark.parametrize("ns", STAGES)
@pytest.mark.parametrize("readers", [1, 2, 4])
def test_readers_never_pass_before_their_block(lib, ns, readers):
    for seed in range(12):
        for who in deals(readers, seed):
            assert early(lib, ns, readers, 200, seed, who) is None


@pytest.mark.parametrize("ns,readers", [(10, 4), (7, 2), (9, 2)])
def test_parity_alone_would_let_them_pass(lib, ns, readers):
    # the model sees the fault
    assert any(early(lib, ns, readers, 400, seed, who, guarded=False) is not None
               for seed in range(20) for who in deals(readers, seed))


@pytest.mark.parametrize("ns", STAGES)
def test_counts_may_wrap(lib, ns):
    may_wait = getattr(lib, f"may_wait_{ns}")
    top = 2 ** 32
    for issued, block, want in ((1, 0, 1), (0, 0, 0), (5, 7, 0), (3, top - 2, 1), (top - 2, 3, 0), (top - 1, top - 1, 0)):
        assert may_wait(issued, block) == want
