"""The exchange of row sums between the elementwise warpgroups of the dq pass, modelled on
the host: its barriers and shared slots as in dense_tc_bwd.cu, every interleaving of the
warps explored.  What a run on a GPU meets is one of them."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "block_sparse_gqa_04_b200", "csrc", "dense_tc_bwd.cu")

# arrivals that complete a phase, with one warp for each warpgroup
COUNTS = {"first_full": 1, "q_empty": 1, "s_full0": 1, "s_full1": 1, "dp_full": 1, "ds_full": 5,
          "acc_full": 1, "acc_empty": 4, "r_full0": 2, "r_full1": 1}
BARRIERS = list(COUNTS)


def sums_follow_the_accumulator():
    """Whether warpgroups 2 and 3 write their sums after the wait for the item's dQ."""
    src = open(SOURCE).read()
    write, wait = "bars->rest[wg - 2][row] =", "warp_wait(&bars->acc_full, ii & 1"
    assert src.count(write) == 1 and src.count(wait) == 1
    return src.index(write) > src.index(wait)


def programs(tiles, late):
    """One list of operations per warp, for items of `tiles` key tiles each."""
    mma, gather, warps = [], [], [[] for _ in range(4)]
    n, scores = 0, [0, 0]
    for i, nt in enumerate(tiles):
        gather += [("wait", "q_empty", (i & 1) ^ 1), ("arrive", "first_full")]
        mma += [("wait", "first_full", i & 1), ("arrive", "s_full0"), ("arrive", "dp_full")]
        if nt > 1:
            mma.append(("arrive", "s_full1"))
        for j in range(nt):
            step = n + j
            if step > 0:
                gather.append(("wait", "ds_full", (step & 1) ^ 1))
            if j == 0:
                gather.append(("wait", "acc_empty", (i & 1) ^ 1))
            gather.append(("arrive", "ds_full"))
            mma.append(("wait", "ds_full", step & 1))
            if j + 1 < nt:
                mma.append(("arrive", "dp_full"))
            if j + 2 < nt:
                mma.append(("arrive", f"s_full{j & 1}"))
            for w in warps:
                w += [("wait", f"s_full{j & 1}", (scores[j & 1]) & 1),
                      ("wait", "dp_full", step & 1), ("arrive", "ds_full")]
            scores[j & 1] += 1
        n += nt
        mma += [("arrive", "q_empty"), ("arrive", "acc_full")]
        for wg, w in enumerate(warps):
            give = [("write", wg - 2, ("part", i)), ("arrive", "r_full0")] if wg >= 2 else []
            acc = [("wait", "acc_full", i & 1)]
            w += acc + give if late else give + acc
            w.append(("arrive", "acc_empty"))
            if wg < 2:
                w += [("wait", "r_full0", i & 1), ("read", wg, ("part", i))]
            if wg == 1:
                w += [("write", 1, ("sum", i)), ("arrive", "r_full1")]
            if wg == 0:
                w += [("wait", "r_full1", i & 1), ("read", 1, ("sum", i))]
    return [mma, gather] + warps


def faults(progs):
    """What goes wrong in some interleaving: reads of another item's sums, waits that never
    end.  A barrier is (arrivals, phases completed); a wait for a parity passes while the
    phase that runs has the other one."""
    start = ((0,) * len(progs), ((0, 0),) * len(BARRIERS), (None, None))
    seen, stack, found = {start}, [start], set()
    while stack:
        at, bars, rest = stack.pop()
        moved = False
        for a, prog in enumerate(progs):
            if at[a] == len(prog):
                continue
            op = prog[at[a]]
            nbars, nrest = bars, rest
            if op[0] == "wait":
                if bars[BARRIERS.index(op[1])][1] & 1 == op[2]:
                    continue
            elif op[0] == "arrive":
                x = BARRIERS.index(op[1])
                arrived, phase = bars[x]
                now = (0, phase + 1) if arrived + 1 == COUNTS[op[1]] else (arrived + 1, phase)
                nbars = bars[:x] + (now,) + bars[x + 1:]
            elif op[0] == "write":
                nrest = tuple(op[2] if i == op[1] else v for i, v in enumerate(rest))
            elif rest[op[1]] != op[2]:
                found.add("a read of other sums")
            moved = True
            state = (at[:a] + (at[a] + 1,) + at[a + 1:], nbars, nrest)
            if state not in seen:
                seen.add(state)
                stack.append(state)
        if not moved and any(at[a] < len(p) for a, p in enumerate(progs)):
            found.add("a wait that never ends")
    return found


ITEMS = [(1, 1, 1), (2, 1, 1), (1, 3, 1), (2, 2, 1)]


@pytest.mark.parametrize("tiles", ITEMS)
def test_sums_of_an_item_reach_their_readers(tiles):
    assert not faults(programs(tiles, sums_follow_the_accumulator()))


def test_the_model_sees_sums_that_run_ahead():
    """Written as soon as the steps are over, sums of an item of one key tile meet readers
    that are an item behind."""
    assert faults(programs((1, 1, 1), False)) == {"a read of other sums", "a wait that never ends"}
