"""A fork's copy is enqueued ahead of every write into a block handed out after the fork: the parent may be gone by
then, and its last block, the copy's source, another sequence's or another fork's destination."""

import numpy as np
import pytest


@pytest.fixture(scope="module")
def Manager(cuda_lib_path):
    from paged_kv_cache_85_gb300.block_manager import BlockManager

    return BlockManager


def test_the_source_may_be_handed_out_again(Manager):
    bm = Manager(6, 4)
    bm.allocate(1, range(6))
    rows = np.full(24, -1)
    rows[bm.slots(1, 0, 6)] = range(6)
    (src, dst), = bm.fork(1, 2)
    bm.deallocate(1)
    bm.allocate(3, range(100, 116))  # every block that is free, the source among them
    assert src in bm.block_table(3) and dst == bm.block_table(2)[1] and bm.ref_count(int(src)) == 1
    late = rows.copy()
    # the order asked for: the copy, then the new sequence's rows
    rows.reshape(6, 4)[dst] = rows.reshape(6, 4)[src]
    rows[bm.slots(3, 0, 16)] = range(100, 116)
    assert rows[bm.slots(2, 0, 6)].tolist() == list(range(6))
    assert rows[bm.slots(3, 0, 16)].tolist() == list(range(100, 116))
    # the other one gives the child rows of the new sequence
    late[bm.slots(3, 0, 16)] = range(100, 116)
    late.reshape(6, 4)[dst] = late.reshape(6, 4)[src]
    assert late[bm.slots(2, 0, 6)].tolist() != list(range(6))


@pytest.mark.parametrize("seed", range(5))
def test_steps_that_allocate_first_and_write_after(Manager, seed):
    """Each step forks, drops, allocates and appends on the host, then copies (in a call of its own what follows a
    deallocation), then stores."""
    rng = np.random.default_rng(seed)
    bm, size = Manager(30, 4), 4
    rows, tokens, fresh = np.full(120, -1), {}, iter(range(10 ** 6))
    for _ in range(60):
        copies, writes = [[]], []
        for s in list(tokens):
            what = rng.random()
            if what < 0.25:
                child = next(fresh) + 1000
                if bm.num_free_blocks and len(tokens) < 14:
                    copies[-1] += bm.fork(s, child).tolist()
                    tokens[child] = list(tokens[s])
                    if rng.random() < 0.5:  # the parent goes before the copy is enqueued
                        bm.deallocate(s)
                        del tokens[s]
                        copies.append([])
            elif what < 0.5:
                bm.deallocate(s)
                del tokens[s]
                copies.append([])
        for _ in range(int(rng.integers(1, 4))):
            n = int(rng.integers(1, 15))
            if bm.can_allocate(n) and len(tokens) < 12:
                s, t = next(fresh) + 1000, rng.integers(0, 1000, n).tolist()
                bm.allocate(s, t)
                tokens[s] = t
                writes.append((bm.slots(s, 0, n), list(t)))
        for s in list(tokens):
            if rng.random() < 0.5 and bm.can_append(s):
                t = int(rng.integers(0, 1000))
                writes.append((np.array([bm.append(s, t)]), [t]))
                tokens[s].append(t)
        table = rows.reshape(-1, size)
        for pairs in copies:
            assert len({b for _, b in pairs}) == len(pairs) and not {a for a, _ in pairs} & {b for _, b in pairs}
            for a, b in pairs:
                table[b] = table[a]
        for at, t in writes:
            rows[at] = t
        for s, t in tokens.items():
            assert rows[bm.slots(s, 0, len(t))].tolist() == t
