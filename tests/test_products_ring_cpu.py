"""The ring of stages that the products' loading warps fill, as a model on the host: every order in which its actors
can go on is tried, and none may leave one of them waiting for good.

A wait names the parity of the phase that it waits for, so it passes while that phase is the last one completed, and
no longer when the barrier is a phase further.  What keeps an actor from being overtaken is that the stage cannot
become full without it.  A warp that follows the ring without bytes to load lacks that, and the model finds the order
in which it is left behind; the tail-row warp of the weight gradient skips the blocks that it has no part in without a
wait, so nothing overtakes it there."""
import pytest

STAGES = 2
BLOCKS = 7


def _waits(completed, k):
    """Whether the wait for phase k (0, 1, ...) of a barrier with `completed` phases goes on waiting."""
    return (completed & 1) == (k & 1)


def _stuck(with_bytes, followers, tails=()):
    """A reachable state in which someone is not done and no one can go on, or None.

    State: the block that each loader, the consumer and the tail warp (index into `tails`) have come to.  The
    barriers' phases follow from it: stage s has been emptied as often as the consumer took blocks of it, and its
    block b is full once every loader with bytes is past b (and the tail warp, if b has tail rows)."""
    n = with_bytes + followers
    tails = sorted(tails)

    def emptied(consumer, s):
        return len(range(s, consumer, STAGES))

    def moves(state):
        loaders, consumer, tail = state
        for i, b in enumerate(loaders):
            if b < BLOCKS:
                # block b needs its stage emptied b // STAGES times: the wait is for phase b // STAGES - 1, of parity
                # one before the first
                if not _waits(emptied(consumer, b % STAGES), b // STAGES - 1):
                    yield tuple(x + (j == i) for j, x in enumerate(loaders)), consumer, tail
        loaded = min(loaders[:with_bytes])
        if tail < len(tails) and loaded > tails[tail]:
            # its landed barrier has completed once for each earlier tail of the stage and once for this one
            yield loaders, consumer, tail + 1
        if consumer < BLOCKS and loaded > consumer and (consumer not in tails or tail > tails.index(consumer)):
            yield loaders, consumer + 1, tail

    start = ((0,) * n, 0, 0)
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        following = list(moves(state))
        if not following and (min(state[0]) < BLOCKS or state[1] < BLOCKS or state[2] < len(tails)):
            return state
        for s in following:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


@pytest.mark.parametrize("loaders", [1, 2, 3])
@pytest.mark.parametrize("tails", [(), (6,), (0, 3, 6), (2, 4), tuple(range(BLOCKS))])
def test_loading_warps_with_bytes_are_never_left_behind(loaders, tails):
    assert _stuck(loaders, 0, tails) is None


@pytest.mark.parametrize("loaders", [1, 2])
def test_a_warp_without_bytes_is_left_behind(loaders):
    loaders_at, consumer, _ = _stuck(loaders, 1)
    assert loaders_at[-1] < BLOCKS and consumer == BLOCKS
