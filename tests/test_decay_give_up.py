"""How the blocks of the head-decay attention's tensor-core kernel leave after a wait was given up, as a model of their
barriers: whenever each warp learns of it, none may stay behind at a barrier that the others do not come to."""
import itertools

import pytest


def run(warps, count):
    """Walks generators that yield barrier ids; count[id]: arrivals that complete it.  True: all of them end."""
    at = [next(w, None) for w in warps]
    while any(b is not None for b in at):
        ready = [b for b in set(at) - {None} if sum(x == b for x in at) == count[b]]
        if not ready:
            return False
        for b in ready:
            at = [next(w, None) if x == b else x for x, w in zip(at, warps)]
    return True


def seen(warps, checks):
    """For each warp the number of the check from which on it sees the flag (`checks`: never)."""
    return itertools.product(range(checks + 1), repeat=warps)


# ------------------------------------------------------------------ the workers of one lane quarter, chunk by chunk
GROUP, PIECE = 1, 0


def worker(terms, sees, votes, leaves):
    """One warp's barriers: those of chunks whose keys come in three terms, with a vote of the warps; the piece's end."""
    gone = False
    for i, n in enumerate(terms):
        if n == 3:
            gone = gone or i >= sees
            votes[i] = votes.get(i, False) or gone
            yield GROUP
            gone = votes[i]
        else:
            gone = gone or i >= sees
        if gone and leaves:
            break
    yield PIECE


def workers_end(terms, leaves):
    for sees in seen(4, len(terms)):
        votes = {}
        if not run([worker(terms, s, votes, leaves) for s in sees], {GROUP: 4, PIECE: 4}):
            return False
    return True


@pytest.mark.parametrize("terms", [[2, 2, 2], [3, 3, 3], [2, 2, 3], [2, 3, 3], [3, 2, 3], [0, 2, 3, 2]])
def test_workers_come_to_the_same_barriers(terms):
    assert workers_end(terms, leaves=False)


def test_workers_that_left_their_loop_would_not():
    """Leaving is safe only where every chunk has the vote (heads of up to 64 channels), or none."""
    assert workers_end([2, 2, 2], leaves=True) and workers_end([3, 3, 3], leaves=True)
    assert not workers_end([2, 2, 3], leaves=True)


# ------------------------------------------------------------------ all roles, piece by piece
def role(pieces, gives_up, flag, late, barriers):
    """One role's barriers: those at the end of each piece, then the block's.  gives_up: the piece in which it puts up the
    flag; late: with one barrier a piece, whether it reads the flag only when others are through the next piece's waits."""
    for i in range(pieces):
        if i == gives_up:
            flag.add(i)
        yield PIECE
        gone = any(j <= i + (late and barriers == 1) for j in flag)
        if barriers == 2:
            yield PIECE
        if gone:
            break
    yield PIECE


def roles_end(barriers):
    """Three roles, each giving up in any piece or never, and reading early or late."""
    for gives in seen(3, 3):
        for late in itertools.product((False, True), repeat=3):
            flag = set(gives) - {3}
            if not run([role(3, g, flag, x, barriers) for g, x in zip(gives, late)], {PIECE: 3}):
                return False
    return True


def test_roles_leave_at_the_same_piece():
    assert roles_end(barriers=2)


def test_roles_with_one_barrier_a_piece_would_not():
    assert not roles_end(barriers=1)
