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


# ------------------------------------------------------------------ the loads that a block leaves behind
def fetches(pieces, per, st, stop):
    """The fetching warp's loads, as (barrier, phase) in order, up to the step at which it gives up, and what it keeps of
    them: (loads, tiles asked for, cleaned pieces, whether the last chunk is yet to be cleaned).  pieces: (chunks, whether
    the last one is cleaned after it landed)."""
    loads, asked, cleaned, unclean, m, step = [], 0, 0, False, 0, 0
    for chunks, ends_inside in pieces:
        for i in range(chunks):
            clean = ends_inside and i == chunks - 1
            for x in ([0, 2, 1] if per == 3 else [0, 1]):
                if step == stop:
                    return loads, asked, cleaned, unclean
                step += 1
                if x == 0:
                    unclean = clean
                asked += 1
                loads.append((("landed", x), cleaned) if clean and x < 2 else (("full", x, m % st), m // st))
            if clean:
                for x in (0, 1):
                    if step == stop:
                        return loads, asked, cleaned, unclean
                    step += 1
                unclean, cleaned = False, cleaned + 1
            m += 1
    return loads, asked, cleaned, unclean


@pytest.mark.parametrize("per, st", [(2, 3), (3, 2)])
def test_a_block_that_gives_up_waits_for_its_loads(per, st):
    """The barriers it waits for in the end cover the last load into every place (those before have been waited for by the
    warps that freed the place), in the phase of that load."""
    for pieces in itertools.product([(1, False), (1, True), (2, True), (5, False), (4, True)], repeat=3):
        steps = sum(per * n + 2 * c for n, c in pieces)
        for stop in range(steps + 1):
            loads, asked, cleaned, unclean = fetches(pieces, per, st, stop)
            waits = set()
            for i in range(max(asked - per * st, 0), asked):
                m, x = i // per, 0 if i % per == 0 else (1 if i % per == per - 1 else 2)
                landed = unclean and m == (asked - 1) // per and x < 2
                waits.add((("landed", x), cleaned) if landed else (("full", x, m % st), m // st))
            for (bar, phase), n in zip(loads, itertools.count()):
                if n < asked - per * st or (bar[0] == "landed" and phase < cleaned):
                    continue    # its place was freed since, or it was waited for before it was cleaned
                assert (bar, phase) in waits, (pieces, stop, bar, phase)
            # a barrier waited for in vain would hold the block up for two seconds: each has its load, or was signalled
            signalled = {(("full", x, m % st), m // st) for m in range(asked // per + 1) for x in (0, 1)}
            assert all(w in set(loads) or (w in signalled and not (unclean and w[0][1] < 2 and w[1] * st + w[0][2] == (asked - 1) // per))
                       for w in waits)
