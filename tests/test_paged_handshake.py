"""The handshakes between the softmax warps and the product issuers of the paged attention on
tcgen05, walked through every order in which the four actors of a CTA can run.

A segment has L key tiles; both groups take every tile, or (share) they take them in turn. A
group's softmax brings Q in and completes its q_full once per segment; its issuer waits for that by
parity, issues S of its tiles and, when P has arrived, the value products. At the end of a segment
the two softmax groups meet. An mbarrier shows the parity of its last phase alone: a waiter that is
two phases behind sees the one it waits for as still to come."""
import itertools

import pytest


def first_tile(share, n, g):
    return (n ^ g) & 1 if share else 0


def programs(segments, counted):
    """The steps of (softmax 0, softmax 1, issuer 0, issuer 1). counted(first, L): is q_full
    counted in a segment whose first tile of the group is `first`?"""
    out = []
    for g in (0, 1):
        own, q_at = [], []
        n = 0
        for L, share in segments:
            i0 = first_tile(share, n, g)
            own.append(len(range(i0, L, 2 if share else 1)))
            q_at.append(counted(i0, L))
            n += L
        softmax, issuer, tiles, qs = [], [], 0, 0
        if q_at[0]:
            softmax.append(("arrive", "q", g))
        for s, m in enumerate(own):
            if q_at[s]:
                issuer.append(("wait parity", "q", g, qs))
                qs += 1
            for _ in range(m):
                softmax += [("wait", "s", g, tiles), ("arrive", "p", g), ("wait", "o", g, tiles)]
                issuer += [("arrive", "s", g), ("wait", "p", g, tiles), ("arrive", "o", g)]
                tiles += 1
            softmax.append(("meet", s))
            if s + 1 < len(own) and q_at[s + 1]:
                softmax.append(("arrive", "q", g))
        out.append((softmax, issuer))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def fault(segments, counted):
    """The first fault in some order of running: a wait that passes for another phase than its
    own, or actors that wait for ever. None if there is none."""
    prog = programs(segments, counted)
    totals = [[{} for _ in range(len(p) + 1)] for p in prog]       # arrivals of an actor before its step i
    for a, p in enumerate(prog):
        for i, step in enumerate(p):
            totals[a][i + 1] = dict(totals[a][i])
            if step[0] == "arrive":
                totals[a][i + 1][step[1:]] = totals[a][i].get(step[1:], 0) + 1
    seen, todo = set(), [(0, 0, 0, 0)]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        moved = False
        for a in range(4):
            if at[a] == len(prog[a]):
                continue
            step = prog[a][at[a]]
            done = sum(totals[x][at[x]].get(step[1:3], 0) for x in range(4))
            nxt = list(at)
            nxt[a] += 1
            if step[0] == "wait" and done <= step[3]:
                continue
            if step[0] == "wait parity":
                if done & 1 == step[3] & 1:
                    continue                       # the phase shown is not the one waited for
                if done != step[3] + 1:
                    return "early", segments, at
            if step[0] == "meet":
                other = 1 - a
                if at[other] == len(prog[other]) or prog[other][at[other]] != step:
                    continue
                nxt[other] += 1
            moved = True
            todo.append(tuple(nxt))
        if not moved and any(at[a] < len(prog[a]) for a in range(4)):
            return "stuck", segments, at
    return None


SEGMENTS = [(L, share) for L in (0, 1, 2, 3) for share in (False, True)]


@pytest.mark.parametrize("count", [1, 2, 3, 4])
def test_q_counted_where_the_group_has_a_tile(count):
    for segments in itertools.product(SEGMENTS, repeat=count):
        assert fault(segments, lambda i0, L: i0 < L) is None


def test_q_counted_in_every_segment_gets_stuck():
    """What the rule is for: two shared segments of one tile, the second group's issuer late."""
    assert fault([(1, True), (1, True)], lambda i0, L: True)[0] == "stuck"
    assert fault([(0, False), (1, False)], lambda i0, L: True)[0] == "stuck"
    assert fault([(2, True), (3, False)], lambda i0, L: True) is None
