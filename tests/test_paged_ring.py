"""The ring of tile stages of the paged attention over e4m3 pages, as a model on the host: every order in which its
roles can run is followed, for pieces of one tile and of several.

A ring position is a piece's queries (two positions) or one of its tiles; position r lies in stage r % 4.  Barriers
are waited for by parity, as an mbarrier is: a wait for phase n passes when the phase under way is not of n's parity,
so a waiter that looks too late, after two phases, waits for good."""
import pytest

STAGES, QUERIES = 4, 2


class Bar:
    """count arrivals complete a phase."""

    def __init__(self, count):
        self.count = count


def ring(pieces, producers=2, score_waits_for_producers=True):
    """(barriers, roles): a role is its list of steps, (kind, ..), done in order."""
    bars = {}
    for s in range(STAGES):
        bars["raw_full", s] = Bar(1)                     # the load has landed
        bars["lat_full", s] = Bar(producers)             # the producers are done with it
        bars["lat_empty", s] = Bar(1)                    # the stage may be loaded again
    load, tma, score, pv, send = [], [], [], [], []
    prod = [[] for _ in range(producers)]

    def wait(name, r):
        return ("wait", (name, r % STAGES), r // STAGES)

    r = tiles = 0
    for k, n in enumerate(pieces):
        for q in range(QUERIES + n):
            if r >= STAGES:
                load.append(("wait", ("lat_empty", r % STAGES), r // STAGES - 1))
            load.append(("add", "issued"))
            tma += [("until", "issued", r + 1), ("fill", r), ("arrive", ("raw_full", r % STAGES))]
            for p in prod:
                p.append(wait("raw_full", r))
                if q >= QUERIES:
                    p.append(("read", r))
                p.append(("arrive", ("lat_full", r % STAGES)))
            if q < QUERIES:
                send += [wait("raw_full", r), ("read", r)]
                if q == QUERIES - 1:
                    send.append(("add", "q_ready"))
            else:
                if q == QUERIES:
                    score.append(("until", "q_ready", k + 1))
                    first = r - QUERIES
                    for x in range(first, r):
                        if score_waits_for_producers:
                            score.append(wait("lat_full", x))
                    for x in range(first, r):
                        score.append(("arrive", ("lat_empty", x % STAGES)))
                score += [wait("lat_full", r), ("read", r), ("add", "scores")]
                tiles += 1
                send.append(("until", "scores", tiles))  # the senders take a piece's scores before its successor
                pv += [("until", "scores", tiles), ("read", r), ("arrive", ("lat_empty", r % STAGES))]
            r += 1
    return bars, [load, tma, score, pv, send] + prod


def explore(bars, roles):
    """Follow every order of the roles' steps; the stuck states' counts of steps done."""
    names = sorted(bars)
    at = {b: i for i, b in enumerate(names)}
    counters = {"issued": 0, "q_ready": 1, "scores": 2}
    # (steps done by each role, (phase, arrivals) of each barrier, position in each stage, counters)
    start = ((0,) * len(roles), ((0, 0),) * len(names), (-1,) * STAGES, (0, 0, 0))
    seen, todo, stuck = {start}, [start], []
    while todo:
        pcs, bs, stage, cs = state = todo.pop()
        moved = False
        for i, steps in enumerate(roles):
            if pcs[i] == len(steps):
                continue
            step = steps[pcs[i]]
            nb, ns, nc = bs, stage, cs
            if step[0] == "wait":
                if (bs[at[step[1]]][0] & 1) == (step[2] & 1):
                    continue
            elif step[0] == "until":
                if cs[counters[step[1]]] < step[2]:
                    continue
            elif step[0] == "arrive":
                j = at[step[1]]
                phase, n = bs[j]
                n += 1
                nb = bs[:j] + ((phase + 1, 0) if n == bars[step[1]].count else (phase, n),) + bs[j + 1:]
            elif step[0] == "fill":
                ns = tuple(step[1] if s == step[1] % STAGES else x for s, x in enumerate(stage))
            elif step[0] == "read":
                assert stage[step[1] % STAGES] == step[1], f"role {i} reads {stage} for position {step[1]}"
            else:
                j = counters[step[1]]
                nc = cs[:j] + (cs[j] + 1,) + cs[j + 1:]
            moved = True
            new = (pcs[:i] + (pcs[i] + 1,) + pcs[i + 1:], nb, ns, nc)
            if new not in seen:
                seen.add(new)
                todo.append(new)
        if not moved and any(p < len(s) for p, s in zip(pcs, roles)):
            stuck.append(pcs)
    return stuck


@pytest.mark.parametrize("pieces", [[1], [1, 1, 1], [2, 1], [3, 1], [1, 4], [5]], ids=str)
def test_the_ring_always_goes_on(pieces):
    assert explore(*ring(pieces)) == []


def test_queries_released_without_the_producers_stop_the_ring():
    """The model finds what the score warp's wait for the producers is there for: a producer that has not looked at
    the queries' load when the next load into their stage lands, waits for good."""
    assert explore(*ring([3], score_waits_for_producers=False))
