"""Barrier schedules of the tensor-core passes of differential attention
(csrc/diff_tc.cu), explored on the CPU over every order in which their roles
can run.

A model of one thread block: a producer whose loads land at any later time and
in any order, an MMA issuer, the tensor pipe (which runs what is issued in order,
at any later time) and two elementwise warps, one of which may fall behind the
other without limit.  mbarriers behave as on the
device: a wait knows its phase by parity only, and an arrival counts for
whatever phase is current.  Every reachable state is held to:
  - a waiter finds its barrier in the awaited phase or the one after: further on
    it would wait for what cannot come, and one phase short of it the parity
    reads as if the awaited phase were over;
  - an arrival for tile a lands in the phase of tile a;
  - products and warps find in tensor memory and in the ring of stages what
    the tile they work on put there;
  - every role reaches its end.
"""
import pytest

WARPS = 2


class Violation(Exception):
    pass


def explore(roles, counts):
    """Runs `roles` (name -> list of steps) in every order.  Steps:
      ("wait", bar, n)         until phase n of bar has completed
      ("arrive", bar, n)       one of counts[bar] arrivals of phase n
      ("load", bar, n, writes) a copy, which arrives when it lands
      ("issue", reads, writes) a product, run later in order by the pipe
      ("commit", bar, n)       an arrival behind everything issued before
      ("read", cell, value) and ("write", cell, value)
    Returns the number of states."""
    names = list(roles)
    bars = list(counts)
    start = (tuple(0 for _ in names), tuple((0, 0) for _ in bars), (), frozenset(), frozenset())
    at = {b: i for i, b in enumerate(bars)}
    seen, todo = {start}, [start]

    def arrive(bs, bar, n):
        i = at[bar]
        done, have = bs[i]
        if done != n:
            raise Violation(f"arrival of phase {n} of {bar} counts for phase {done}")
        have += 1
        new = (done + 1, 0) if have == counts[bar] else (done, have)
        return bs[:i] + (new,) + bs[i + 1:]

    def expect(cells, reads, who):
        for cell, value in reads:
            if cells.get(cell) != value:
                raise Violation(f"{who}: {cell} holds {cells.get(cell)}, not {value}")

    while todo:
        pcs, bs, queue, mem, flying = todo.pop()
        cells = dict(mem)
        out = []
        for r, name in enumerate(names):
            if pcs[r] == len(roles[name]):
                continue
            step = roles[name][pcs[r]]
            kind = step[0]
            nbs, nq, nm, nf = bs, queue, mem, flying
            if kind == "wait":
                done = bs[at[step[1]]][0]
                if done not in (step[2], step[2] + 1):
                    raise Violation(f"{name} waits for phase {step[2]} of {step[1]}, which is in {done}")
                if done == step[2]:
                    continue
            elif kind == "arrive":
                nbs = arrive(bs, step[1], step[2])
            elif kind == "load":
                nf = flying | {(r, pcs[r])}
                nm = frozenset({**cells, **{cell: "on its way" for cell, _ in step[3]}}.items())
            elif kind in ("issue", "commit"):
                nq = queue + ((r, pcs[r]),)
            elif kind == "read":
                expect(cells, [step[1:]], name)
            else:
                new = dict(cells)
                new[step[1]] = step[2]
                nm = frozenset(new.items())
            out.append((pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], nbs, nq, nm, nf))
        for role, pc in flying:
            _, bar, n, writes = roles[names[role]][pc]
            out.append((pcs, arrive(bs, bar, n), queue, frozenset({**cells, **dict(writes)}.items()),
                        flying - {(role, pc)}))
        if queue:
            role, pc = queue[0]
            step, nbs, nm = roles[names[role]][pc], bs, mem
            if step[0] == "commit":
                nbs = arrive(bs, step[1], step[2])
            else:
                expect(cells, step[1], "pipe")
                new = dict(cells)
                new.update(step[2])
                nm = frozenset(new.items())
            out.append((pcs, nbs, queue[1:], nm, flying))
        if not out and any(pcs[r] < len(roles[n]) for r, n in enumerate(names)):
            stuck = [f"{n}: {roles[n][pcs[r]]}" for r, n in enumerate(names) if pcs[r] < len(roles[n])]
            raise Violation("nothing can run: " + "; ".join(stuck))
        for s in out:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


def explore_abort(roles, counts, producer_looks):
    """Any wait may run out and raise the block's flag.  From then on the MMA
    warp's waits return at once, and it goes on with whatever the buffers hold;
    the producer stops at a wait that runs out, and (where it looks) behind one
    that did not if the flag is up.  No copy may be started on a barrier whose
    last copy has not landed: it would arrive once more than the barrier counts.
    Contents do not matter any more, nor what the elementwise warps do (the first
    wait for them runs out), and a commit may as well arrive when it is issued:
    the MMA warp takes as long as it likes."""
    names = ["producer", "mma"]
    steps = {n: [x for x in roles[n] if x[0] not in ("issue", "read", "write")] for n in names}
    bars = list(counts)
    at = {b: i for i, b in enumerate(bars)}
    start = ((0, 0), tuple((0, 0) for _ in bars), frozenset(), False)
    seen, todo = {start}, [start]

    def arrive(bs, bar):
        done, have = bs[at[bar]]
        new = (done + 1, 0) if have + 1 == counts[bar] else (done, have + 1)
        return bs[:at[bar]] + (new,) + bs[at[bar] + 1:]

    while todo:
        pcs, bs, flying, flag = todo.pop()
        out = []
        for r, name in enumerate(names):
            if pcs[r] == len(steps[name]):
                continue
            step = steps[name][pcs[r]]
            nbs, nf, after = bs, flying, [(pcs[r] + 1, flag)]
            if step[0] == "wait":
                over = (bs[at[step[1]]][0] & 1) != (step[2] & 1)  # what the parity tells
                if name == "producer":
                    end = len(steps[name])
                    after = [(end if flag and producer_looks else pcs[r] + 1, flag)] if over else [(end, True)]
                elif not over and not flag:
                    after = [(pcs[r] + 1, True)]
            elif step[0] == "load":
                if any(steps["producer"][pc][1] == step[1] for pc in flying):
                    raise Violation(f"a copy on {step[1]} is started before the last one has landed")
                nf = flying | {pcs[r]}
            else:
                nbs = arrive(bs, step[1])
            for pc, f in after:
                out.append((pcs[:r] + (pc,) + pcs[r + 1:], nbs, nf, f))
        for pc in flying:
            out.append((pcs, arrive(bs, steps["producer"][pc][1]), flying - {pc}, flag))
        for s in out:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


# A tensor-memory block is one cell per warp (its columns or lanes); a product
# reads and writes all of them.
def block(name, value):
    return [((name, w), value) for w in range(WARPS)]


def producer(T, stages):
    steps = []
    for a in range(T):
        if a >= stages:
            steps.append(("wait", ("empty", a % stages), a // stages - 1))
        steps.append(("load", ("full", a % stages), a // stages, ((("tile", a % stages), a),)))
    return steps


def ring_counts(stages, full="full", empty="empty"):
    return {(k, s): 1 for k in (full, empty) for s in range(stages)}


def column_narrow(T, stages=4, s2_full=2, ds2_full=2):
    """d <= 64: S^T of map 2 has two buffers, and a barrier for each, for its
    scores and for the operands that go over them."""
    pairs = {"s2_full": s2_full, "ds2_full": ds2_full}

    def second(bar, a):
        return (bar, a % pairs[bar]), a // pairs[bar]

    def tile(a):
        return (("tile", a % stages), a)

    def scores(a):
        return [("issue", [tile(a)], block("S1", ("S", a))), ("commit", "s_full", a),
                ("issue", [tile(a)], block(("S2", a & 1), ("S", a))), ("commit", *second("s2_full", a))]

    def dp(a):
        return ("issue", [tile(a)], block("dP", a))

    mma = [("wait", ("full", 0), 0), dp(0)] + scores(0)
    for a in range(T):
        more = a + 1 < T
        if more:
            mma += [("wait", "dp_read", a), dp(a + 1)]
        mma += [("wait", "ds_full", a), ("issue", [tile(a)] + block("S1", ("dS", a)), [])]
        if more:
            mma += scores(a + 1)
        mma += [("wait", *second("ds2_full", a)),
                ("issue", [tile(a)] + block(("S2", a & 1), ("dS", a)), []),
                ("commit", ("empty", a % stages), a // stages)]
    roles = {"producer": producer(T, stages), "mma": mma}
    for w in range(WARPS):
        steps = [("wait", ("full", 0), 0)]
        for a in range(T):
            if a + 1 < T:
                steps.append(("wait", ("full", (a + 1) % stages), (a + 1) // stages))
            s2 = (("S2", a & 1), w)
            steps += [("wait", "s_full", a), ("read", ("S1", w), ("S", a)), ("read", ("dP", w), a),
                      ("arrive", "dp_read", a), ("read", *tile(a)), ("write", ("S1", w), ("dS", a)),
                      ("arrive", "ds_full", a), ("wait", *second("s2_full", a)), ("read", s2, ("S", a)),
                      ("read", *tile(a)), ("write", s2, ("dS", a)), ("arrive", *second("ds2_full", a))]
        roles[f"warp {w}"] = steps
    counts = ring_counts(stages)
    counts.update({"s_full": 1, "dp_read": WARPS, "ds_full": WARPS})
    counts.update({("s2_full", b): 1 for b in range(s2_full)})
    counts.update({("ds2_full", b): WARPS for b in range(ds2_full)})
    return roles, counts


def column_wide(T, stages=2):
    """d > 64: S^T of map 2 goes over dP^T."""
    def tile(a):
        return (("tile", a % stages), a)

    def s1(a):
        return ("issue", [tile(a)], block("S1", ("S", a)))

    def dp(a):
        return ("issue", [tile(a)], block("dP", ("dP", a)))

    mma = [("wait", ("full", 0), 0), s1(0), dp(0), ("commit", "s_full", 0)]
    for a in range(T):
        more = a + 1 < T
        mma += [("wait", "dp_read", a), ("issue", [tile(a)], block("dP", ("S", a))),
                ("commit", "s2_full", a)]
        if more:
            mma.append(("wait", ("full", (a + 1) % stages), (a + 1) // stages))
        mma += [("wait", "ds_full", a), ("issue", [tile(a)] + block("S1", ("dS", a)), [])]
        if more:
            mma.append(s1(a + 1))
        mma += [("wait", "ds2_full", a), ("issue", [tile(a)] + block("dP", ("dS", a)), []),
                ("commit", ("empty", a % stages), a // stages)]
        if more:
            mma += [dp(a + 1), ("commit", "s_full", a + 1)]
    roles = {"producer": producer(T, stages), "mma": mma}
    for w in range(WARPS):
        steps = []
        for a in range(T):
            steps += [("wait", ("full", a % stages), a // stages), ("wait", "s_full", a),
                      ("read", ("S1", w), ("S", a)), ("read", ("dP", w), ("dP", a)),
                      ("arrive", "dp_read", a), ("read", *tile(a)), ("write", ("S1", w), ("dS", a)),
                      ("arrive", "ds_full", a), ("wait", "s2_full", a), ("read", ("dP", w), ("S", a)),
                      ("read", *tile(a)), ("write", ("dP", w), ("dS", a)), ("arrive", "ds2_full", a)]
        roles[f"warp {w}"] = steps
    counts = ring_counts(stages)
    counts.update({"s_full": 1, "s2_full": 1, "dp_read": WARPS, "ds_full": WARPS, "ds2_full": WARPS})
    return roles, counts


def row(T, k_stages=3, v_stages=2):
    def k(t):
        return (("k", t % k_stages), t)

    def v(t):
        return (("v", t % v_stages), t)

    def s(t, m):
        return ("issue", [k(t)], block(f"S{m}", ("S", t)))

    def dp(t):
        return [("issue", [v(t)], block("dP", t)), ("commit", ("v_empty", t % v_stages), t // v_stages)]

    def dq(t, m):
        return ("issue", [k(t)] + block(f"S{m}", ("dS", t)), [])

    mma = [("wait", ("full", 0), 0)] + dp(0) + [s(0, 0), ("commit", "s_full", 0)]
    for t in range(T):
        more = t + 1 < T
        mma += [s(t, 1), ("commit", "s2_full", t)]
        if more:
            mma += [("wait", "dp_read", t)] + dp(t + 1)
        mma += [("wait", "ds_full", t), dq(t, 0)]
        if more:
            mma += [s(t + 1, 0), ("commit", "s_full", t + 1)]
        mma += [("wait", "ds2_full", t), dq(t, 1), ("commit", ("k_empty", t % k_stages), t // k_stages)]
    load = []
    for t in range(T):
        if t >= v_stages:
            load.append(("wait", ("v_empty", t % v_stages), t // v_stages - 1))
        if t >= k_stages:
            load.append(("wait", ("k_empty", t % k_stages), t // k_stages - 1))
        load.append(("load", ("full", t % k_stages), t // k_stages, (v(t), k(t))))
    roles = {"producer": load, "mma": mma}
    for w in range(WARPS):
        steps = []
        for t in range(T):
            if w == 0 and t + 1 < T:
                steps.append(("wait", ("full", (t + 1) % k_stages), (t + 1) // k_stages))
            steps += [("wait", "s_full", t), ("read", ("S0", w), ("S", t)), ("read", ("dP", w), t),
                      ("arrive", "dp_read", t), ("write", ("S0", w), ("dS", t)), ("arrive", "ds_full", t),
                      ("wait", "s2_full", t), ("read", ("S1", w), ("S", t)), ("write", ("S1", w), ("dS", t)),
                      ("arrive", "ds2_full", t)]
        roles[f"warp {w}"] = steps
    counts = {(b, i): 1 for b, n in (("full", k_stages), ("k_empty", k_stages), ("v_empty", v_stages))
              for i in range(n)}
    counts.update({"s_full": 1, "s2_full": 1, "dp_read": WARPS, "ds_full": WARPS, "ds2_full": WARPS})
    return roles, counts


def forward(T, one, early=False):
    """Warp m holds map m's rows.  one: a stage holds K^1, K^2 and V; otherwise
    a ring of three K^m and one of two V, whose loads a warp awaits behind its
    scores (early: before them)."""
    vs, ks = 3 if one else 2, 3

    def k(t, m):
        return (("v", t % vs), t) if one else (("k", (2 * t + m) % ks), 2 * t + m)

    def s(t, m):
        out = [("issue", [k(t, m)], [(("S", m), ("S", t, 0)), (("Sb", m), ("S", t, 1))]),
               ("commit", ("s_full", m), t)]
        if not one:
            u = 2 * t + m
            out.append(("commit", ("k_empty", u % ks), u // ks))
        return out

    mma = [("wait", ("v_full", 0), 0)] if one else [("wait", ("k_full", 0), 0), ("wait", ("k_full", 1), 0)]
    mma += s(0, 0) + s(0, 1)
    for t in range(T):
        for m in (0, 1):
            for half, cell in ((0, "S"), (1, "Sb")):
                last = [(("O", m), t)] if half else []
                mma += [("wait", ("p_full", m, half), t),
                        ("issue", [(("v", t % vs), t), ((cell, m), ("P", t, half))], last)]
            if m == 1:
                mma.append(("commit", ("v_empty", t % vs), t // vs))
            if t + 1 < T:
                mma += s(t + 1, m)
    load = []
    for t in range(T):
        if not one:
            for u in (2 * t, 2 * t + 1):
                if u >= ks:
                    load.append(("wait", ("k_empty", u % ks), u // ks - 1))
                load.append(("load", ("k_full", u % ks), u // ks, ((("k", u % ks), u),)))
        if t >= vs:
            load.append(("wait", ("v_empty", t % vs), t // vs - 1))
        load.append(("load", ("v_full", t % vs), t // vs, ((("v", t % vs), t),)))
    roles = {"producer": load, "mma": mma}
    for m in (0, 1):
        steps = []
        for t in range(T):
            scores = [("wait", ("s_full", m), t), ("read", ("S", m), ("S", t, 0)),
                      ("read", ("Sb", m), ("S", t, 1))]
            if t > 0:  # O is rescaled where the maximum moves
                scores.append(("read", ("O", m), t - 1))
            tile, key = [], []
            if one and m == 0 and t + 1 < T:
                tile = [("wait", ("v_full", (t + 1) % vs), (t + 1) // vs)]
            elif not one:
                u = 2 * (t + 1) + m
                tile = [("wait", ("v_full", t % vs), t // vs)] if m == 0 else []
                key = [("wait", ("k_full", u % ks), u // ks)] if t + 1 < T else []
            if one or early:
                steps += tile + key + scores
                tile, key = [], []
            else:
                steps += scores
            steps += [("write", ("S", m), ("P", t, 0))] + tile + [("arrive", ("p_full", m, 0), t)]
            steps += [("write", ("Sb", m), ("P", t, 1))] + key + [("arrive", ("p_full", m, 1), t)]
        roles[f"map {m}"] = steps
    counts = {("s_full", m): 1 for m in (0, 1)}
    counts.update({("p_full", m, h): 1 for m in (0, 1) for h in (0, 1)})
    counts.update(ring_counts(vs, "v_full", "v_empty"))
    if not one:
        counts.update(ring_counts(ks, "k_full", "k_empty"))
    return roles, counts


@pytest.mark.parametrize("schedule", [
    lambda: column_narrow(5), lambda: column_narrow(5, stages=2), lambda: column_wide(5), lambda: row(5),
    lambda: forward(5, True), lambda: forward(5, False)],
    ids=["dK_dV", "dK_dV_two_stages", "dK_dV_wide", "dQ", "forward", "forward_wide"])
def test_schedule_holds_in_every_order(schedule):
    roles, counts = schedule()
    assert explore(roles, counts) > 100


@pytest.mark.parametrize("s2_full,ds2_full", [(1, 1), (1, 2), (2, 1)])
def test_one_barrier_for_two_buffers_is_found(s2_full, ds2_full):
    """With one barrier for the scores, a warp that falls behind is overtaken
    by a phase; with one for the operands, the MMA warp is, or a faster warp's
    arrival for the next tile counts for this one."""
    with pytest.raises(Violation):
        explore(*column_narrow(5, s2_full=s2_full, ds2_full=ds2_full))


def test_a_load_awaited_too_early_is_found():
    """Before its scores a warp does not know that the ring slot's earlier load
    has landed: the parity of the phase before the awaited one is that of the
    phase after it, and the wait returns with the keys still on their way."""
    with pytest.raises(Violation, match="k_full"):
        explore(*forward(5, False, early=True))


def test_planted_mistakes_are_found():
    """A product issued without its operands' wait, and an early refill."""
    roles, counts = column_narrow(4)
    roles["mma"].remove(("wait", "ds_full", 2))
    with pytest.raises(Violation):
        explore(roles, counts)
    roles, counts = row(4)
    roles["producer"] = [s for s in roles["producer"] if s[0] != "wait" or s[1][0] != "v_empty"]
    with pytest.raises(Violation):
        explore(roles, counts)
    roles, counts = forward(4, True)
    roles["mma"].remove(("wait", ("p_full", 1, 1), 1))
    with pytest.raises(Violation):
        explore(roles, counts)


# tiles enough that every ring is filled once more
ABORTING = {"dK_dV": lambda: column_narrow(6), "dK_dV_wide": lambda: column_wide(4), "dQ": lambda: row(5),
            "forward": lambda: forward(5, True), "forward_wide": lambda: forward(4, False)}


@pytest.mark.parametrize("name", ABORTING)
def test_a_wait_that_runs_out_starts_no_copy_too_many(name):
    assert explore_abort(*ABORTING[name](), producer_looks=True) > 100


@pytest.mark.parametrize("name", ABORTING)
def test_a_producer_that_does_not_look_is_found(name):
    """Behind the flag the MMA warp's commits free stages that are not filled yet."""
    with pytest.raises(Violation, match="before the last one has landed"):
        explore_abort(*ABORTING[name](), producer_looks=False)
