"""The dK/dV kernel's barrier protocol (csrc/cross_bwd_sm100.cu) as a state machine.

Every role may stop for any time between two steps, so all interleavings are walked; an
mbarrier wait sees the parity of its barrier's phase only, as the hardware's does.  Copies
and the order of MMAs in the pipe are left out: they delay steps but release no waiter."""


def stuck_states(iterations, s_issued_barriers):
    """States in which no role can step though not all are done.

    s_issued_barriers: how many barriers `s_issued` goes round."""
    n = s_issued_barriers

    def wait(name, i):          # phase i of a barrier that every iteration completes once
        return ("wait", name, i & 1)

    def issued(kind, i):        # the same over n barriers in turn
        return (kind, "s_issued%d" % (i % n)) + (((i // n) & 1,) if kind == "wait" else ())

    s_dv, dp_dk, weights = [("arrive", "s_full")], [("arrive", "dp_full")], []
    for i in range(iterations):
        more = i + 1 < iterations
        s_dv += [wait("p_full", i)] + ([("arrive", "s_full")] if more else []) + [issued("arrive", i)]
        dp_dk += [wait("ds_full", i), issued("wait", i)] + ([("arrive", "dp_full")] if more else [])
        weights += [wait("s_full", i), ("arrive", "p_full"), wait("dp_full", i), ("arrive", "ds_full")]
    roles = (s_dv, dp_dk, weights)
    names = sorted({step[1] for role in roles for step in role})

    start = ((0,) * len(roles), (0,) * len(names))   # program counters, phases completed
    seen, todo, stuck = {start}, [start], []
    while todo:
        pcs, phases = todo.pop()
        moved = False
        for r, role in enumerate(roles):
            if pcs[r] == len(role):
                continue
            step = role[pcs[r]]
            b = names.index(step[1])
            if step[0] == "wait":
                if phases[b] & 1 == step[2]:     # the phase of that parity is still open
                    continue
                after = phases
            else:
                after = phases[:b] + (phases[b] + 1,) + phases[b + 1:]
            moved = True
            state = (pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], after)
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(pcs[r] < len(role) for r, role in enumerate(roles)):
            stuck.append(pcs)
    return stuck
