"""The barriers between the roles of the latent-attention kernels, as a model on the CPU: every order in which
the roles, the copies and the MMAs can take their steps.

A role is the list of its steps, in the order of the kernel's code.  A wait knows which phase of its barrier it is
for, but passes, as the hardware's does, by that phase's parity alone.  Checked in every state that can be
reached: no wait passes before its phase, or stays shut behind it; operands and results hold what their readers take
them for, from issue to completion of an MMA; nothing stops short of its end."""
import pytest


class Fault(Exception):
    pass


def wait(bar, phase):
    return ("wait", bar, phase)


def explore(roles, counts):
    """Walks all interleavings of `roles` ({name: steps}); `counts`: arrivals that complete a phase (1 where not given).
    Steps: ("wait", bar, phase), ("arrive", bar), ("copy", bar, place, tag), ("mma", reads, writes) and ("commit", bar)
    (both asynchronous, in a role's order), ("read", place, tag), ("write", place, tag), and ("note", place, tag): a write
    that others may rely on from the role's next own arrival on, as a copy's arrival or a commit's does not publish it."""
    progs = list(roles.values())
    bars = sorted({s[1] for p in progs for s in p if s[0] in ("wait", "arrive", "copy", "commit")})
    index = {b: i for i, b in enumerate(bars)}
    places = sorted({s[2] for p in progs for s in p if s[0] == "copy"} | {s[1] for p in progs for s in p if s[0] in ("read", "write", "note")} |
                    {x for p in progs for s in p if s[0] == "mma" for part in s[1:] for x, _ in part})
    where = {x: i for i, x in enumerate(places)}
    need = [counts.get(b, 1) for b in bars]
    issued = [[s for s in p if s[0] in ("mma", "commit")] for p in progs]      # a role's MMAs and commits, in order
    before = [[0] * (len(p) + 1) for p in progs]
    for p, prog in enumerate(progs):
        for i, s in enumerate(prog):
            before[p][i + 1] = before[p][i] + (s[0] in ("mma", "commit"))
    notes = []                                       # what an arrival publishes, by role and step
    for prog in progs:
        notes.append([])
        held = []
        for s in prog:
            notes[-1].append(tuple(held))
            held = [] if s[0] == "arrive" else held + [s[1:]] if s[0] == "note" else held
    # state: steps done by each role, MMAs and commits completed of each, copies in flight, (phases, arrivals), tags; what
    # a role has noted and not published follows from its steps
    start = ((0,) * len(progs), (0,) * len(progs), frozenset(), ((0, 0),) * len(bars), (None,) * len(places))

    def arrive(state, b):
        i = index[b]
        done, n = state[i]
        n += 1
        state = list(state)
        state[i] = (done + 1, 0) if n == need[i] else (done, n)
        return tuple(state)

    def put(tags, x, tag):
        tags = list(tags)
        tags[where[x]] = tag
        return tuple(tags)

    def moves(state):
        pcs, fin, copies, bs, tags = state
        for p, prog in enumerate(progs):
            # nobody sees a commit's issue or a note: taken at once
            if pcs[p] < len(prog) and prog[pcs[p]][0] in ("commit", "note"):
                yield (pcs[:p] + (pcs[p] + 1,) + pcs[p + 1:], fin, copies, bs, tags)
                return
        for p, prog in enumerate(progs):
            if fin[p] < before[p][pcs[p]]:
                s = issued[p][fin[p]]
                f = fin[:p] + (fin[p] + 1,) + fin[p + 1:]
                if s[0] == "commit":
                    yield (pcs, f, copies, arrive(bs, s[1]), tags)
                else:
                    t = tags
                    for x, tag in s[1]:
                        if tags[where[x]] != tag:
                            raise Fault(f"an MMA ends with {x} = {tags[where[x]]} for {tag}")
                    for x, tag in s[2]:
                        t = put(t, x, tag)
                    yield (pcs, f, copies, bs, t)
            if pcs[p] == len(prog):
                continue
            s = prog[pcs[p]]
            nxt = pcs[:p] + (pcs[p] + 1,) + pcs[p + 1:]
            if s[0] == "wait":
                done = bs[index[s[1]]][0]
                if ((done - 1) & 1) == (s[2] & 1):
                    if done <= s[2]:
                        raise Fault(f"{s[1]} passed before phase {s[2]}: {done} complete")
                    yield (nxt, fin, copies, bs, tags)
                elif done > s[2]:
                    raise Fault(f"{s[1]} shut behind phase {s[2]}: {done} complete")
            elif s[0] == "arrive":
                t = tags
                for x, tag in notes[p][pcs[p]]:
                    t = put(t, x, tag)
                yield (nxt, fin, copies, arrive(bs, s[1]), t)
            elif s[0] == "copy":
                yield (nxt, fin, copies | {s[1:]}, bs, put(tags, s[2], "arriving"))
            elif s[0] == "read":
                if tags[where[s[1]]] != s[2]:
                    raise Fault(f"{s[1]} holds {tags[where[s[1]]]}, read for {s[2]}")
                yield (nxt, fin, copies, bs, tags)
            elif s[0] == "write":
                yield (nxt, fin, copies, bs, put(tags, s[1], s[2]))
            else:
                t = tags
                for x, tag in s[1]:
                    if tags[where[x]] != tag:
                        raise Fault(f"an MMA reads {x} = {tags[where[x]]} for {tag}")
                for x, tag in s[2]:
                    t = put(t, x, ("under way", tag))
                yield (nxt, fin, copies, bs, t)
        for c in copies:
            yield (pcs, fin, copies - {c}, arrive(bs, c[0]), put(tags, c[1], c[2]))

    seen, todo = {start}, [start]
    end = tuple(len(p) for p in progs)
    while todo:
        state = todo.pop()
        any_move = False
        for n in moves(state):
            any_move = True
            if n not in seen:
                seen.add(n)
                todo.append(n)
        if not any_move and state[0] != end:
            raise Fault(f"stuck at {[p[i] if i < len(p) else 'end' for p, i in zip(progs, state[0])]}")
    return len(seen)


def dq_roles(tiles, waits_ahead=True, exact=2):
    """latent_dq_kernel: K in three stages, V in two; two element-wise halves.  `waits_ahead`: the steps of
    the pass ahead wait for the step before them as the others do."""
    ahead = tiles if tiles <= exact else 0
    steps = ahead + tiles
    produce, first, second, halves = [], [], [], [[], []]
    for i in range(steps):
        k, v = i % 3, i % 2
        if i >= 3:
            produce.append(wait(f"k_empty{k}", i // 3 - 1))
        produce.append(("copy", f"k_full{k}", f"K{k}", i))
        if i >= 2:
            produce.append(wait(f"v_empty{v}", i // 2 - 1))
        produce.append(("copy", f"v_full{v}", f"V{v}", i))
        first.append(wait(f"k_full{k}", i // 3))
        if i > 0:
            first.append(wait("s_free", i - 1))
        first += [("mma", ((f"K{k}", i),), (("S0", i), ("S1", i))), ("commit", "s_ready"), wait(f"v_full{v}", i // 2)]
        if i > 0:
            first.append(wait("dp_free", i - 1))
        first += [("mma", ((f"V{v}", i),), (("dP0", i), ("dP1", i))), ("commit", f"v_empty{v}"), ("commit", "dp_ready")]
        second.append(wait("ds_ready", i))
        if i >= ahead:
            second.append(("mma", (("dS0", i), ("dS1", i), (f"K{k}", i)), (("dQ", i),)))
        second += [("commit", f"k_empty{k}"), ("commit", "dq_done")]
        for h, e in enumerate(halves):
            e += [wait("s_ready", i), ("read", f"S{h}", i), ("arrive", "s_free"), wait("dp_ready", i), ("read", f"dP{h}", i),
                  ("arrive", "dp_free")]
            if i < ahead:
                if i == ahead - 1:
                    e += [("arrive", "named"), wait("named", 0)]
                if waits_ahead and i > 0:
                    e.append(wait("dq_done", i - 1))
            else:
                if i > 0:
                    e.append(wait("dq_done", i - 1))
                e.append(("write", f"dS{h}", i))
            e.append(("arrive", "ds_ready"))
    for e in halves:
        e += [wait("dq_done", steps - 1), ("read", "dQ", steps - 1)]
    counts = dict.fromkeys(("s_free", "dp_free", "ds_ready", "named"), 2)
    return dict(produce=produce, first=first, second=second, e0=halves[0], e1=halves[1]), counts


def dkv_roles(steps, stages=3):
    """latent_dkv_kernel: Q, dO and their statistics in three stages."""
    produce, first, second, halves = [], [], [], [[], []]
    for i in range(steps):
        s = i % stages
        if i >= stages:
            produce.append(wait(f"q_empty{s}", i // stages - 1))
        produce.append(("copy", f"q_full{s}", f"Q{s}", i))
        first.append(wait(f"q_full{s}", i // stages))
        if i > 0:
            first.append(wait("s_free", i - 1))
        first += [("mma", ((f"Q{s}", i),), (("S0", i), ("S1", i))), ("commit", "s_ready")]
        if i > 0:
            first.append(wait("dp_free", i - 1))
        first += [("mma", ((f"Q{s}", i),), (("dP0", i), ("dP1", i))), ("commit", "dp_ready")]
        second += [wait("p_ready", i), ("mma", (("P0", i), ("P1", i), (f"Q{s}", i)), (("dV", i),)), ("commit", "dv_done"),
                   wait("ds_ready", i), ("mma", (("dS0", i), ("dS1", i), (f"Q{s}", i)), (("dK", i),)),
                   ("commit", f"q_empty{s}"), ("commit", "dk_done")]
        for h, e in enumerate(halves):
            e += [wait("s_ready", i), ("read", f"S{h}", i), ("arrive", "s_free"), wait(f"q_full{s}", i // stages),
                  ("read", f"Q{s}", i)]
            if i > 0:
                e.append(wait("dv_done", i - 1))
            e += [("write", f"P{h}", i), ("arrive", "p_ready"), wait("dp_ready", i), ("read", f"dP{h}", i),
                  ("arrive", "dp_free"), ("read", f"Q{s}", i)]
            if i > 0:
                e.append(wait("dk_done", i - 1))
            e += [("write", f"dS{h}", i), ("arrive", "ds_ready")]
    for e in halves:
        e += [wait("dk_done", steps - 1), ("read", "dV", steps - 1), ("read", "dK", steps - 1)]
    counts = dict.fromkeys(("s_free", "dp_free", "p_ready", "ds_ready"), 2)
    return dict(produce=produce, first=first, second=second, e0=halves[0], e1=halves[1]), counts


def prefill_roles(n0, n1, stages=2):
    """latent_prefill_kernel: two query tiles that see n0 and n1 key tiles, K and V in two stages."""
    nt, n = max(n0, n1), (n0, n1)
    produce, scores, values, soft = [], [], [], [[], []]
    if n0:
        produce.append(("copy", "q_full0", "Q0", 0))
    for j in range(nt):
        s = j % stages
        if j >= stages:
            produce.append(wait(f"k_empty{s}", j // stages - 1))
        produce.append(("copy", f"k_full{s}", f"K{s}", j))
        if j == 0 and n1:
            produce.append(("copy", "q_full1", "Q1", 0))
        if j >= stages:
            produce.append(wait(f"v_empty{s}", j // stages - 1))
        produce.append(("copy", f"v_full{s}", f"V{s}", j))
        scores.append(wait(f"k_full{s}", j // stages))
        values.append(wait(f"v_full{s}", j // stages))
        for q in (0, 1):
            if j >= n[q]:
                continue
            scores += [wait(f"s_free{q}", j - 1) if j else wait(f"q_full{q}", 0),
                       ("mma", ((f"Q{q}", 0), (f"K{s}", j)), ((f"S{q}", j),)), ("commit", f"s_ready{q}")]
            values += [wait(f"p_ready{q}", j), ("mma", ((f"P{q}", j), (f"V{s}", j)), ((f"O{q}", j),)), ("commit", f"pv_done{q}")]
            soft[q] += [wait(f"s_ready{q}", j), ("read", f"S{q}", j), ("arrive", f"s_free{q}")]
            if j:
                soft[q] += [wait(f"pv_done{q}", j - 1), ("read", f"O{q}", j - 1)]
            soft[q].append(("write", f"P{q}", j))
            if j == nt - 1:                               # rows of V behind the sequence are zeroed
                soft[q] += [wait(f"v_full{s}", j // stages), ("read", f"V{s}", j)]
            soft[q].append(("arrive", f"p_ready{q}"))
        scores.append(("commit", f"k_empty{s}"))
        values.append(("commit", f"v_empty{s}"))
    for q in (0, 1):
        if n[q]:
            soft[q] += [wait(f"pv_done{q}", n[q] - 1), ("read", f"O{q}", n[q] - 1)]
    return dict(produce=produce, scores=scores, values=values, s0=soft[0], s1=soft[1]), {}


def decode_roles(segments, shared, publishes=True, slots=4, ns=2):
    """latent_decode_kernel: segments of as many tiles, a tile in `ns` slots, two copying warps and two halves of the
    softmax.  The MMA thread takes what can go next: a role for the scores and one for the values, which knows more
    orders than the thread has.  `publishes`: the copying warps arrive for their masks themselves."""
    copy, scores, values, soft, queries = [[], []], [], [], [[], []], []
    it = 0
    for seg, tiles in enumerate(segments):
        if seg:
            queries.append(wait("q_empty", seg - 1))
        queries.append(("copy", "q_full", "Q", seg))
        for t in range(tiles):
            first = it * ns % slots
            for w, c in enumerate(copy):
                c.append(("note", f"seen{it % 16}.{w}", it))
                for n in range(ns):
                    at = it * ns + n
                    if n == ns - 1 and it >= shared:
                        c.append(wait(f"s_full{(it - shared) & 1}", (it - shared) >> 1))
                    if at >= slots:
                        c.append(wait(f"empty{at % slots}", at // slots - 1))
                    c.append(("copy", f"full{at % slots}", f"L{at % slots}.{w}", it))
                    if n == ns - 1:
                        c.append(("copy", f"full{at % slots}", f"R{it % shared}.{w}", it))
                    if publishes:
                        c.append(("arrive", f"full{at % slots}"))
            if it >= 2:
                scores.append(wait(f"values{it - 2}", 0))
            for n in range(ns):
                at = it * ns + n
                scores.append(wait(f"full{at % slots}", at // slots))
                if t == 0 and n == 0:
                    scores.append(wait("q_full", seg))
                own = [(f"L{at % slots}.{w}", it) for w in (0, 1)]
                if n == ns - 1:
                    own += [(f"R{it % shared}.{w}", it) for w in (0, 1)]
                scores.append(("mma", (("Q", seg), *own), ((f"S{it & 1}.0", it), (f"S{it & 1}.1", it))))
            scores += [("commit", f"s_full{it & 1}"), ("arrive", f"scores{it}")]
            if t == tiles - 1:
                scores.append(("commit", "q_empty"))
            values += [wait(f"scores{it}", 0), wait("p_ready", it)]
            if t == 0 and seg:
                values.append(wait("o_empty", seg - 1))
            for n in range(ns):
                at = it * ns + n
                own = [(f"L{at % slots}.{w}", it) for w in (0, 1)]
                values += [("mma", (("P0", it), ("P1", it), *own), ((f"O{n}", it),)), ("commit", f"empty{at % slots}")]
            values += [("commit", "pv_done"), ("arrive", f"values{it}")]
            for h, e in enumerate(soft):
                e += [wait(f"s_full{it & 1}", it >> 1), ("read", f"S{it & 1}.{h}", it), wait(f"full{first}", it * ns // slots),
                      ("read", f"seen{it % 16}.0", it), ("read", f"seen{it % 16}.1", it)]
                if it:
                    e.append(wait("pv_done", it - 1))
                    e += [("read", f"O{n}", it - 1) for n in range(ns) if t]
                e += [("write", f"P{h}", it), ("arrive", "p_ready")]
            it += 1
        for e in soft:
            e += [wait("pv_done", it - 1), *(("read", f"O{n}", it - 1) for n in range(ns)), ("arrive", "o_empty")]
    counts = dict.fromkeys(("p_ready", "o_empty"), 2)
    for i in range(slots):
        counts[f"full{i}"] = 2 * ((2 if i % ns == ns - 1 else 1) + publishes)
    return dict(c0=copy[0], c1=copy[1], scores=scores, values=values, s0=soft[0], s1=soft[1], queries=queries), counts


@pytest.mark.parametrize("tiles", [1, 2, 3, 4])
def test_dq(tiles):
    """1 and 2 key tiles have a pass ahead, more do not."""
    assert explore(*dq_roles(tiles)) > 100


def test_dq_without_the_wait_of_the_pass_ahead():
    """Two steps ahead that do not wait for the issuing thread complete two phases of ds_ready under its eyes."""
    with pytest.raises(Fault):
        explore(*dq_roles(2, waits_ahead=False))
    assert explore(*dq_roles(1, waits_ahead=False)) > 100      # a single one cannot


@pytest.mark.parametrize("steps", [1, 2, 4])
def test_dkv(steps):
    assert explore(*dkv_roles(steps)) > 50


@pytest.mark.parametrize("n0,n1", [(1, 1), (0, 2), (2, 0), (1, 3), (3, 3)])
def test_prefill(n0, n1):
    assert explore(*prefill_roles(n0, n1)) > 20


@pytest.mark.parametrize("segments,shared,ns", [((3,), 1, 1), ((1, 1), 2, 1), ((2,), 1, 2)])
def test_decode(segments, shared, ns):
    assert explore(*decode_roles(segments, shared, slots=2 * ns, ns=ns)) > 100


def test_decode_whose_masks_nobody_publishes():
    with pytest.raises(Fault, match="seen"):
        explore(*decode_roles((1,), 1, publishes=False))
