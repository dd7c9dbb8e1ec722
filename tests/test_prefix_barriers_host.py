"""The barriers of the attention's prefix kernel, explored on the CPU.

The kernel's loaders, issuing warps and softmax warps meet at mbarriers and wait by parity: a
wait for phase k passes while the barrier has completed an odd (k even) or even (k odd)
number of phases.  It is sound if it can neither pass before phase k has completed nor miss
it, however long any warp, copy or product is held up.  This walks through every order of
events of a model with the kernel's ring: no wait may pass early, and every order has to
come to its end.  The second stream's start is read from the kernel's source, the ring's
order of use is asserted to be the source's.

In the model a stream's four softmax warps are one, and copies into one stage of the ring, or
products of one issuing warp, complete in their order."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_plane_select_gb300", "csrc",
                   "trit_attn_prefix.cu")
RING = 4


def source():
    with open(SRC) as f:
        return f.read()


def start_waits(text, n):
    """[(barrier, phase's parity)] that the second stream's issuing warp waits for before its first product."""
    body = re.search(r"if \(s == 1\)\s*(\{.*?\n        \}|[^\n]*;)", text, re.S).group(1)
    out = []
    for line in body.splitlines():
        for bar, parity in re.findall(r"warp_wait\(&?(\w+(?:\[\d+\])?), (\d)", line):
            if "n >= 8" not in line or n >= 8:
                out.append((re.sub(r"\[(\d+)\]", r"\1", bar), int(parity)))
    return out


def k_at(pair, j):
    return 2 * j if pair else (0 if j == 0 else 2 * j - 1)


def v_at(pair, j):
    return 2 * j + 1 if pair else 2 * j + 2


def programs(pair, n, start):
    """Per agent a list of steps ("wait", barrier, phase), ("arrive", barrier) and ("later", queue, barrier): an
    arrival that a copy or product makes when it completes."""
    go = (1, 0) if n >= 8 else (0, 3)        # block and quarter of the first stream that lets the second start
    progs = {"K": [], "V": [], "I0": [], "I1": [], "S0": [], "S1": []}
    for name, place in (("K", k_at), ("V", v_at)):
        for j in range(n):
            at = place(pair, j)
            progs[name] += [("wait", f"empty{at % RING}", at // RING - 1), ("later", f"{name}{at % RING}", f"full{at % RING}")]
    for s in (0, 1):
        mine = n if pair else (n + 1 - s) // 2
        block = (lambda i: i) if pair else (lambda i: 2 * i + s)
        p = progs[f"I{s}"]

        def issue(i):
            at = k_at(pair, block(i))
            return [("later", f"P{s}", f"s_full{s}"), ("later", f"P{s}", f"empty{at % RING}")]

        def there(i):
            at = k_at(pair, block(i))
            return ("wait", f"full{at % RING}", at // RING)
        if s == 1:
            p += [("wait", bar, parity) for bar, parity in start]
        if mine:
            p += [there(0)] + issue(0)
        for i in range(mine):
            at = v_at(pair, block(i))
            p.append(("wait", f"full{at % RING}", at // RING))
            for part in range(4):
                p.append(("wait", f"p_full{4 * s + part}", i))
                if s == 0 and (i, part) == go:
                    p.append(("arrive", "go"))
            p += [("later", f"P{s}", f"o_full{s}" if i + 1 == mine else f"pv_done{s}"),
                  ("later", f"P{s}", f"empty{at % RING}")]
            if i + 1 < mine:
                p += [there(i + 1), ("wait", f"pv_done{s}", i)] + issue(i + 1)
            progs[f"S{s}"].append(("wait", f"s_full{s}", i))
            progs[f"S{s}"] += [("arrive", f"p_full{4 * s + part}") for part in range(4)]
        if mine:
            progs[f"S{s}"].append(("wait", f"o_full{s}", 0))
    return progs


def explore(pair, n, start, most=2000000):
    """None, or what goes wrong in some order of events."""
    progs = programs(pair, n, start)
    names = list(progs)
    queues = sorted({s[1] for a in names for s in progs[a] if s[0] == "later"})
    # arrivals at a barrier follow from how far every agent and queue has come
    per_queue = {q: [s[2] for a in names for s in progs[a] if s[0] == "later" and s[1] == q] for q in queues}
    owner = {q: {"P0": "I0", "P1": "I1"}.get(q, q[0]) for q in queues}
    pushed = {q: [sum(1 for s in progs[owner[q]][:i] if s[0] == "later" and s[1] == q)
                  for i in range(len(progs[owner[q]]) + 1)] for q in queues}
    bars = sorted({s[1] for a in names for s in progs[a] if s[0] != "later"} | {b for q in queues for b in per_queue[q]})
    counts = {b: 2 if pair and b.startswith("empty") else 1 for b in bars}
    by_agent = {(a, b): [sum(1 for s in progs[a][:i] if s[0] == "arrive" and s[1] == b) for i in range(len(progs[a]) + 1)]
                for a in names for b in bars if any(s[0] == "arrive" and s[1] == b for s in progs[a])}
    by_queue = {(q, b): [per_queue[q][:i].count(b) for i in range(len(per_queue[q]) + 1)]
                for q in queues for b in bars if b in per_queue[q]}
    reach = {b: ([(names.index(a), t) for (a, x), t in by_agent.items() if x == b],
                 [(len(names) + queues.index(q), t) for (q, x), t in by_queue.items() if x == b]) for b in bars}

    def done(state, b):
        return sum(t[state[i]] for part in reach[b] for i, t in part) // counts[b]
    first = (0,) * (len(names) + len(queues))
    seen, stack = {first}, [first]
    while stack:
        state = stack.pop()
        moves = []
        for i, a in enumerate(names):
            if state[i] == len(progs[a]):
                continue
            step = progs[a][state[i]]
            if step[0] == "wait":
                have = done(state, step[1])
                if have & 1 == step[2] & 1:
                    continue                      # parity: not passed
                if have <= step[2]:
                    return f"{a} passes {step[1]} phase {step[2]} early"
            moves.append(state[:i] + (state[i] + 1,) + state[i + 1:])
        for k, q in enumerate(queues):
            i = len(names) + k
            if state[i] < pushed[q][state[names.index(owner[q])]]:
                moves.append(state[:i] + (state[i] + 1,) + state[i + 1:])
        if not moves and any(state[i] < len(progs[a]) for i, a in enumerate(names)):
            return "stuck at " + ", ".join(f"{a}: {progs[a][state[i]]}" for i, a in enumerate(names)
                                           if state[i] < len(progs[a]))
        for m in moves:
            if m not in seen:
                seen.add(m)
                stack.append(m)
        assert len(seen) < most
    return None


def test_the_model_is_the_source_s_ring():
    text = source()
    assert "constexpr int kRing = 4;" in text
    assert "return pair ? 2 * j : (j == 0 ? 0 : 2 * j - 1);" in text
    assert "return pair ? 2 * j + 1 : 2 * j + 2;" in text
    assert start_waits(text, 8)


@pytest.mark.parametrize("pair,n", [(p, n) for p in (True, False) for n in (1, 2, 3, 4, 8)])
def test_no_order_of_events_is_stuck_or_early(pair, n):
    assert explore(pair, n, start_waits(source(), n)) is None


def test_a_start_by_a_barrier_that_goes_on_is_found():
    """The exploration sees a missed phase: a second stream that waits for the first one's
    quarters, which complete again without it."""
    for pair in (True, False):
        assert "p_full3" in explore(pair, 4, [("p_full3", 0)])
    assert "early" in explore(False, 4, [])      # K0 and V1 share a stage: no start before K0 is there
