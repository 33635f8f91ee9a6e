"""The prompt attention's work plan, modelled on the CPU with the kernel's formulas: every step of every item is taken by
exactly one worker, parts are numbered and joined as the merge expects, and shares are even."""
import random

import pytest

KEYS, MIN_SPLIT, SNAP, BUCKETS, EXACT_ROUNDS = 128, 6, 3, 64, 64
COST_TWO, COST_ONE, COST_ITEM = 4, 3, 12


def items_of(n, L, tok_tile, causal):
    out = []
    tpi = 2 * tok_tile
    for b, (nb, lb) in enumerate(zip(n, L)):
        for tile in range(-(-nb // tpi)):
            tok = min(tpi, nb - tile * tpi)
            limit0 = lb - nb + tile * tpi + 1 if causal else lb
            seen = min(max(limit0 + tok - 1, 0), lb) if causal else lb
            steps = -(-seen // KEYS)
            out.append(dict(req=b, tile=tile, steps=steps, two=tok > tok_tile,
                            cost=COST_ITEM + steps * (COST_TWO if tok > tok_tile else COST_ONE)))
    top = max([1] + [i["cost"] for i in out])
    return sorted(out, key=lambda i: BUCKETS - 1 - i["cost"] * (BUCKETS - 1) // top), top


def plan(items, top, HB, W, may_split):
    total = len(items) * HB
    prefix = [0]
    for i in items:
        prefix.append(prefix[-1] + i["cost"])
    small = min(top, COST_ITEM + MIN_SPLIT * COST_TWO)
    goal = max(-(-prefix[-1] * HB // W), small)
    number = lambda r, w: r * W + (W - 1 - w if r & 1 else w)  # noqa: E731
    cost = lambda k: items[k // HB]["cost"]  # noqa: E731
    exact = total // W <= EXACT_ROUNDS
    if exact:
        rounds = total // W
        for w in range(W):
            load = 0
            for r in range(rounds):
                load += cost(number(r, w))
                if load > goal:
                    rounds = r
                    break
    else:
        rounds, load = 0, 0
        while (rounds + 2) * W <= total:
            load += cost(rounds * W) + cost((rounds + 2) * W - 1)
            if load > goal:
                break
            rounds += 2
    n0 = rounds * W
    line = prefix[n0 // HB] * HB + n0 % HB * items[n0 // HB]["cost"] if n0 < total else prefix[-1] * HB
    need = []
    for w in range(W):
        load = sum(cost(number(r, w)) for r in range(rounds)) if exact else line // W
        need.append(max(goal - load, small))
    n0, cuts, x = rounds * W, [], 0
    for w in range(W):
        cut = (total, 0)
        if w == 0:
            cut = (n0, 0)
        elif n0 < total:
            pos = line + x
            if pos < prefix[-1] * HB:
                lo = max(i for i in range(len(items)) if prefix[i] * HB <= pos)
                it = items[lo]
                head, y = divmod(pos - prefix[lo] * HB, it["cost"])
                step = max(0, y - COST_ITEM) // (COST_TWO if it["two"] else COST_ONE)
                if not may_split:
                    step = it["steps"] if 2 * y >= it["cost"] else 0
                if it["steps"] - step < SNAP and 2 * y >= it["cost"]:
                    cut = (lo * HB + head + 1, 0)
                else:
                    cut = (lo * HB + head, step if step >= SNAP and it["steps"] - step >= SNAP else 0)
        cuts.append(cut)
        x += need[w]
    return rounds, cuts + [(total, 0)], goal


def pieces(items, HB, W, rounds, cuts, w):
    got = [(r * W + (W - 1 - w if r & 1 else w), None) for r in range(rounds)]
    got = [(n, 0, items[n // HB]["steps"], -1) for n, _ in got]
    n, s0 = cuts[w]
    end = cuts[w + 1]
    while not (n > end[0] or (n == end[0] and s0 >= end[1])):
        steps = items[n // HB]["steps"]
        s1 = end[1] if n == end[0] else steps
        got.append((n, s0, s1, 2 * w if s0 > 0 else 2 * w + 1 if s1 < steps else -1))
        n, s0 = n + 1, 0
    return got


@pytest.mark.parametrize("seed", range(200))
def test_plan_covers_every_step_once(seed):
    r = random.Random(seed)
    W = r.choice([1, 2, 7, 152])
    HB = r.choice([1, 2, 8])
    B = r.choice([1, 3, 40, 200])
    most = r.choice([1, 40, 700, 5000])
    n = [r.randint(0, r.choice([1, 8, 300, 2000])) for _ in range(B)]
    L = [max(0, x + r.randint(-5, most)) for x in n]
    items, top = items_of(n, L, r.choice([1, 16, 25, 128]), r.random() < 0.7)
    may_split = max(L) > (MIN_SPLIT + SNAP - 1) * KEYS
    rounds, cuts, goal = plan(items, top, HB, W, may_split)
    assert all(a <= b for a, b in zip(cuts, cuts[1:]))
    taken, slots, loads = {}, {}, []
    for w in range(W):
        load = 0
        for k, s0, s1, slot in pieces(items, HB, W, rounds, cuts, w):
            it = items[k // HB]
            taken.setdefault(k, []).append((s0, s1))
            load += COST_ITEM + (s1 - s0) * (COST_TWO if it["two"] else COST_ONE)
            assert (slot < 0) == (s0 == 0 and s1 == it["steps"])
            assert s1 > s0 or it["steps"] == 0
            if slot >= 0:
                assert may_split and slot not in slots
                slots[slot] = k
        loads.append(load)
    assert sorted(taken) == list(range(len(items) * HB))
    for k, parts in taken.items():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == items[k // HB]["steps"]
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
    joined = set()  # as the merge kernel finds them
    for w in range(1, W):
        n_, step = cuts[w]
        if step == 0 or (cuts[w - 1][0] == n_ and cuts[w - 1][1] > 0):
            continue
        last = w
        while last + 1 < W and cuts[last + 1][0] == n_ and cuts[last + 1][1] > 0:
            last += 1
        for x in range(w - 1, last + 1):
            slot = 2 * x + 1 if x == w - 1 else 2 * x
            assert slots[slot] == n_  # no share without steps among them
            joined.add(slot)
    assert joined == set(slots)
    if may_split and items:
        slack = 2 * COST_ITEM + 2 * SNAP * COST_TWO + min(top, COST_ITEM + MIN_SPLIT * COST_TWO)
        assert max(loads) <= goal + slack + (0 if len(items) * HB // W <= EXACT_ROUNDS else 2 * top)
