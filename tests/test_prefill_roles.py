"""The roles of prompt attention's CTA, modelled on the CPU: what each waits for and hands on, over the pieces that the plan
gives a worker, with bf16 pools whose pages go through registers (the loader hands a step's copies on when later ones are under
way, or before it waits).  A CTA stalls when every role waits for another.  And the copies of codes by the loader of coded pools,
whose order only waits give."""
import random

import pytest

import test_prefill_schedule as sched

RING, K_STAGES, V_STAGES = 4, 3, 2  # pieces known ahead, stages at d 128


class Cta:
    """Barriers as counts of what has happened so far."""

    def __init__(self, pieces, hands_on):
        self.pieces = pieces  # (steps, two tiles)
        self.hands_on = hands_on  # the loader hands on before it waits for a piece that is not there yet
        self.published = 0
        self.released = [0] * (len(pieces) + 1)  # roles that are done with a piece
        self.q_loaded = self.q_free = 0  # pieces with steps: rows there, last scores done
        self.k_full = self.k_free = self.v_full = self.v_free = 0  # steps
        self.scores, self.weights, self.outputs = [0, 0], [0, 0], [0, 0]
        self.stat_full = self.stat_free = 0

    def planner(self):
        some = 0
        for n in range(len(self.pieces) + 1):  # the last one says that there are no more
            yield lambda: n < RING or self.released[n - RING] == 4
            self.published = n + 1
            if n < len(self.pieces) and self.pieces[n][0]:
                yield lambda: self.q_free >= some
                some += 1
                self.q_loaded += 1

    def loader(self):
        held = []  # copies under way, oldest first

        def hand_on(keep):
            while len(held) > keep:
                if held.pop(0):
                    self.v_full += 1
                else:
                    self.k_full += 1

        at = 0
        for n in range(len(self.pieces) + 1):
            if self.hands_on and self.published <= n:
                hand_on(0)
            yield lambda: self.published > n
            if n == len(self.pieces):
                break
            self.released[n] += 1
            for _ in range(self.pieces[n][0]):
                for v, stages in ((False, K_STAGES), (True, V_STAGES)):
                    free = (lambda: at < stages + self.v_free) if v else (lambda: at < stages + self.k_free)
                    if not free():
                        hand_on(0)
                        yield free
                    held.append(v)
                    hand_on(1)
                at += 1
        hand_on(0)

    def issuer(self):
        q = k = v = 0
        done = [0, 0]  # units of either row group whose weights were used
        for n in range(len(self.pieces) + 1):
            yield lambda: self.published > n
            if n == len(self.pieces):
                return
            self.released[n] += 1
            steps, two = self.pieces[n]
            units = steps * (2 if two else 1)
            if not units:
                continue
            q += 1
            yield lambda: self.q_loaded >= q

            def scores(u):
                nonlocal k
                if not two or u % 2 == 0:
                    yield lambda: self.k_full > k
                self.scores[u % 2] += 1
                if not two or u % 2:
                    k += 1
                    self.k_free += 1
                if u == units - 1:
                    self.q_free += 1

            for u in range(min(2, units)):
                yield from scores(u)
            for u in range(units):
                t = u % 2
                if not two or t == 0:
                    yield lambda: self.v_full > v
                done[t] += 1
                yield lambda: self.weights[t] >= done[t]
                if not two or t:
                    v += 1
                    self.v_free += 1
                if u + 2 >= units:
                    self.outputs[t] += 1
                else:
                    yield from scores(u + 2)

    def softmax(self, t):
        seen = outs = joins = 0
        for n in range(len(self.pieces) + 1):
            yield lambda: self.published > n
            if n == len(self.pieces):
                return
            steps, two = self.pieces[n]
            units = steps if two else (steps + 1 - t) // 2
            for _ in range(units):
                seen += 1
                yield lambda: self.scores[t] >= seen
                self.weights[t] += 1
            if units:
                outs += 1
                yield lambda: self.outputs[t] >= outs
            if not two and steps > 1:
                joins += 1
                if t == 0:
                    yield lambda: self.stat_full >= joins
                    self.stat_free += 1
                else:
                    self.stat_full += 1
                    yield lambda: self.stat_free >= joins
            self.released[n] += 1


def ends(pieces, hands_on, seed=0):
    """Whether every role comes to its end, whoever runs first."""
    c = Cta(pieces, hands_on)
    r = random.Random(seed)
    roles = [[x, lambda: True] for x in (c.planner(), c.loader(), c.issuer(), c.softmax(0), c.softmax(1))]
    while roles:
        able = [x for x in roles if x[1]()]
        if not able:
            return False
        x = r.choice(able)
        try:
            x[1] = next(x[0])
        except StopIteration:
            roles.remove(x)
    return True


def works(n, L, causal, tok_tile=16, HB=8, W=152):
    """Every worker's pieces, as (steps, two tiles)."""
    items, top = sched.items_of(n, L, tok_tile, causal)
    rounds, cuts, _ = sched.plan(items, top, HB, W, max(L) > (sched.MIN_SPLIT + sched.SNAP - 1) * sched.KEYS)
    out = []
    for w in range(W):
        p = sched.pieces(items, HB, W, rounds, cuts, w)
        out.append([(s1 - s0, items[k // HB]["two"]) for k, s0, s1, _ in p])
    return out


# batches in which some requests see no key: no cached prefix, padded slots, more new rows than keys
BATCHES = [
    ([512] * 48, [0] * 32 + [640] * 16, False),
    ([1] * 64, [1000] * 32 + [0] * 32, True),
    ([1] * 128, [20000] * 64 + [0] * 64, True),
    ([1] * 256, [1000] * 20 + [0] * 236, True),
    ([1] * 128, [500] * 40 + [0] * 88, True),
    ([5000], [10], True),
]


@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_no_worker_stalls(batch):
    for seed, w in enumerate(works(*BATCHES[batch])):
        assert ends(w, True, seed), w


@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_model_sees_what_is_held_back(batch):
    """A loader that holds the last step of a piece back while it waits for the next one stalls on these batches."""
    assert not all(ends(w, False, seed) for seed, w in enumerate(works(*BATCHES[batch])))


@pytest.mark.parametrize("seed", range(200))
def test_no_list_stalls(seed):
    r = random.Random(seed)
    some = r.choice([0.1, 0.3, 0.7, 1.0])
    pieces = [(r.choice([1, 2, 3, 9]) if r.random() < some else 0, r.random() < 0.5) for _ in range(r.randint(0, 40))]
    for run in range(5):
        assert ends(pieces, True, run)


@pytest.mark.parametrize("seed", range(30))
def test_no_planned_list_stalls(seed):
    r = random.Random(seed)
    B = r.choice([1, 40, 200])
    n = [r.randint(0, r.choice([1, 8, 300])) for _ in range(B)]
    L = [0 if r.random() < 0.6 else max(0, x + r.randint(-5, 2000)) for x in n]
    for s, w in enumerate(works(n, L, r.random() < 0.5, r.choice([1, 16, 25, 128]), r.choice([1, 8]), r.choice([2, 7, 152]))):
        assert ends(w, True, s)


def copies(pieces, zeros_behind):
    """A thread's asynchronous copies into its places of K and of V, its waits ("all groups but the newest n are there") and its
    reads, over pieces of so many steps.  zeros_behind: something is copied behind a piece's last step too."""
    for steps in pieces:
        if not steps:
            continue
        yield from (("copy", "K"), ("commit",), ("copy", "V"), ("commit",))
        for step in range(steps):
            for place in "KV":
                yield ("wait", 1)
                yield ("read", place)
                if step + 1 < steps or zeros_behind:
                    yield ("copy", place)
                yield ("commit",)


def in_order(events):
    """No copy to a place that an older one may still reach, no read of a place that one may."""
    groups, now = [], []
    for e in events:
        if e[0] == "copy":
            if any(e[1] in g for g in groups + [now]):
                return False
            now.append(e[1])
        elif e[0] == "commit":
            groups.append(now)
            now = []
        elif e[0] == "wait":
            del groups[:max(0, len(groups) - e[1])]
        elif any(e[1] in g for g in groups + [now]):
            return False
    return True


@pytest.mark.parametrize("pieces", [[1], [1, 1], [3, 1, 2], [0, 2, 0, 0, 5, 1, 1], [9, 9]])
def test_copies_of_codes_are_ordered(pieces):
    assert in_order(copies(pieces, False))
    # the model sees zeros copied behind a piece, beside the next piece's codes
    assert in_order(copies(pieces, True)) == (sum(x > 0 for x in pieces) < 2)
