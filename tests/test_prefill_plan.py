"""The model of prompt attention's work plan (test_prefill_schedule) against the code: its constants against the headers', and on a
GPU its items, rounds, cuts and joins against those that the planning kernels leave in the workspace."""
import os
import random
import re

import pytest
import torch

import prefill_ref as ref
import test_prefill_schedule as sched

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gqa_decode_attention_gb300", "csrc")


def constant(name):
    for f in ("gqa_prefill.h", "gqa_prefill_plan.cuh", "gqa_prefill_kernel.cuh", "gqa_prefill_load.cuh"):
        with open(os.path.join(CSRC, f)) as src:
            m = re.search(r"constexpr int [^;]*\b%s = (\d+)" % name, src.read())
        if m:
            return int(m[1])
    raise AssertionError(f"no constant {name}")


def test_model_has_the_headers_constants():
    assert constant("kPreKeys") == sched.KEYS
    assert constant("kPreMinSplit") == sched.MIN_SPLIT
    assert constant("kPreSnap") == sched.SNAP
    assert constant("kPlanBuckets") == sched.BUCKETS
    assert constant("kPlanExactRounds") == sched.EXACT_ROUNDS
    assert constant("kPreCostTwo") == sched.COST_TWO
    assert constant("kPreCostOne") == sched.COST_ONE
    assert constant("kPreCostItem") == sched.COST_ITEM


def test_roles_model_has_the_headers_constants():
    import test_prefill_roles as roles
    assert constant("kPrePieces") == roles.RING


class Workspace:
    """What the planning kernel leaves in a call's workspace, by the layout that the call's launch gives it."""

    def __init__(self, ws, T, B, Hkv, G, W):
        blocks = -(-G // 128)
        g_tile = -(-G // blocks)
        self.tok_tile, self.HB = 128 // g_tile, Hkv * blocks
        room = T // (2 * self.tok_tile) + B
        self.at, self.ws = 0, ws.cpu()
        plan = self.take(4, 1)[0]
        items = self.take(8, room)
        self.take(8, room), self.take(1, B + 1), self.take(2, room + 1)
        joins, cuts = self.take(4, W), self.take(2, W + 1)
        self.n_items, self.rounds, self.total, n_joins = plan.tolist()
        self.items = [dict(zip(("q_row", "n_tok", "req", "steps", "limit0", "L", "k_row", "cost"), x)) for x in items[:self.n_items].tolist()]
        self.joins, self.cuts = [tuple(x[:3]) for x in joins[:n_joins].tolist()], [tuple(x) for x in cuts.tolist()]

    def take(self, words, n):
        x = self.ws[self.at:self.at + 4 * words * n].view(torch.int32).view(n, words)
        self.at += -(-4 * words * n // 256) * 256
        return x


def joins_of(cuts, W):
    """Items that several workers hold steps of, the worker with the beginning and the one with the end."""
    out = []
    for w in range(1, W):
        n, step = cuts[w]
        if step == 0 or (cuts[w - 1][0] == n and cuts[w - 1][1] > 0):
            continue
        last = w
        while last + 1 < W and cuts[last + 1][0] == n:
            last += 1
        out.append((n, w - 1, last))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(24))
def test_kernels_plan_is_the_models(seed):
    from gqa_decode_attention_gb300 import build as gbuild
    gbuild.build()
    import gqa_decode_attention_gb300 as gq
    W = torch.cuda.get_device_properties(0).multi_processor_count
    r = random.Random(seed)
    B = [3, 150, 400, 600][seed % 4]  # one thread a sequence in 256 and 512 of them, and through the workspace
    Hkv, G = r.choice([(1, 8), (8, 8), (4, 1), (2, 5), (3, 12), (1, 160)])
    most = r.choice([40, 700, 5000, 60000])
    n = [r.randint(0, r.choice([1, 8, 90] if B > 100 else [8, 600, 3000])) for _ in range(B)]
    n[-1] = max(n[-1], 1)
    L = [0 if r.random() < 0.2 else max(0, x + r.randint(-5, most)) for x in n]
    causal = r.random() < 0.7
    ps = 16
    ppr = -(-max(max(L), 1) // ps)
    T, D = sum(n), 64
    q = torch.zeros(T, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(1, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, ppr, dtype=torch.int32, device="cuda")
    ws = torch.full((gq.gqa_prefill_paged_workspace_bytes(T, B, Hkv * G, Hkv, D),), 255, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0] + n).cumsum(0).int().cuda()
    gq.gqa_prefill_paged(q, pool, pool, table, torch.tensor(L, dtype=torch.int32).cuda(), cu, causal=causal, workspace=ws)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
    may_split = -(-ppr * ps // sched.KEYS) >= sched.MIN_SPLIT + sched.SNAP
    x = Workspace(ws, T, B, Hkv, G, W)
    if not may_split and (T // (2 * x.tok_tile) + B) * x.HB <= W:
        assert (ws[:16] == 255).all()  # each CTA finds its item itself
        return
    items, top = sched.items_of(n, L, x.tok_tile, causal)
    rounds, cuts, _ = sched.plan(items, top, x.HB, W, may_split)
    assert x.n_items == len(items) and x.total == len(items) * x.HB and x.rounds == rounds
    starts = cu.tolist()
    for got, want in zip(x.items, items):
        first = want["tile"] * 2 * x.tok_tile
        b = want["req"]
        assert got["req"] == b and got["q_row"] == starts[b] + first and got["n_tok"] == min(2 * x.tok_tile, n[b] - first)
        assert got["steps"] == want["steps"] and got["cost"] == want["cost"] and got["L"] == L[b]
        assert got["limit0"] == (L[b] - n[b] + first + 1 if causal else L[b])
    assert x.cuts == cuts
    assert x.joins == (joins_of(cuts, W) if may_split else [])
