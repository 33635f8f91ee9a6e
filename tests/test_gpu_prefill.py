"""GPU parity of prompt attention (packed, and over the paged cache) and of the merge of attentions over parts, through
the Python binding, against a plain 64-bit computation."""
import math

import pytest
import torch

import cache_ref as cref
import prefill_ref as ref

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp8", "int8", "int4"]


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_gb300 import build as gbuild
    gbuild.build()
    import gqa_decode_attention_gb300 as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def run(gq, d, causal=True, **kw):
    out, lse = ref.call(gq, d, causal, **kw)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
    return out, lse


# ------------------------------------------------------------------------------------------------ packed prompts
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,Hq,Hkv,D,Dv", [
    ([1], 8, 2, 64, 64),
    ([17], 8, 2, 64, 64),
    ([1], 1, 1, 128, 128),
    ([128], 8, 1, 128, 128),
    ([129, 1, 0, 31, 256], 4, 4, 128, 128),      # one row a KV head: items of 256 tokens
    ([300, 127, 2, 513], 8, 8, 64, 64),
    ([40, 77, 16, 33], 64, 8, 128, 128),
    ([200, 5], 12, 4, 128, 128),                 # groups that leave rows of a tile empty
    ([61, 140], 5, 1, 64, 64),
    ([50, 3], 14, 2, 128, 128),
    ([9, 30], 32, 1, 128, 128),
    ([7, 2, 1], 128, 1, 128, 128),
    ([5, 3], 160, 1, 64, 64),                    # more query heads a KV head than a tile has rows
    ([33, 260], 16, 4, 192, 128),
    ([700], 24, 8, 192, 128),
    ([1000, 400], 16, 2, 128, 128),
])
def test_prompts(gq, n, Hq, Hkv, D, Dv, causal):
    d = ref.make(n, n, Hq, Hkv, D, seed=sum(n) + D + Hq, Dv=Dv, fused=D == Dv)
    ref.check(d, *run(gq, d, causal), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,L,Hq,Hkv,D", [
    ([5, 3, 8, 0, 4], [7, 2, 0, 9, 4], 8, 2, 128),             # rows that see no key, sequences without keys or rows
    ([300, 10], [20, 11], 8, 8, 64),                           # most rows of a tile see nothing
    ([260, 1, 64], [1000, 4097, 640], 32, 8, 128),
    ([1], [20000], 8, 1, 128),                                 # one row over a long axis
    ([3, 1, 2], [9000, 129, 30011], 16, 2, 64),
    ([37], [12345], 4, 1, 128),
])
def test_keys_of_their_own(gq, n, L, Hq, Hkv, D, causal):
    d = ref.make(n, L, Hq, Hkv, D, seed=sum(n) + sum(L))
    ref.check(d, *run(gq, d, causal), causal)


def test_many_sequences(gq):
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 90, (333,), generator=g).tolist()
    d = ref.make(n, n, 8, 2, 64, seed=4, fused=True)
    ref.check(d, *run(gq, d))


def test_long_prompt(gq):
    d = ref.make([4321], [4321], 16, 2, 128, seed=5, fused=True)
    ref.check(d, *run(gq, d))


def test_uniform_without_offsets(gq):
    d = ref.make([70] * 3, [70] * 3, 8, 4, 64, seed=6, pad=0)
    lib, q, k, v = gq.load_library(), d["q"], d["k"], d["v"]
    out, lse = torch.empty_like(q), torch.empty(210, 8, device="cuda")
    st = lib.gqa_prefill(q.data_ptr(), 512, k.data_ptr(), 256, v.data_ptr(), 256, None, None, out.data_ptr(), lse.data_ptr(), 210, 210, 3,
                         8, 4, 64, 64, 1, 0.0, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    ref.check(d, out, lse)
    out, lse = gq.gqa_prefill(q[:70], k[:70], v[:70])  # one sequence
    one = dict(d, n=[70], L=[70])
    ref.check(one, out, lse)


def test_scale_and_large_scores(gq):
    """Scores far past exp's range, and a scale of the caller's."""
    d = ref.make([130, 20], [130, 20], 8, 2, 128, seed=7, gain=300.0)
    ref.check(d, *run(gq, d, scale=0.37), scale=0.37)
    d = ref.make([130, 20], [130, 20], 8, 2, 128, seed=8, kind="fp8", gain=3000.0)
    ref.check(d, *run(gq, d))


def test_growing_scores(gq):
    """Each key's score far above the one before it: the running maximum moves at every key, for every row."""
    d = ref.make([600], [600], 4, 2, 64, seed=9)
    d["k"][:600] = (torch.arange(600, device="cuda") * 0.25)[:, None, None].to(torch.bfloat16)
    d["q"][:600] = 1.0
    d["kv"] = [(d["k"][:600].double(), d["v"][:600].double())]
    ref.check(d, *run(gq, d))
    d["k"][:600] = d["k"][:600].flip(0)
    d["kv"] = [(d["k"][:600].double(), d["v"][:600].double())]
    ref.check(d, *run(gq, d))


# ------------------------------------------------------------------------------------------------ over the paged cache
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,L,Hq,Hkv,D,ps", [
    ([5], [1000], 8, 2, 64, 5),
    ([1, 1, 1], [1, 300, 17], 8, 2, 128, 16),                  # decode steps
    ([1, 200, 8, 0, 1], [333, 200, 130, 40, 128], 64, 8, 128, 16),
    ([33, 129], [129, 1290], 16, 4, 64, 7),
    ([100, 64], [100, 512], 5, 5, 128, 1),
    ([20, 300], [900, 300], 12, 4, 64, 24),
    ([64, 3], [2000, 700], 32, 8, 128, 64),
    ([17, 140], [400, 777], 7, 1, 128, 128),
    ([12], [260], 8, 4, 64, 300),                              # pages longer than a tile, of an odd size
    ([2, 9], [5, 3], 8, 2, 128, 8),                            # rows that see no key
    ([6, 1], [9000, 20011], 16, 2, 64, 32),                    # few rows over a long axis
    ([4], [30], 160, 1, 128, 16),
])
def test_chunks(gq, kind, n, L, Hq, Hkv, D, ps):
    d = ref.make(n, L, Hq, Hkv, D, seed=sum(L) + ps, kind=kind, ps=ps)
    ref.check(d, *run(gq, d))
    ref.check(d, *run(gq, d, causal=False), causal=False)


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_device_scales(gq, kind):
    """A scale a KV head, read on the device; negative ones and zero among them."""
    d = ref.make([9, 40], [200, 40], 16, 4, 128, seed=11, kind=kind)
    ks, vs = torch.tensor([0.01, -0.02, 0.0, 0.03]).cuda(), torch.tensor([0.05, 0.01, -0.02, 0.0]).cuda()
    d["kv"] = [(k / d["scale"] * ks[:, None].double(), v / d["scale"] * vs[:, None].double()) for k, v in d["kv"]]
    ref.check(d, *run(gq, d, k_scales=ks, v_scales=vs))
    one = ref.make([9, 40], [200, 40], 16, 4, 128, seed=11, kind=kind)
    a = run(gq, one)
    b = run(gq, one, k_scales=torch.tensor([one["scale"]]).cuda(), v_scales=torch.tensor([one["scale"]]).cuda())
    assert torch.equal(a[0], b[0]) and (a[1] - b[1]).abs().max() < 1e-5


def test_paged_is_packed(gq):
    """A bf16 cache gives what the same keys packed give, bit for bit, whatever the pages."""
    for ps in (16, 7, 128):
        d = ref.make([50, 3, 200], [300, 3, 201], 16, 4, 128, seed=12, kind="bf16", ps=ps)
        a = run(gq, d)
        p = dict(d, kind="dense", k=torch.cat([k for k, _ in d["kv"]]).to(torch.bfloat16),
                 v=torch.cat([v for _, v in d["kv"]]).to(torch.bfloat16), cu_k=torch.tensor([0, 300, 303, 504]).int().cuda())
        b = run(gq, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_lengths(gq, kind):
    d = ref.make([3, 5], [100, 60], 8, 2, 64, seed=13, kind=kind)
    d["table"][0, 2] = 1 << 30  # tokens 32 .. 47 read as zeros
    d["table"][1, 0] = -1       # tokens 0 .. 15
    for (k, v), at in zip(d["kv"], (slice(32, 48), slice(0, 16))):
        k[at], v[at] = 0.0, 0.0
    out, lse = ref.call(gq, d)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 7
    ref.check(d, out, lse)
    d = ref.make([3, 5], [112, 64], 8, 2, 64, seed=14, kind=kind)  # seven pages a request
    d["table"][1] = d["table"][0]  # the second request's length is clamped to them
    d["lens"] = torch.tensor([-5, 1000], dtype=torch.int32).cuda()
    out, lse = ref.call(gq, d)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 7
    d["L"], d["rows"], d["kv"] = [0, 112], [d["rows"][0][:0], d["rows"][0]], [(d["kv"][0][0][:0], d["kv"][0][1][:0]), d["kv"][0]]
    ref.check(d, out, lse)


def test_bad_offsets(gq):
    """Offsets that decrease or leave the tensors are clamped and flagged; nothing outside is touched."""
    d = ref.make([50, 30, 20], [50, 30, 20], 8, 2, 64, seed=15, pad=0)
    for cu in ([0, 50, 40, 100], [-9, 50, 80, 1 << 30], [0, 2 ** 31 - 1, -(2 ** 31), 100], [100, 0, 100, 0], [0, 100, 0, 100]):
        guard = torch.full((300, 8, 64), -7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((300, 8), -7.0, device="cuda")
        gq.gqa_prefill(d["q"], d["k"], d["v"], torch.tensor(cu, dtype=torch.int32).cuda(), out=guard[100:200], lse=lse[100:200])
        torch.cuda.synchronize()
        assert gq.gqa_device_status() == 7
        for t in (guard, lse):
            assert torch.all(t[:100] == -7) and torch.all(t[200:] == -7)
    assert torch.isfinite(guard).all()


def test_bad_offsets_of_many(gq):
    """Thousands of sequences that each claim all rows: far more items than there is room for."""
    d = ref.make([90], [90], 8, 8, 64, seed=59, pad=0)
    cu = torch.tensor([0, 90] * 20000, dtype=torch.int32).cuda()
    guard = torch.full((270, 8, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    gq.gqa_prefill(d["q"], d["k"], d["v"], cu, out=guard[90:180])
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 7
    assert torch.all(guard[:90] == -7) and torch.all(guard[180:] == -7)
    out, lse = run(gq, d)
    ref.check(d, out, lse)


# ------------------------------------------------------------------------------------------------ what is not finite
@pytest.mark.parametrize("kind", ["dense", "bf16", "fp8", "int4"])
def test_keys_not_seen_never_reach_a_row(gq, kind):
    """Later tokens of the same sequence hold NaN and infinities: rows before them stay as they are, and an element of V
    that is not finite reaches that element of the rows that see it."""
    n = L = [150, 20]
    d = ref.make(n, L, 8, 4, 64, seed=16, kind=kind)
    want = run(gq, d)
    bad = 100  # token of sequence 0
    if kind == "dense":
        d["k"][bad, 1] = float("nan")
        d["v"][bad, 2, 5] = float("inf")
        d["v"][bad + 1, 3] = float("nan")
    else:
        at = d["rows"][0][bad:bad + 2]
        kp, vp = d["k_pool"].flatten(0, 1), d["v_pool"].flatten(0, 1)
        if kind == "int4":
            params = d["params"].flatten(0, 1)
            params[at[0], 1, 0] = float("nan")
            params[at[0], 2, 3] = float("inf")
            params[at[1], 3, 2] = float("nan")
        elif kind == "fp8":
            kp[at[0], 1] = 127
            vp[at[0], 2, 5] = 127
            vp[at[1], 3] = 255
        else:
            kp[at[0], 1] = float("nan")
            vp[at[0], 2, 5] = float("inf")
            vp[at[1], 3] = float("nan")
    got = run(gq, d)
    for a, b in zip(want, got):
        assert torch.equal(a[:bad], b[:bad]) and torch.equal(a[150:], b[150:]), "rows that do not see the token"
    o, l = got[0][bad:150], got[1][bad:150]
    assert torch.isnan(l[:, 2:4]).all() and torch.isnan(o[:, 2:4]).all()  # KV head 1: scores of NaN
    assert torch.isfinite(l[:, [0, 1, 4, 5, 6, 7]]).all()
    cols = slice(None) if kind == "int4" else slice(5, 6)
    assert not torch.isfinite(o[:, 4:6, cols]).any()
    if kind != "int4":
        rest = [i for i in range(64) if i != 5]
        assert torch.equal(o[:, 4:6][..., rest], want[0][bad:150, 4:6][..., rest])
    assert not torch.isfinite(o[1:, 6:8]).any() and torch.equal(o[0, 6:8], want[0][bad, 6:8])
    assert torch.equal(o[:, :2], want[0][bad:150, :2])


def test_extreme_queries(gq):
    """A query row of infinities is NaN and no other row is; bf16's largest and smallest values pass."""
    for kind in ("dense", "fp8", "int4"):
        d = ref.make([20], [40], 8, 2, 64, seed=17, kind=kind)
        base = run(gq, d)
        d["q"][3, 5] = float("inf")
        d["q"][4, 1] = 0.0
        out, lse = run(gq, d)
        assert torch.isnan(out[3, 5]).all() and torch.isnan(lse[3, 5])
        keep = torch.ones(20, 8, dtype=torch.bool)
        keep[3, 5] = keep[4, 1] = False
        assert torch.equal(out[:20][keep], base[0][:20][keep])
        d["q"][3, 5] = 0.0
        ref.check(d, *run(gq, d))
        d["q"][:20] *= 2.0 ** -100
        ref.check(d, *run(gq, d))


# ------------------------------------------------------------------------------------------------ calls
@pytest.mark.parametrize("kind", ["dense", "bf16", "int8", "int4"])
def test_workspace_stream_and_repeat(gq, kind):
    d = ref.make([40, 1, 7], [40, 1, 7] if kind == "dense" else [5000, 900, 7], 16, 2, 128, seed=18, kind=kind)
    a = run(gq, d)
    T, B = d["q"].shape[0], 3
    need = gq.gqa_prefill_workspace_bytes(T, B, 16, 2, 128, 128) if kind == "dense" else gq.gqa_prefill_paged_workspace_bytes(T, B, 16, 2, 128)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    b = run(gq, d, workspace=ws)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    c = run(gq, d, workspace=ws, stream=stream)
    e = run(gq, d, out=None, lse=None, stream=stream)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    assert torch.equal(a[0][:48], e[0][:48]) and torch.equal(a[1][:48], e[1][:48])
    assert run(gq, d, out=None, lse=None, with_lse=False)[1] is None
    if need:
        with pytest.raises(gq.GQAError, match="NO_MEMORY"):
            run(gq, d, workspace=ws[:need - 1])
        with pytest.raises(gq.GQAError, match="ALIGNMENT"):
            run(gq, d, workspace=torch.empty(need + 256, dtype=torch.uint8, device="cuda")[8:])


@pytest.mark.parametrize("kind", ["dense", "bf16", "fp8"])
def test_graph(gq, kind):
    """Captured once, replayed on other lengths, offsets and values."""
    n, L = [20, 100, 3], [20, 100, 3] if kind == "dense" else [2000, 100, 700]
    d = ref.make(n, L, 16, 4, 128, seed=19, kind=kind)
    run(gq, d)
    out = torch.zeros(126, 16, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(126, 16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ref.call(gq, d, out=out, lse=lse)
    for n, L in (([20, 100, 3], L), ([0, 60, 63], [0, 60, 63]), ([1, 1, 1], [1, 1, 1])):
        e = ref.make(n, L, 16, 4, 128, seed=20 + n[0], kind=kind, pad=126 - sum(n))
        for name in ("q", "cu", "cu_k", "k", "v", "lens"):
            if name in e and torch.is_tensor(e[name]):
                d[name][:e[name].shape[0]].copy_(e[name])
        if kind != "dense":
            ppr = e["table"].shape[1]
            d["table"].fill_(-1)
            d["table"][:, :ppr].copy_(e["table"])
            d["k_pool"][:e["k_pool"].shape[0]].copy_(e["k_pool"][:d["k_pool"].shape[0]])
            d["v_pool"][:e["v_pool"].shape[0]].copy_(e["v_pool"][:d["v_pool"].shape[0]])
        out.fill_(-7)
        lse.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        ref.check(e, out, lse)
    assert gq.gqa_device_status() == 0


def test_two_calls_at_once(gq):
    """Calls on two streams, each with the library's own workspaces."""
    ds = [ref.make([3, 200], [6000, 2000], 16, 2, 128, seed=30 + i, kind="bf16") for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    got = [[] for _ in ds]
    for _ in range(5):
        for i, d in enumerate(ds):
            got[i].append(ref.call(gq, d, out=None, lse=None, stream=streams[i]))
    torch.cuda.synchronize()
    for d, runs in zip(ds, got):
        for out, lse in runs:
            ref.check(d, out, lse, untouched=False)


# ------------------------------------------------------------------------------------------------ plans and sizes
def test_many_sequences_through_the_workspace(gq):
    """More sequences than the planning CTA holds by itself, and more rounds of items than it adds up one by one; one of
    them long enough to be divided."""
    g = torch.Generator().manual_seed(50)
    n = torch.randint(0, 17, (1200,), generator=g).tolist()
    d = ref.make(n, n, 32, 32, 64, seed=51, fused=True)
    ref.check(d, *run(gq, d))
    n[700] = 3000
    L = list(n)
    L[20] = 9000
    d = ref.make(n, L, 4, 2, 64, seed=52)
    ref.check(d, *run(gq, d))
    d = ref.make(n[:620], L[:620], 4, 2, 64, seed=53, kind="fp8")
    ref.check(d, *run(gq, d))


def test_many_items(gq):
    """More items than the planning CTA has threads: a group of 64 heads leaves four tokens an item."""
    d = ref.make([9001, 3], [9001, 3], 64, 1, 64, seed=54, fused=True)
    out, lse = run(gq, d)
    at = [0, 1, 2, 500, 4000, 8191, 8999, 9000]  # rows checked
    k, v = d["kv"][0]
    for i in at:
        e = dict(n=[1], L=[i + 1], q=d["q"][i:i + 1], kv=[(k[:i + 1], v[:i + 1])], kind="dense", Hq=64, Hkv=1, D=64, Dv=64)
        ref.check(e, out[i:i + 1], lse[i:i + 1], untouched=False, what=f"row {i}")
    ref.check(dict(n=[3], L=[3], q=d["q"][9001:9004], kv=[d["kv"][1]], kind="dense", Hq=64, Hkv=1, D=64, Dv=64), out[9001:], lse[9001:])


@pytest.mark.parametrize("B,n,L", [(1, 3, 40), (19, 5, 300), (37, 1, 1100), (40, 2, 129)])
def test_items_found_without_a_plan(gq, B, n, L):
    """No more items than SMs and keys that are not divided: no plan, no workspace (some sequences are empty)."""
    ns, Ls = [n if b % 5 else 0 for b in range(B)], [max(0, L - 7 * b) if b % 3 else 0 for b in range(B)]
    ns[-1] = n
    for kind in ("dense", "int8"):
        d = ref.make(ns, Ls, 8, 2, 64, seed=55 + B, kind=kind)
        ref.check(d, *run(gq, d))


@pytest.mark.parametrize("kind,ps", [("bf16", 16), ("bf16", 5), ("fp8", 16), ("int4", 16)])
def test_large_pool(gq, kind, ps):
    """Pools whose far end is past 4 GB."""
    Hkv, D, lens = 8, 128, [300, 40]
    row = Hkv * D * {"bf16": 2, "fp8": 1, "int4": 0.5}[kind]
    pages = int((1 << 32) / (row * ps)) + 200
    small = ref.make([20, 3], lens, 16, Hkv, D, seed=56, kind=kind, ps=ps)
    want = run(gq, small)
    big = dict(small)
    for name in ("k_pool", "v_pool", "params"):
        x = small[name]
        if x is not None:
            big[name] = torch.empty(pages, *x.shape[1:], dtype=x.dtype, device="cuda")
            big[name][pages - x.shape[0]:] = x
    used = small["table"] >= 0
    used &= small["table"] < small["k_pool"].shape[0]
    big["table"] = torch.where(used, small["table"] + (pages - small["k_pool"].shape[0]), small["table"])
    got = run(gq, big)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_shared_pages(gq):
    """Two requests whose tables name the same pages."""
    d = ref.make([30, 30], [400, 400], 16, 4, 128, seed=57, kind="bf16")
    d["table"][1] = d["table"][0]
    d["rows"][1] = d["rows"][0]
    d["kv"][1] = d["kv"][0]
    d["q"][30:60] = d["q"][:30]
    out, lse = run(gq, d)
    ref.check(d, out, lse)
    assert torch.equal(out[:30], out[30:60]) and torch.equal(lse[:30], lse[30:60])


@pytest.mark.parametrize("kind,ps", [("dense", 16), ("bf16", 16), ("bf16", 7), ("fp8", 16), ("int4", 16)])
def test_wait_limit(gq, kind, ps):
    """A tile that never comes: the call ends with the error flagged, and the next one is right."""
    d = ref.make([200, 3], [700, 1500], 16, 4, 128, seed=58, kind=kind, ps=ps)
    run(gq, d)
    gq.gqa_set_wait_limit_ns(50_000_000)
    gq.gqa_debug_set_fault_mode(1)
    try:
        ref.call(gq, d)
        assert gq.gqa_device_status() == 6
    finally:
        gq.gqa_debug_set_fault_mode(0)
        gq.gqa_set_wait_limit_ns(0)
    ref.check(d, *run(gq, d))


@pytest.mark.parametrize("kind,ps", [("bf16", 64), ("bf16", 7), ("fp8", 16), ("int4", 16)])
def test_items_longer_than_the_wait_limit(gq, kind, ps):
    """Two whole items an SM of 4096 steps each, some milliseconds, with the least wait limit that can be set."""
    Hq, Hkv, D, pages, L = 8, 1, 64, 90, (1 << 19) + 37
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    d = ref.make([1], [pages * ps], Hq, Hkv, D, seed=59, kind=kind, ps=ps)
    g = torch.Generator(device="cuda").manual_seed(60)
    d["q"] = torch.randn(2 * 32 * sms, Hq, D, device="cuda", generator=g).to(torch.bfloat16)
    d["table"] = d["table"][0][torch.randint(0, pages, (1, -(-L // ps)), device="cuda", generator=g)]
    d["lens"] = torch.tensor([L], dtype=torch.int32, device="cuda")
    d["cu"] = torch.tensor([0, d["q"].shape[0]], dtype=torch.int32, device="cuda")
    want = run(gq, d)
    gq.gqa_set_wait_limit_ns(1)  # raised to 1 ms
    try:
        got = run(gq, d)
    finally:
        gq.gqa_set_wait_limit_ns(0)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("n,L", [([5, 7], [3, 20]), ([1500], [1400])])
def test_device_scale_of_nan(gq, kind, n, L):
    """A K scale of NaN is NaN for rows that see a key; rows that see none are zeros all the same."""
    d = ref.make(n, L, 8, 2, 128, seed=61, kind=kind)
    nan, one = torch.full((1,), math.nan, device="cuda"), torch.ones(1, device="cuda")
    out, lse = ref.call(gq, d, k_scales=nan, v_scales=one)
    assert gq.gqa_device_status() == 0
    at = 0
    for ni, Li in zip(n, L):
        none = max(0, ni - Li)
        assert torch.all(out[at:at + none] == 0) and torch.all(lse[at:at + none] == -math.inf)
        assert torch.all(out[at + none:at + ni].isnan()) and torch.all(lse[at + none:at + ni].isnan())
        at += ni


def test_nothing_to_do(gq):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out, lse = gq.gqa_prefill(z(0, 8, 64), z(5, 2, 64), z(5, 2, 64))
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    out, lse = gq.gqa_prefill(z(4, 8, 64), z(0, 2, 64), z(0, 2, 64))
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = gq.gqa_prefill(z(4, 8, 64), z(4, 2, 64), z(4, 2, 64), cu, out=z(4, 8, 64) + 3)
    assert torch.all(out == 3)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0


# ------------------------------------------------------------------------------------------------ merge
def parts(N, T, H, D, seed, none=0.2):
    g = torch.Generator().manual_seed(seed)
    outs = [torch.randn(T, H, D, generator=g).to(torch.bfloat16).cuda() for _ in range(N)]
    lses = [(torch.randn(T, H, generator=g) * 4 + 100 * i * (T % 2)).cuda() for i in range(N)]
    for o, l in zip(outs, lses):
        gone = (torch.rand(T, H, generator=g) < none).cuda()
        l[gone] = -math.inf
        o[gone] = float("nan")  # must not matter
    return outs, lses


def check_merge(outs, lses, out, lse):
    s = torch.stack(lses).double()
    want_l = torch.logsumexp(s, 0)
    w = torch.where(s == -math.inf, 0.0, torch.exp(s - torch.where(want_l == -math.inf, 0.0, want_l)))[..., None]
    o = torch.stack(outs).double().nan_to_num()
    want, mag = (w * o).sum(0), (w * o.abs()).sum(0)
    # a share: the exponential's argument, its own error and the sum's, the division; then a product and a sum a part
    rel = (s.masked_fill(s == -math.inf, 0.0).abs().amax(0) * 2.0 ** -22 + 40 * 2.0 ** -23)[..., None]
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + rel * mag + 1e-30).all())
    empty = want_l == -math.inf
    assert torch.equal(lse == -math.inf, empty) and torch.all(out[empty] == 0)
    assert bool((torch.where(empty, 0.0, (lse.double() - want_l).abs()) <= rel[..., 0] + 2.0 ** -22 * want_l.abs().nan_to_num(posinf=0.0, neginf=0.0)).all())


@pytest.mark.parametrize("N", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("T,H,D", [(1, 1, 8), (33, 6, 64), (50, 8, 128), (7, 3, 200), (300, 5, 256)])
def test_merge(gq, N, T, H, D):
    outs, lses = parts(N, T, H, D, seed=N * T + D)
    check_merge(outs, lses, *gq.gqa_merge(outs, lses))
    out, lse = outs[-1].clone(), lses[-1].clone()  # in place
    got = gq.gqa_merge(outs[:-1] + [out], lses[:-1] + [lse], out=out, lse=lse)
    check_merge(outs, lses, *got)
    assert got[0].data_ptr() == out.data_ptr()


def test_merge_not_finite(gq):
    outs, lses = parts(2, 5, 4, 64, seed=1, none=0.0)
    lses[0][0, 0] = float("nan")
    lses[1][1, 1] = float("inf")
    outs[0][2, 2, 3] = float("inf")
    out, lse = gq.gqa_merge(outs, lses)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0])
    assert torch.isnan(out[1, 1]).all() and torch.isnan(lse[1, 1])
    bad = ~torch.isfinite(out)
    bad[0, 0] = bad[1, 1] = False
    assert bad.sum() == 1 and bad[2, 2, 3]
    with pytest.raises(gq.GQAError, match="UNSUPPORTED"):
        gq.gqa_merge([torch.zeros(2, 12, dtype=torch.bfloat16, device="cuda")], [torch.zeros(2, device="cuda")])


# ------------------------------------------------------------------------------------------------ used together
@pytest.mark.parametrize("kind", KINDS)
def test_serving_step(gq, kind):
    """Prompts go into the cache in two chunks, each attended as it is appended; the same in one piece over the keys read
    back from the cache; and prefix and own tokens apart, merged."""
    Hq, Hkv, D, ps, lens = 16, 4, 128, 16, [200, 37, 90]
    B, ppr = 3, 16
    scale = 0.04
    kc = {"bf16": torch.bfloat16, "fp8": torch.uint8, "int8": torch.int8, "int4": torch.uint8}[kind]
    pools = [torch.zeros(B * ppr, ps, Hkv, D // 2 if kind == "int4" else D, dtype=kc, device="cuda") for _ in range(2)]
    params = torch.zeros(B * ppr, ps, Hkv, 4, dtype=torch.float16, device="cuda") if kind == "int4" else None
    kw = dict(kv_params=params, k_scale=scale, v_scale=scale)
    g = torch.Generator().manual_seed(40)
    table = torch.randperm(B * ppr, generator=g).view(B, ppr).int().cuda()
    qkv = [torch.randn(n, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda() for n in lens]
    cos_sin = cref.rope_table(256, D).cuda()
    first = [120, 37, 1]
    got_o, got_l, q_rot = [[] for _ in lens], [[] for _ in lens], [[] for _ in lens]
    before = torch.zeros(B, dtype=torch.int32)
    for part in (first, [n - f for n, f in zip(lens, first)]):
        x = torch.cat([qkv[b][int(before[b]):int(before[b]) + m] for b, m in enumerate(part)])
        cu = torch.tensor([0] + part).cumsum(0).int().cuda()
        before = before + torch.tensor(part, dtype=torch.int32)
        seq = before.cuda()
        q = gq.gqa_paged_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *pools, table, seq, cu_tokens=cu, q=x[:, :Hq], cos_sin=cos_sin, **kw)
        out, lse = gq.gqa_prefill_paged(q, *pools, table, seq, cu, **kw)
        for b in range(B):
            got_o[b].append(out[cu[b]:cu[b + 1]])
            got_l[b].append(lse[cu[b]:cu[b + 1]])
            q_rot[b].append(q[cu[b]:cu[b + 1]])
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    d = dict(n=lens, L=lens, kind=kind, q=torch.cat([torch.cat(x) for x in q_rot]), Hq=Hq, Hkv=Hkv, D=D, Dv=D, ps=ps, scale=scale if kind in ("fp8", "int8") else 1.0,
             k_pool=pools[0], v_pool=pools[1], params=params, table=table)
    d["rows"] = [cref.slots(table[b].cpu(), ps, range(n)).cuda() for b, n in enumerate(lens)]
    d["kv"] = [ref.held(d, r) for r in d["rows"]]
    ref.check(d, torch.cat([torch.cat(x) for x in got_o]), torch.cat([torch.cat(x) for x in got_l]), untouched=False, what="chunks")
    # one piece over dense keys, read back
    kd, vd = gq.gqa_paged_gather(*pools, table, seq, rows=200, **kw)
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    k, v = (torch.cat([x[b, :n] for b, n in enumerate(lens)]) for x in (kd, vd))
    one = gq.gqa_prefill(d["q"], k, v, cu)
    e = dict(d, kind="dense", kv=[(k[cu[b]:cu[b + 1]].double(), v[cu[b]:cu[b + 1]].double()) for b in range(B)])
    ref.check(e, *one, untouched=False, what="one piece")
    # the second chunk's rows over the cached prefix and over their own keys, merged
    part = [n - f for n, f in zip(lens, first)]
    cu2 = torch.tensor([0] + part).cumsum(0).int().cuda()
    q2, k2, v2 = (torch.cat([x[int(cu[b]) + f:int(cu[b + 1])] for b, f in enumerate(first)]) for x in (d["q"], k, v))
    prefix = gq.gqa_prefill_paged(q2, *pools, table, torch.tensor(first, dtype=torch.int32).cuda(), cu2, causal=False, **kw)
    own = gq.gqa_prefill(q2, k2, v2, cu2)
    out, lse = gq.gqa_merge([prefix[0], own[0]], [prefix[1], own[1]])
    for b, f in enumerate(first):
        a = slice(int(cu2[b]), int(cu2[b + 1]))
        whole = one[0][int(cu[b]) + f:int(cu[b + 1])].float()
        # two more roundings to bf16 of parts that share the row, and those of a weight on either side; what the keys' bf16
        # and their codes differ by
        assert bool(((out[a].float() - whole).abs() <= 0.05).all()) and bool(((lse[a] - one[1][int(cu[b]) + f:int(cu[b + 1])]).abs() <= 0.02).all())
    assert gq.gqa_device_status() == 0


def test_decode_over_a_shared_prefix(gq):
    """One token a request over a prefix that all share (read once, as one sequence of the batch's rows) and over its own
    tokens, merged, is the decode over all of them."""
    B, Hq, Hkv, D, ps, prefix, own = 6, 16, 4, 128, 16, 320, [1, 40, 17, 100, 64, 3]
    g = torch.Generator().manual_seed(60)
    ppr = 30
    k, v = (torch.randn(200, ps, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    pages = torch.randperm(200, generator=g).int()
    shared, rest = pages[:prefix // ps], pages[prefix // ps:prefix // ps + B * 8].view(B, 8)
    table = torch.cat([shared.expand(B, -1), rest], 1).contiguous().cuda()
    q = torch.randn(B, Hq, D, generator=g).to(torch.bfloat16).cuda()
    lens = torch.tensor(own, dtype=torch.int32).cuda()
    whole, whole_lse = gq.gqa_decode_paged(q[:, None].contiguous(), k, v, table, lens + prefix)
    a = gq.gqa_prefill_paged(q, k, v, shared[None].contiguous().cuda(), torch.tensor([prefix], dtype=torch.int32).cuda(), causal=False)
    b = gq.gqa_decode_paged(q[:, None].contiguous(), k, v, rest.contiguous().cuda(), lens)
    out, lse = gq.gqa_merge([a[0], b[0][:, 0].contiguous()], [a[1], b[1][..., 0].contiguous()])
    # roundings of either side to bf16 (out of about 1 at most: 2^-8 each, and of the parts), of weights on either side
    assert bool(((out.float() - whole[:, 0].float()).abs() <= 4 * 2.0 ** -8 * (1 + whole[:, 0].float().abs())).all())
    assert bool(((lse - whole_lse[..., 0]).abs() <= 1e-4).all())
    assert gq.gqa_device_status() == 0
