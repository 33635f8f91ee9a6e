"""GPU tests of prompt attention at its edges, against plain 64-bit computations."""
import math

import pytest
import torch

import cache_ref as cref
import prefill_ref as ref

pytestmark = pytest.mark.gpu


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


# ------------------------------------------------------------------------------------------------ items without a key
@pytest.mark.parametrize("kind,ps", [("bf16", 1), ("bf16", 5), ("bf16", 7), ("bf16", 16), ("fp8", 1), ("int8", 7), ("int4", 5)])
@pytest.mark.parametrize("n,L,causal", [
    ([1] * 64, [1000, 0] * 32, True),                      # decode tokens beside padded slots
    ([1] * 256, [1000] * 20 + [0] * 236, True),
    ([5, 2000, 3], [10, 10, 10], True),                    # far more new rows than keys
    ([40] * 128, [0] * 100 + [300] * 28, False),           # requests without a cached prefix
])
def test_many_items_without_a_key(gq, kind, ps, n, L, causal):
    """A worker's list ends in items that see no key: behind the last one that does, the loader waits for pieces that are
    published as the softmax comes by, so it must not keep that one's values to itself."""
    d = ref.make(n, L, 64, 8, 64, seed=len(n) + ps, kind=kind, ps=ps)
    ref.check(d, *run(gq, d, causal), causal)


@pytest.mark.parametrize("ps", [1, 5, 7])
def test_prefixes_of_some(gq, ps):
    """Long chunks over cached prefixes that two thirds of the requests do not have."""
    n, L = [512] * 48, [0] * 32 + [640] * 16
    d = ref.make(n, L, 64, 8, 128, seed=ps, kind="bf16", ps=ps)
    out, lse = run(gq, d, False)
    assert torch.all(out[:512 * 32] == 0) and torch.all(lse[:512 * 32] == -float("inf"))
    last = dict(d, n=n[32:], L=L[32:], q=d["q"][512 * 32:], kv=d["kv"][32:], rows=d["rows"][32:])
    ref.check(last, out[512 * 32:], lse[512 * 32:], False)


@pytest.mark.parametrize("kind", ["fp8", "int8", "int4"])
def test_short_pieces_of_codes(gq, kind):
    """Many pieces of one to three steps a worker: the codes of each piece's first step come while those before are in use.
    The same bits every time."""
    n, L = [1, 20, 3] * 60, [100, 300, 257] * 60
    d = ref.make(n, L, 32, 8, 128, seed=3, kind=kind)
    want = run(gq, d)
    ref.check(d, *want)
    for _ in range(20):
        got = run(gq, d)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


# ------------------------------------------------------------------------------------------------ weights in 16 bits
def one_large_score(gq, kind, first, large):
    """One key's weight is 2^25.4 times that of each of the 2^20 - 1 others, which together are 2.3 % of the row: they count in
    the sum, so they must count in the product with V.  Its value is `large`, theirs 1.  (Whole items, two an SM: parts of a
    divided one have references of their own.)"""
    Hq, Hkv, D, ps, L = 8, 1, 64, 16, 1 << 20
    T = 2 * 32 * torch.cuda.get_device_properties(0).multi_processor_count
    scale = 1 / 8 if kind in ("fp8", "int8") else 1.0
    k, v = torch.zeros(2, ps, Hkv, D), torch.ones(2, ps, Hkv, D)
    at = 0 if first else ps - 1  # page 0 holds the large key, page 1 is all the others
    k[0, at, 0, 7], v[0, at] = 2.0, large
    (kc, kp), (vc, vp) = cref.encode(kind, k, scale), cref.encode(kind, v, scale)
    params = torch.cat([kp, vp], -1).cuda() if kind == "int4" else None
    table = torch.ones(1, L // ps, dtype=torch.int32)
    table[0, 0 if first else -1] = 0
    q = torch.zeros(T, Hq, D)
    q[..., 7] = 25.4 * math.log(2) * math.sqrt(D) / 2
    d = dict(kind=kind, q=q.to(torch.bfloat16).cuda(), k_pool=kc.cuda(), v_pool=vc.cuda(), params=params, table=table.cuda(), scale=scale,
             lens=torch.tensor([L], dtype=torch.int32).cuda(), cu=torch.tensor([0, T], dtype=torch.int32).cuda(), Hq=Hq, Dv=D)
    out, lse = run(gq, d, causal=False)
    s = float(d["q"][0, 0, 7].double()) * float(cref.values(kind, kc, kp, scale)[0, at, 0, 7]) / math.sqrt(D)
    rest = (L - 1) * math.exp(-s)
    want, mag, want_lse = (rest + large) / (rest + 1), (rest + abs(large)) / (rest + 1), s + math.log1p(rest)
    # as prefill_ref.bounds, but small weights are off by 2^-32 of the largest at most
    steps, ds = (L / 128 + 160) * 2.0 ** -23, (D + 8) * 2.0 ** -23 * s
    half = ref.HALF[torch.bfloat16] if kind == "bf16" else ref.HALF[torch.float16] * (2 if kind == "int4" else 1)
    rel = half + 2 * ds + 2.0 ** -20 + 2 * steps
    bound = ref.HALF[torch.bfloat16] * abs(want) + rel * mag + (0.0 if kind == "bf16" else L * 2.0 ** -32)
    assert bound < 0.5 * rest  # what the others' part is
    assert float((out.double() - want).abs().max()) <= bound
    assert float((lse.double() - want_lse).abs().max()) <= ds + steps + 2.0 ** -20 + 2.0 ** -22 * want_lse


@pytest.mark.parametrize("kind", ["fp8", "int8", "int4"])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_weights(gq, kind, first):
    """The others' values are all that the row's result consists of: their weights must not be rounded to nothing."""
    one_large_score(gq, kind, first, 0.0)


@pytest.mark.parametrize("kind", ["fp8", "int8", "int4"])
def test_scores_of_great_magnitude(gq, kind):
    """Scores up to 2^27: a row is the value of its largest score's key."""
    n, L, Hq, Hkv, D = [70, 5], [70, 900], 8, 2, 64
    d = ref.make(n, L, Hq, Hkv, D, seed=21, kind=kind, gain=2.0 ** 23)
    out, lse = run(gq, d)
    at = 0
    for (k, v), nb, Lb in zip(d["kv"], n, L):
        x = torch.einsum("nhgd,lhd->nhgl", d["q"][at:at + nb].double().view(nb, Hkv, Hq // Hkv, D), k) / math.sqrt(D)
        hide = torch.arange(Lb, device="cuda") > (Lb - nb + torch.arange(nb, device="cuda"))[:, None]
        x = x.masked_fill(hide[:, None, None], -math.inf)
        assert 2.0 ** 24 < float(x.nan_to_num(neginf=0.0).abs().max()) < 2.0 ** 27
        best = x.topk(min(2, Lb), -1)
        # what the scores may be off by: (D + 8) 2^-23 of their magnitude, below 2^29 with a 4-bit scale and zero apart
        clear = best.values[..., 0] - best.values[..., 1] > 72 * 2.0 ** -23 * 2.0 ** 29 + 64
        assert clear.float().mean() > 0.8
        want = torch.gather(v.permute(1, 0, 2)[None].expand(nb, -1, -1, -1), 2, best.indices[..., :1].expand(-1, -1, -1, D))
        got = out[at:at + nb].double().view(nb, Hkv, Hq // Hkv, D)
        assert torch.isfinite(got).all() and torch.isfinite(lse[at:at + nb]).all()
        e = (got - want).abs() - (2.0 ** -8 + 2 * 2.0 ** -11) * want.abs() - 2.0 ** -20
        assert float(e[clear].max()) <= 0
        at += nb


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8", "int4"])
@pytest.mark.parametrize("ps", [16, 7])
def test_rows_past_the_scores_range(gq, kind, ps):
    """A row of queries up to 2^125 may be NaN; the call ends, and every other row is as before."""
    d = ref.make([50, 3], [50, 500], 12, 4, 64, seed=22, kind=kind, ps=ps)  # (groups that leave rows of a tile empty)
    want = run(gq, d)
    for up in (40, 90, 122):
        e = dict(d, q=d["q"].clone())
        e["q"][[7, 51]] *= 2.0 ** up
        got = run(gq, e)
        keep = [i for i in range(53) if i not in (7, 51)]
        for a, b in zip(want, got):
            assert torch.equal(a[keep], b[keep])


# ------------------------------------------------------------------------------------------------ sums over many steps
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8", "int4"])
@pytest.mark.parametrize("first", [True, False])
def test_small_weights_beside_a_large_value(gq, kind, first):
    """As above, and the large key's value is what the row mostly consists of: the others' products lie 2^-25 below."""
    one_large_score(gq, kind, first, -1.0)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_long_sums_of_one_sign(gq, kind):
    """2^20 keys with values between 1 and 2: nothing is lost on the way (what the tensor core cuts off is always towards zero)."""
    Hq, Hkv, D, ps, pages, L = 8, 1, 64, 16, 64, 1 << 20
    T = 2 * 32 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(23)
    scale = 5 / 448 if kind == "fp8" else 1.0
    k, v = torch.randn(pages, ps, Hkv, D, generator=g), torch.rand(pages, ps, Hkv, D, generator=g) * 0.3 + torch.linspace(1.0, 1.7, D)
    (kc, kp), (vc, vp) = cref.encode(kind, k, scale), cref.encode(kind, v, scale)
    params = torch.cat([kp, vp], -1) if kind == "int4" else None
    table = torch.randint(0, pages, (1, L // ps), generator=g).int()
    q = torch.randn(32, Hq, D, generator=g).to(torch.bfloat16).cuda().repeat(T // 32, 1, 1)
    d = dict(kind=kind, q=q, k_pool=kc.cuda(), v_pool=vc.cuda(), params=None if params is None else params.cuda(), table=table.cuda(), scale=scale,
             lens=torch.tensor([L], dtype=torch.int32).cuda(), cu=torch.tensor([0, T], dtype=torch.int32).cuda(), Hq=Hq, Dv=D)
    out, lse = run(gq, d, causal=False)
    kd, vd = cref.values(kind, kc, kp, scale).view(-1, D).cuda(), cref.values(kind, vc, vp, scale).view(-1, D).cuda()
    times = torch.bincount(table[0], minlength=pages).double().repeat_interleave(ps).cuda()
    p = torch.softmax(q[:32].double().view(-1, D) @ kd.T / math.sqrt(D) + times.log(), -1)
    want = (p @ vd).view(32, Hq, D)
    # bf16 rounds either way over values between 1 and 2: their mean moves little.  A product loses less than 2^-24 of the sum that
    # it is added to, over 32768 keys.
    off = float(((out[:32].double() - want) / want).mean())
    assert abs(off) <= 2.0 ** -24 * 32768 + 2.0 ** -12
    assert torch.equal(out[:32], out[32:64]) and torch.equal(lse[:32], lse[-32:])


@pytest.mark.parametrize("kind,ps", [("bf16", 16), ("bf16", 7), ("fp8", 16), ("int4", 16)])
@pytest.mark.parametrize("n", [[1500], [16] * 90])  # items of two tiles, and of one, whose steps the row groups take in turns
@pytest.mark.parametrize("rise", [False, True])
def test_sums_that_leave_the_tensor_core(gq, kind, ps, n, rise):
    """Whole items and parts of more steps than a sum stays in the tensor core for, the largest scores at the end or anywhere."""
    Hq, Hkv, D, L = 16, 2, 64, 70000
    d = ref.make([1], [L], Hq, Hkv, D, seed=24, kind=kind, ps=ps, pad=0)
    B, T = len(n), sum(n)
    g = torch.Generator().manual_seed(25)
    if rise:  # keys grow along the sequence
        up = torch.linspace(0.25, 2.0, L)
        k = torch.randn(L, Hkv, D, generator=g) * up[:, None, None]
        kc, kp = cref.encode(kind, k, d["scale"])
        d["k_pool"].view(-1, *kc.shape[1:])[d["rows"][0]] = kc.cuda()
        if kind == "int4":
            d["params"].view(-1, Hkv, 4)[d["rows"][0], :, :2] = kp.cuda()
        d["kv"] = [ref.held(d, d["rows"][0])]
    q = torch.randn(T + 3, Hq, D, generator=g)
    d.update(n=n, L=[L] * B, q=(q * 2).to(torch.bfloat16).cuda(), cu=torch.tensor([0] + n).cumsum(0).int().cuda(), table=d["table"].expand(B, -1).contiguous(),
             lens=torch.full((B,), L, dtype=torch.int32).cuda(), rows=d["rows"] * B, kv=d["kv"] * B)
    out, lse = run(gq, d)
    step = 1 if B == 1 else 13  # requests checked
    for b in range(0, B, step):
        at = sum(n[:b])
        one = dict(d, n=[n[b]], L=[L], q=d["q"][at:at + n[b]], kv=[d["kv"][b]], rows=[d["rows"][b]])
        ref.check(one, out[at:at + n[b]], lse[at:at + n[b]], untouched=False, what=f"request {b}")
    again = run(gq, d)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


# ------------------------------------------------------------------------------------------------ values past fp16's largest
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,L,Hq,Hkv,D", [([150, 20], [400, 20], 8, 4, 64), ([3, 40], [1500, 700], 16, 2, 128)])
def test_large_values_of_4_bits(gq, n, L, Hq, Hkv, D, causal):
    """15 scales and a zero reach 2^20: tokens here and there, fp16's largest parameters among them."""
    d = ref.make(n, L, Hq, Hkv, D, seed=26, kind="int4")
    base = run(gq, d, causal)
    params = d["params"].flatten(0, 1)
    at = d["rows"][0][100:]
    for i, (vs, vz) in enumerate([(65504.0, 65504.0), (30000.0, -225000.0 / 15), (65504.0, -65504.0), (4400.0, -500.0), (9000.0, -65504.0), (0.0, 65504.0)]):
        params[at[i * 41], i % Hkv, 2:] = torch.tensor([vs, vz]).half().cuda()
    params[d["rows"][1][7], :, 2] = 50000.0
    d["kv"] = [ref.held(d, r) for r in d["rows"]]
    assert float(d["kv"][0][1].abs().max()) == 16 * 65504.0
    out, lse = run(gq, d, causal)
    assert torch.equal(lse, base[1])
    t = 0
    for b, (nb, Lb) in enumerate(zip(n, L)):
        q, (k, v) = d["q"][t:t + nb].double(), d["kv"][b]
        want, want_lse, mag, _, v_max = ref.attend(q, k, v, causal)
        p = params[d["rows"][b]].double()
        s_mag = q.abs().sum(-1) * (15 * p[..., 0] + p[..., 1].abs()).amax(0).repeat_interleave(Hq // Hkv) / math.sqrt(D)
        steps, ds = (Lb / 128 + 160) * 2.0 ** -23, (D + 8) * 2.0 ** -23 * s_mag
        # weights and values are off by 2^-11 each; small weights by 2^-32 of the largest, small values beside a large one by 2^-16
        rel = 2 * ref.HALF[torch.float16] + 2 * ds + 2.0 ** -20 + 2 * steps
        bound = 1.01 * (ref.HALF[torch.bfloat16] * want.abs() + rel[..., None] * mag) + (Lb * 2.0 ** -32 * v_max)[..., None] + 2.0 ** -16
        e = (out[t:t + nb].double() - want).abs()
        assert bool((e <= bound).all()), f"request {b}: {float((e - bound).max())} past the bound"
        t += nb
    if causal and L[0] > n[0]:  # rows that see no large value stay within what they were
        before = max(0, 96 - (L[0] - n[0]))
        assert torch.equal(out[:before], base[0][:before])


# ------------------------------------------------------------------------------------------------ V that is not finite
@pytest.mark.parametrize("kind,ps", [("bf16", 16), ("bf16", 7), ("fp8", 16), ("int4", 16)])
def test_values_of_nan_under_the_least_wait_limit(gq, kind, ps):
    """Every element of V is NaN: rows get theirs back in the epilogue, which must not take so long that the warps that wait for
    it give up (many items an SM, each of short keys, and the least limit that can be set)."""
    d = ref.make([256] * 4, [256] * 4, 8, 8, 128, seed=27, kind=kind, ps=ps)
    if kind == "int4":
        d["params"][..., 2] = math.nan
    else:
        d["v_pool"].fill_(127 if kind == "fp8" else math.nan)
    B = 300
    d["q"] = torch.cat([d["q"][:1024]] * (B // 4))
    e = dict(d, cu=(torch.arange(B + 1) * 256).int().cuda(), table=d["table"].repeat(B // 4, 1), lens=d["lens"].repeat(B // 4))
    gq.gqa_set_wait_limit_ns(1)  # raised to 1 ms
    try:
        out, lse = run(gq, e)
    finally:
        gq.gqa_set_wait_limit_ns(0)
    assert torch.isnan(out).all()
    for b in range(4):
        want = ref.attend(d["q"][256 * b:256 * b + 256].double(), d["kv"][b][0], torch.zeros_like(d["kv"][b][0]), True)[1]
        assert bool(((lse[256 * b:256 * b + 256].double() - want).abs() < 1e-4).all())
    assert torch.equal(lse, lse[:1024].repeat(B // 4, 1))


@pytest.mark.parametrize("kind", ["dense", "bf16", "fp8"])
def test_some_values_not_finite(gq, kind):
    """Single elements in the last tokens, each sign and NaN: they reach that element of the rows that see them."""
    L = [200, 60]
    d = ref.make(L, L, 8, 4, 64, seed=28, kind=kind)
    base = run(gq, d)
    bad = [(150, 1, 3, math.inf), (151, 1, 3, -math.inf), (160, 2, 63, -math.inf), (161, 3, 8, math.nan), (199, 0, 0, math.inf), (170, 2, 62, math.inf)]
    want = base[0][:200].float().clone()
    for t, g, e, x in bad:
        x = math.nan if kind == "fp8" else x
        if kind == "dense":
            d["v"][t, g, e] = x
        else:
            d["v_pool"].flatten(0, 1)[d["rows"][0][t], g, e] = 127 if kind == "fp8" else x
        want[t:, 2 * g:2 * g + 2, e] += x
    out, lse = run(gq, d)
    assert torch.equal(lse, base[1]) and torch.equal(out[200:], base[0][200:])
    got = out[:200].float()
    assert torch.equal(torch.nan_to_num(got, nan=9e9), torch.nan_to_num(want, nan=9e9))


@pytest.mark.parametrize("D,Dv", [(64, 64), (128, 128), (192, 128)])
def test_packed_sums_that_leave_the_tensor_core(gq, D, Dv):
    """The same over packed keys, in a workspace of NaN, called and as a captured graph."""
    n, L, Hq, Hkv = [1500], [70000], 16, 2
    d = ref.make(n, L, Hq, Hkv, D, seed=29, Dv=Dv)
    need = gq.gqa_prefill_workspace_bytes(d["q"].shape[0], 1, Hq, Hkv, D, Dv)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out, lse = run(gq, d, workspace=ws)
    ref.check(d, out, lse)
    got = torch.full_like(out, -7.0), torch.full_like(lse, -7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ref.call(gq, d, workspace=ws, out=got[0], lse=got[1])
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
