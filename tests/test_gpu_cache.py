"""GPU tests of appending to a paged cache and gathering from it, against plain computations, and of the run that a
server makes: append, decode, gather, dense attention."""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp8", "int8", "int4"]
SCALE = {"bf16": 1.0, "fp8": 0.011, "int8": 0.043, "int4": 1.0}


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_gb300 import build as gbuild
    gbuild.build()
    import gqa_decode_attention_gb300 as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def pools(kind, num_pages, ps, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    out, params = [], []
    for _ in range(2):
        c, p = ref.encode(kind, torch.randn(num_pages, ps, Hkv, D, generator=g), SCALE[kind])
        out.append(c)
        params.append(p)
    return out[0], out[1], torch.cat(params, -1) if kind == "int4" else None


def case(kind, B, new, before, Hq, Hkv, D, ps, seed, pad=0):
    """New tokens (in rows of a fused projection, `pad` rows behind the last) for requests that hold `before` already."""
    g = torch.Generator().manual_seed(seed)
    lens = [a + n for a, n in zip(before, new)]
    ppr = max(1, -(-max(lens) // ps)) + 1
    num_pages = B * ppr + 2
    T = sum(new)
    qkv = torch.randn(T + pad, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    k_pool, v_pool, params = pools(kind, num_pages, ps, Hkv, D, seed + 1)
    table = torch.randperm(num_pages, generator=g)[:B * ppr].view(B, ppr).to(torch.int32)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    return dict(kind=kind, qkv=qkv, Hq=Hq, Hkv=Hkv, k_pool=k_pool, v_pool=v_pool, params=params, table=table, cu=cu,
                lens=torch.tensor(lens, dtype=torch.int32), new=new, T=T, D=D, ps=ps)


def appended(d, rot, inter, table):
    """What the append leaves: (q_out of the real rows, k_pool, v_pool, params), every step in fp32 as stated."""
    Hq, Hkv, T = d["Hq"], d["Hkv"], d["T"]
    req = torch.repeat_interleave(torch.arange(len(d["new"])), torch.tensor(d["new"]))
    pos = d["lens"].long()[req] - torch.tensor(d["new"])[req] + torch.arange(T) - d["cu"].long()[req]
    x = d["qkv"][:T].float()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if rot:
        cos, sin = table[pos].chunk(2, -1)
        q, k = ref.rotate(q, cos, sin, rot, inter), ref.rotate(k, cos, sin, rot, inter)
    at = torch.tensor([int(ref.slots(d["table"][b], d["ps"], [p])) for b, p in zip(req.tolist(), pos.tolist())], dtype=torch.long)
    k_pool, v_pool = d["k_pool"].clone(), d["v_pool"].clone()
    params = None if d["params"] is None else d["params"].clone()
    for i, (pool, y) in enumerate(((k_pool, k), (v_pool, v))):
        c, p = ref.encode(d["kind"], y, SCALE[d["kind"]])
        pool.flatten(0, 1)[at] = c
        if p is not None:
            params.flatten(0, 1)[at, :, 2 * i:2 * i + 2] = p
    return q.to(torch.bfloat16), k_pool, v_pool, params


def append(gq, d, c, rot_table, inter, cu=True, **kw):
    Hq, Hkv = d["Hq"], d["Hkv"]
    qkv = c["qkv"]
    return gq.gqa_paged_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], c["k_pool"], c["v_pool"], c["table"], c["lens"],
                               cu_tokens=c["cu"] if cu else None, q=qkv[:, :Hq] if Hq else None,
                               cos_sin=rot_table, interleaved=inter, kv_params=c["params"], k_scale=SCALE[d["kind"]],
                               v_scale=SCALE[d["kind"]], **kw)


def cuda(d):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in d.items()}


def same(a, b):
    a, b = a.cpu(), b.cpu()
    if a.dtype == torch.bfloat16:
        a, b = a.view(torch.int16), b.view(torch.int16)
    elif a.dtype == torch.float16:
        a, b = a.view(torch.int16), b.view(torch.int16)
    return torch.equal(a, b)


# (B, new, before, Hq, Hkv, D, page size, rot, interleaved)
SHAPES = [
    (1, [1], [0], 1, 1, 64, 1, 64, False),
    (3, [1, 1, 1], [5, 0, 100], 8, 2, 128, 16, 128, False),
    (4, [7, 0, 33, 1], [3, 9, 0, 40], 6, 3, 64, 5, 32, True),
    (2, [40, 65], [0, 17], 64, 8, 128, 16, 128, True),
    (2, [3, 2], [1, 30], 5, 1, 128, 24, 16, False),
    (2, [19, 4], [2, 0], 0, 4, 64, 8, 64, False),       # no queries
    (2, [6, 6], [2, 0], 16, 16, 128, 7, 0, False),      # no rotation
    (70, [1] * 69 + [0], list(range(70)), 4, 2, 64, 16, 48, False),
    (1, [300], [0], 40, 5, 128, 128, 96, True),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "b%d_h%dx%d_d%d_ps%d_rot%d%s" % (s[0], *s[3:8], "i" if s[8] else ""))
def test_append_bytes(gq, kind, shape):
    """Bit for bit: the rotated queries, every pool byte and parameter, and nothing else touched."""
    B, new, before, Hq, Hkv, D, ps, rot, inter = shape
    d = case(kind, B, new, before, Hq, Hkv, D, ps, seed=sum(new) + D + ps, pad=2)
    table = ref.rope_table(max(a + b for a, b in zip(new, before)), rot) if rot else None
    q, k_pool, v_pool, params = appended(d, rot, inter, table)
    c = cuda(d)
    q_out = torch.full((d["T"] + 2, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda") if Hq else None
    got = append(gq, d, c, None if table is None else table.cuda(), inter, q_out=q_out)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
    assert same(c["k_pool"], k_pool) and same(c["v_pool"], v_pool)
    if params is not None:
        assert same(c["params"], params)
    if Hq:
        assert got is q_out and same(q_out[:d["T"]], q)
        assert torch.all(q_out[d["T"]:] == 3.0)  # rows behind the last request
    else:
        assert got is None


@pytest.mark.parametrize("kind", KINDS)
def test_rotation_against_64_bits(gq, kind):
    """Far positions: the rotated q and k against the formula in 64 bits with the table's fp32 entries.  Two products
    and a sum in fp32 are off by 2^-24 each of at most |x| + |y|; q is then rounded once (2^-8 of itself)."""
    d = case(kind, 1, [9], [999_990], 4, 2, 128, 64, seed=3)
    rot_table = ref.rope_table(1_000_000, 128)
    c = cuda(d)
    got = append(gq, d, c, rot_table.cuda(), False).cpu().double()
    assert gq.gqa_device_status() == 0
    cos, sin = rot_table[999_990:999_999].double().chunk(2, -1)
    x = d["qkv"][:9, :4].double()
    want = ref.rotate(x, cos, sin, 128, False)
    mag = x.abs() + x.abs().roll(64, -1)
    assert torch.all((got - want).abs() <= 3 * 2.0 ** -24 * mag + 2.0 ** -8 * want.abs())


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_device_scales(gq, kind):
    """Scales in device memory, one for all and one a head, give the host scales' bytes."""
    d = case(kind, 2, [5, 9], [0, 3], 4, 4, 64, 16, seed=4)
    table = ref.rope_table(32, 64).cuda()
    one = cuda(d)
    append(gq, d, one, table, False)
    for n in (1, 4):
        c = cuda(d)
        s = torch.full((n,), SCALE[kind], device="cuda")
        gq.gqa_paged_append(c["qkv"][:, 4:8], c["qkv"][:, 8:], c["k_pool"], c["v_pool"], c["table"], c["lens"],
                            cu_tokens=c["cu"], cos_sin=table, k_scales=s, v_scales=s)
        assert same(c["k_pool"], one["k_pool"]) and same(c["v_pool"], one["v_pool"])
        a = gq.gqa_paged_gather(c["k_pool"], c["v_pool"], c["table"], c["lens"], rows=12, k_scales=s, v_scales=s)
        b = gq.gqa_paged_gather(c["k_pool"], c["v_pool"], c["table"], c["lens"], rows=12, k_scale=SCALE[kind], v_scale=SCALE[kind])
        assert same(a[0], b[0]) and same(a[1], b[1])
    heads = torch.tensor([0.01, 0.02, 0.04, 0.08], device="cuda")
    c = cuda(d)
    gq.gqa_paged_append(c["qkv"][:, 4:8], c["qkv"][:, 8:], c["k_pool"], c["v_pool"], c["table"], c["lens"],
                        cu_tokens=c["cu"], cos_sin=table, k_scales=heads, v_scales=heads)
    for h in range(4):
        e = cuda(d)
        gq.gqa_paged_append(e["qkv"][:, 4:8], e["qkv"][:, 8:], e["k_pool"], e["v_pool"], e["table"], e["lens"],
                            cu_tokens=e["cu"], cos_sin=table, k_scale=float(heads[h]), v_scale=float(heads[h]))
        assert same(c["k_pool"][:, :, h], e["k_pool"][:, :, h]) and same(c["v_pool"][:, :, h], e["v_pool"][:, :, h])


def test_uniform_rows_and_in_place_queries(gq):
    """cu_tokens left out means T / B tokens each; q_out may be q."""
    d = case("bf16", 3, [4, 4, 4], [0, 7, 20], 8, 2, 128, 16, seed=5)
    table = ref.rope_table(32, 128)
    q, k_pool, v_pool, _ = appended(d, 128, False, table)
    c = cuda(d)
    own = c["qkv"][:, :8].contiguous()
    got = gq.gqa_paged_append(c["qkv"][:, 8:10], c["qkv"][:, 10:], c["k_pool"], c["v_pool"], c["table"], c["lens"], q=own,
                              q_out=own, cos_sin=table.cuda())
    assert same(got, q) and same(c["k_pool"], k_pool) and same(c["v_pool"], v_pool)


@pytest.mark.parametrize("kind", KINDS)
def test_special_values(gq, kind):
    """NaN, infinities, values past the code's range and constant rows, as the header states them."""
    d = case(kind, 1, [6], [0], 0, 2, 64, 16, seed=6)
    x = d["qkv"]
    x[0, 0, 5] = float("nan")
    x[1, 1, 3] = float("inf")
    x[2, 2, 60] = float("-inf")
    x[3] = 0.0
    x[4] = 1.5
    x[5, 3] = 1e5
    x[5, 1] *= 2.0 ** -30
    _, k_pool, v_pool, params = appended(d, 0, False, None)
    c = cuda(d)
    append(gq, d, c, None, False)
    assert gq.gqa_device_status() == 0
    if kind == "bf16":
        assert torch.equal(c["k_pool"].cpu().isnan(), k_pool.isnan())
        assert same(c["k_pool"].nan_to_num(9), k_pool.nan_to_num(9)) and same(c["v_pool"], v_pool)
        return
    k_got = c["k_pool"].cpu()
    if kind == "fp8":  # NaN codes may differ in sign
        nan = (k_pool & 127) == 127
        assert torch.all((k_got[nan] & 127) == 127)
        k_got = torch.where(nan, k_pool, k_got)
    assert torch.equal(k_got, k_pool) and same(c["v_pool"], v_pool)
    if params is not None:
        assert same(c["params"], params)


def test_skipped_tokens_are_flagged(gq):
    """Tokens without a place are left out and flagged: positions past the table, negative ones, bad pages (queries
    still rotated), positions past the rotation's table."""
    base = case("bf16", 2, [3, 3], [0, 20], 4, 2, 64, 16, seed=7)
    table = ref.rope_table(64, 64)

    def go(change, max_pos=64):
        d = {**base, "table": base["table"].clone(), "lens": base["lens"].clone()}
        change(d)
        c = cuda(d)
        q_out = torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        append(gq, d, c, table[:max_pos].contiguous().cuda(), False, q_out=q_out)
        torch.cuda.synchronize()
        assert gq.gqa_device_status() == 7
        return c, q_out.cpu()

    q, k_pool, v_pool, _ = appended(base, 64, False, table)
    old = base["k_pool"].flatten(0, 1)

    def only(d, c, kept):  # request 1's tokens `kept` written, request 0 whole
        want = old.clone()
        for b, ids in ((0, [0, 1, 2]), (1, kept)):
            for j in ids:
                at = int(ref.slots(base["table"][b], 16, [int(base["lens"][b]) - 3 + j]))
                want[at] = k_pool.flatten(0, 1)[at]
        return same(c["k_pool"].flatten(0, 1), want)

    c, q_out = go(lambda d: d["table"].__setitem__((1, 1), 10 ** 6))
    assert only(base, c, []) and same(q_out, q)
    c, q_out = go(lambda d: d["table"].__setitem__((1, 1), -1))
    assert only(base, c, []) and same(q_out, q)
    c, q_out = go(lambda d: None, max_pos=21)     # positions 21, 22 lie past the table
    assert only(base, c, [0]) and same(q_out[:4], q[:4]) and torch.all(q_out[4:] == 3.0)
    c, q_out = go(lambda d: d["lens"].__setitem__(1, 10 ** 6))
    assert only(base, c, []) and torch.all(q_out[3:] == 3.0)
    c, q_out = go(lambda d: d["lens"].__setitem__(1, -4))
    assert only(base, c, []) and torch.all(q_out[3:] == 3.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(3, 2, 64, 5, [0, 17, 40], [0, 3, 39]), (2, 8, 128, 16, [500, 33], [0, 0]), (4, 3, 64, 1, [7, 1, 0, 90], [2, 1, 0, 95])],
                         ids=["ps5", "ps16", "ps1"])
def test_gather(gq, kind, shape):
    """Values bit for bit as fp32 rounded to bf16; rows past a request's tokens untouched."""
    B, Hkv, D, ps, lens, starts = shape
    ppr = max(1, -(-max(lens) // ps))
    k_pool, v_pool, params = pools(kind, B * ppr + 1, ps, Hkv, D, seed=B)
    table = torch.randperm(B * ppr + 1, generator=torch.Generator().manual_seed(1))[:B * ppr].view(B, ppr).to(torch.int32)
    for rows in (max(lens), 20):
        k_out, v_out = (torch.full((B, rows, Hkv, D), 5.0, dtype=torch.bfloat16) for _ in range(2))
        want = [k_out.clone(), v_out.clone()]
        for b in range(B):
            n = min(rows, lens[b] - starts[b])
            if n <= 0:
                continue
            at = ref.slots(table[b], ps, range(starts[b], starts[b] + n))
            for i, pool in enumerate((k_pool, v_pool)):
                p = None if params is None else params.flatten(0, 1)[at][..., 2 * i:2 * i + 2]
                x = ref.values(kind, pool.flatten(0, 1)[at], p, float(torch.tensor(SCALE[kind]))) if kind == "bf16" else None
                if x is None:  # one fp32 rounding (two for 4-bit codes: the product is exact), then one to bf16
                    c = pool.flatten(0, 1)[at]
                    x = (ref.unpack_int4(c).float() * p[..., 0:1].float() + p[..., 1:2].float() if kind == "int4"
                         else c.view(torch.float8_e4m3fn).float() * SCALE[kind] if kind == "fp8" else c.float() * SCALE[kind])
                want[i][b, :n] = x.to(torch.bfloat16)
        kc, vc = k_out.cuda(), v_out.cuda()
        gq.gqa_paged_gather(k_pool.cuda(), v_pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), kc, vc,
                            starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                            kv_params=None if params is None else params.cuda(), k_scale=SCALE[kind], v_scale=SCALE[kind])
        torch.cuda.synchronize()
        assert gq.gqa_device_status() == 0
        assert same(kc, want[0]) and same(vc, want[1])


def test_gather_flags_bad_entries(gq):
    k_pool, v_pool, _ = pools("bf16", 6, 16, 2, 64, seed=1)
    table = torch.tensor([[0, 99], [2, -3]], dtype=torch.int32)
    lens = torch.tensor([32, 40], dtype=torch.int32)  # the second is past its two pages
    k, v = gq.gqa_paged_gather(k_pool.cuda(), v_pool.cuda(), table.cuda(), lens.cuda(), rows=40,
                               starts=torch.tensor([0, -2], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 7
    assert same(k[0, :16], k_pool[0]) and torch.all(k[0, 16:] == 0)
    assert same(v[1, :16], v_pool[2]) and torch.all(v[1, 16:] == 0)


def test_pools_beyond_four_gib(gq):
    """A pool of more than 2^32 bytes, pages at its far end: append and gather."""
    num_pages, ps, Hkv, D = 140_000, 16, 8, 128
    assert num_pages * ps * Hkv * D * 2 > 2 ** 32
    k_pool, v_pool = (torch.empty(num_pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[num_pages - 1, num_pages - 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 20, Hkv, D, device="cuda").to(torch.bfloat16)
    gq.gqa_paged_append(x[0], x[1], k_pool, v_pool, table, lens)
    k, v = gq.gqa_paged_gather(k_pool, v_pool, table, lens, rows=20)
    assert same(k[0], x[0]) and same(v[0], x[1])
    assert same(k_pool[num_pages - 1], x[0, :16]) and same(v_pool[num_pages - 3, :4], x[1, 16:])


def test_nothing_to_do(gq):
    d = case("int4", 2, [0, 0], [3, 5], 4, 2, 64, 16, seed=8)
    c = cuda(d)
    before = c["k_pool"].clone()
    assert append(gq, d, c, ref.rope_table(8, 64).cuda(), False).shape == (0, 4, 64)
    k, _ = gq.gqa_paged_gather(c["k_pool"], c["v_pool"], c["table"], c["lens"], rows=0, kv_params=c["params"])
    assert k.shape == (2, 0, 2, 64) and same(before, c["k_pool"])
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    k, _ = gq.gqa_paged_gather(c["k_pool"], c["v_pool"], c["table"], zero, rows=4, kv_params=c["params"])
    assert torch.all(k == 0)


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_then_decode_steps(gq, kind):
    """A server's run: ragged prompts appended, the prompt's rows attended through the dense call over gathered K and V,
    then decode steps that append one token and attend to the paged cache.  Every result against 64-bit attention over
    the values that the cache holds."""
    B, Hq, Hkv, D, ps = 2, 8, 2, 128, 16
    new = [48, 70]
    d = case(kind, B, new, [0, 0], Hq, Hkv, D, ps, seed=21)
    rot = ref.rope_table(128, D).cuda()
    c = cuda(d)
    sc = dict(k_scale=SCALE[kind], v_scale=SCALE[kind])
    q = append(gq, d, c, rot, False)
    dense = gq.gqa_paged_gather(c["k_pool"], c["v_pool"], c["table"], c["lens"], rows=70, kv_params=c["params"], **sc)

    def cached(b, n):
        at = ref.slots(c["table"][b].cpu(), ps, range(n))
        out = []
        for i, pool in enumerate((c["k_pool"], c["v_pool"])):
            p = None if c["params"] is None else c["params"].cpu().flatten(0, 1)[at][..., 2 * i:2 * i + 2]
            out.append(ref.values(kind, pool.cpu().flatten(0, 1)[at], p, SCALE[kind]))
        return out

    for b in range(B):
        qb = q[int(d["cu"][b]):int(d["cu"][b + 1])][None].contiguous()
        o, _ = gq.gqa_decode(qb, dense[0][b:b + 1, :new[b]].contiguous(), dense[1][b:b + 1, :new[b]].contiguous())
        k, v = cached(b, new[b])
        for i in (0, 1, new[b] - 1):
            want, _ = ref.attend(qb[0, i].cpu(), k, v, i + 1)
            # K and V rounded to bf16 by the gather, the weights and the output to bf16 by the dense call
            assert torch.all((o[0, i].cpu().double() - want).abs() <= 0.05 + 0.03 * want.abs())
    g = torch.Generator().manual_seed(22)
    for step in range(5):
        c["lens"] += 1
        x = torch.randn(B, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
        q1 = gq.gqa_paged_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], c["k_pool"], c["v_pool"], c["table"], c["lens"],
                                 q=x[:, :Hq], cos_sin=rot, kv_params=c["params"], **sc)
        if kind == "int4":
            o, lse = gq.gqa_decode_paged_int4(q1.view(B, 1, Hq, D), c["k_pool"], c["v_pool"], c["params"], c["table"], c["lens"])
        else:
            o, lse = gq.gqa_decode_paged(q1.view(B, 1, Hq, D), c["k_pool"], c["v_pool"], c["table"], c["lens"], **sc)
        assert gq.gqa_device_status() == 0
        for b in range(B):
            n = int(c["lens"][b])
            k, v = cached(b, n)
            want, s = ref.attend(q1[b].cpu(), k, v, n)
            assert torch.all((o[b, 0].cpu().double() - want).abs() <= 1e-2 + 1e-2 * want.abs()), (kind, step)
            assert torch.all((lse[b, :, 0].cpu().double() - s).abs() <= 1e-3)


def test_captured_step(gq):
    """A decode step captured once and replayed as its buffers change: append, then attend."""
    B, Hq, Hkv, D, ps = 3, 16, 4, 64, 16
    d = case("int4", B, [1, 1, 1], [30, 0, 63], Hq, Hkv, D, ps, seed=23)
    rot = ref.rope_table(128, D).cuda()
    c = cuda(d)

    def step(t):
        q = append(gq, d, t, rot, True)
        return gq.gqa_decode_paged_int4(q.view(B, 1, Hq, D), t["k_pool"], t["v_pool"], t["params"], t["table"], t["lens"])

    eager = cuda(d)
    step(eager)  # first call outside the capture
    eager = cuda(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, lse = step(c)
    g = torch.Generator().manual_seed(24)
    for _ in range(6):
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert same(c["k_pool"], eager["k_pool"]) and same(c["v_pool"], eager["v_pool"]) and same(c["params"], eager["params"])
        x = torch.randn(d["qkv"].shape, generator=g).to(torch.bfloat16).cuda()
        for t in (c, eager):
            t["qkv"].copy_(x)
            t["lens"] += 1


def test_on_a_given_stream(gq):
    d = case("int8", 2, [30, 50], [0, 10], 8, 2, 64, 16, seed=25)
    rot = ref.rope_table(64, 64).cuda()
    a, b = cuda(d), cuda(d)
    want = append(gq, d, a, rot, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = append(gq, d, b, rot, False, stream=s)
    k, v = gq.gqa_paged_gather(b["k_pool"], b["v_pool"], b["table"], b["lens"], rows=60, k_scale=0.5, v_scale=0.5, stream=s)
    torch.cuda.synchronize()
    assert same(got, want) and same(a["k_pool"], b["k_pool"])
    k2, v2 = gq.gqa_paged_gather(a["k_pool"], a["v_pool"], a["table"], a["lens"], rows=60, k_scale=0.5, v_scale=0.5)
    assert same(k, k2) and same(v, v2)


def test_same_slot_of_two_requests(gq):
    """Two tokens sent to one slot: whatever lies there after comes from either of them, and no other slot changes."""
    g = torch.Generator().manual_seed(27)
    k, v = (torch.randn(2, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    k_pool, v_pool = (torch.randn(4, 8, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    before = k_pool.clone(), v_pool.clone()
    table = torch.tensor([[2], [2]], dtype=torch.int32).cuda()
    lens = torch.tensor([5, 5], dtype=torch.int32).cuda()
    gq.gqa_paged_append(k, v, k_pool, v_pool, table, lens)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
    for pool, old, x in ((k_pool, before[0], k), (v_pool, before[1], v)):
        assert torch.all((pool[2, 4] == x[0]) | (pool[2, 4] == x[1]))
        pool[2, 4] = old[2, 4]
        assert torch.equal(pool, old)


def test_four_bit_scale_is_a_product(gq):
    """The scale is fp16 of (max - zero) times fp32's 1/15, which differs from fp16 of the quotient for some rows."""
    pairs = [(0.271484375, -0.00099945068359375), (0.55859375, -0.0010223388671875), (0.322265625, -0.00102996826171875),
             (1.1328125, -0.001068115234375)]
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    for i, (high, low) in enumerate(pairs):
        x[i, 0, 5], x[i, 0, 40] = high, low
    high, low = torch.tensor(pairs).T
    assert torch.equal(x[:, 0].float().amax(-1), high) and torch.equal(low.half().float(), low)
    scale = ((high - low) * (torch.tensor(1.0) / 15)).half()
    assert torch.all(scale != ((high - low) / 15).half())
    pool = torch.zeros(1, 16, 1, 32, dtype=torch.uint8, device="cuda")
    params = torch.zeros(1, 16, 1, 4, dtype=torch.float16, device="cuda")
    gq.gqa_paged_append(x.cuda(), x.cuda(), pool, pool.clone(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                        torch.tensor([4], dtype=torch.int32, device="cuda"), kv_params=params)
    want = torch.stack([scale, low.half(), scale, low.half()], -1)
    assert gq.gqa_device_status() == 0
    assert same(params[0, :4, 0], want)


def test_rows_before_the_first_request(gq):
    """Rows before cu_tokens[0] belong to nobody: skipped whole and flagged, as the header says; the others go where
    they belong."""
    d = case("bf16", 2, [3, 2], [4, 0], 4, 2, 64, 16, seed=33)
    d["qkv"] = torch.cat([torch.ones(2, *d["qkv"].shape[1:], dtype=torch.bfloat16), d["qkv"]])
    table = ref.rope_table(32, 64)
    q, k_pool, v_pool, _ = appended({**d, "qkv": d["qkv"][2:]}, 64, False, table)
    c = cuda({**d, "cu": d["cu"] + 2})
    q_out = torch.full((7, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    append(gq, d, c, table.cuda(), False, q_out=q_out)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 7
    assert same(c["k_pool"], k_pool) and same(c["v_pool"], v_pool)
    assert torch.all(q_out[:2] == 3.0) and same(q_out[2:], q)
