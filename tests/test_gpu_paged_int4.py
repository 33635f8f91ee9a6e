"""GPU parity of paged decode over a 4-bit cache, through the Python binding, against a plain 64-bit computation on
the same codes, scales and zeros."""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_gb300 import build as gbuild
    gbuild.build()
    import gqa_decode_attention_gb300 as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def make(B, Sq, Hq, Hkv, D, ps, lens, seed, ppr=None, extra=3, v_gain=1.0):
    """A cache in use.  Slots that hold no token of a request carry NaN and infinite parameters, and table entries past
    a request's pages are out of range: neither may be read into a result."""
    g = torch.Generator().manual_seed(seed)
    ppr = max(1, -(-max(lens) // ps)) if ppr is None else ppr
    num_pages = B * ppr + extra
    q = torch.randn(B, Sq, Hq, D, generator=g).to(torch.bfloat16)
    x = torch.randn(2, num_pages, ps, Hkv, D, generator=g)
    x[1] *= v_gain
    kc, kp = ref.encode_int4(x[0])
    vc, vp = ref.encode_int4(x[1])
    params = torch.cat([kp, vp], -1)
    table = torch.randperm(num_pages, generator=g)[:B * ppr].view(B, ppr).to(torch.int32)
    used = torch.zeros(num_pages * ps, dtype=torch.bool)
    for b, n in enumerate(lens):
        if n:
            used[ref.slots(table[b], ps, range(n))] = True
        table[b, -(-n // ps):] = 2 ** 31 - 1 if b % 2 else -7
    flat = params.view(-1, Hkv, 4)
    flat[~used] = torch.tensor([float("nan"), float("inf"), float("inf"), float("nan")]).half()
    return dict(q=q, k_pool=kc, v_pool=vc, params=params, table=table, lens=torch.tensor(lens, dtype=torch.int32))


def run(gq, d, **kw):
    c = {n: t.cuda() for n, t in d.items()}
    out, lse = gq.gqa_decode_paged_int4(c["q"], c["k_pool"], c["v_pool"], c["params"], c["table"], c["lens"], **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check(d, out, lse, rows=None, what="", skip=None):
    """Every query row (or the batch rows given) against 64 bits, within the bounds of cache_ref.int4_bounds."""
    B, Sq, Hq, D = d["q"].shape
    ps, Hkv = d["k_pool"].shape[1:3]
    for b in range(B) if rows is None else rows:
        n = int(d["lens"][b])
        at = ref.slots(d["table"][b], ps, range(n)) if n else torch.zeros(0, dtype=torch.long)
        p = d["params"].flatten(0, 1)[at]
        k = ref.value_int4(d["k_pool"].flatten(0, 1)[at], p[..., :2])
        v = ref.value_int4(d["v_pool"].flatten(0, 1)[at], p[..., 2:])
        if skip is not None and n:
            keep = skip(b, n)
            k, v, p = k[keep], v[keep], p[keep]
        ds, v_range, v_mag = ref.int4_bounds(d["q"][b], p, D)
        for i in range(Sq):
            seen = n - Sq + i + 1
            if skip is not None and n:
                seen = int(skip(b, n)[:max(seen, 0)].sum())
            o, s = ref.attend(d["q"][b, i], k, v, seen)
            if seen <= 0:
                assert torch.all(out[b, i] == 0) and torch.all(torch.isneginf(lse[b, :, i])), what
                continue
            # a weight is off by its score's error (twice: numerator and sum) and its fp16 rounding; the sum of fp32
            # terms over the tokens by 2^-23 a step of a pairwise-merged walk (2^-17 covers any walk here)
            tol = 2 * ds * v_mag + 2.0 ** -11 * v_range + 2.0 ** -17 * v_mag + 2.0 ** -8 * o.abs()
            err = (out[b, i].double() - o).abs()
            assert torch.all(err <= tol), f"{what}: request {b} row {i}: out off by {float((err - tol).max())} over {float(tol.max())}"
            el = (lse[b, :, i].double() - s).abs()
            assert torch.all(el <= ds + 2.0 ** -17), f"{what}: request {b} row {i}: lse off by {float(el.max())}, bound {ds}"


# (B, Sq, Hq, Hkv, D, page_size, lens)
SHAPES = [
    (1, 1, 1, 1, 64, 1, (1,)),                        # one token, one head, pages of one
    (1, 1, 8, 2, 64, 5, (1000,)),
    (3, 1, 32, 8, 128, 16, (128, 77, 1)),
    (4, 1, 64, 8, 128, 16, (0, 640, 33, 0)),          # empty requests
    (2, 4, 32, 8, 128, 32, (300, 2)),                 # 16 rows a KV head; two rows see nothing
    (2, 3, 10, 2, 128, 24, (97, 500)),                # 15 rows, page size 8 x 3
    (1, 2, 12, 12, 128, 16, (700,)),                  # 12 KV heads: a last block of 4
    (2, 1, 3, 3, 64, 8, (65, 31)),                    # 3 KV heads
    (1, 1, 32, 1, 64, 16, (3001,)),                   # 32 rows on one KV head
    (2, 4, 16, 1, 128, 16, (513, 40)),                # 64 rows on one KV head
    (1, 2, 128, 2, 64, 64, (900,)),                   # 128 rows a KV head
    (2, 16, 8, 1, 128, 7, (150, 10)),                 # 128 rows, odd pages, rows that see nothing
    (1, 1, 48, 16, 64, 128, (260,)),                  # 16 KV heads
    (5, 1, 5, 1, 128, 3, (95, 96, 97, 31, 32)),       # around the stage's 32 tokens
    (1, 1, 20, 20, 64, 2, (333,)),
    (40, 1, 16, 4, 128, 16, tuple(range(1, 41))),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "b%d_sq%d_h%dx%d_d%d_ps%d" % s[:6])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_matches_64_bits(gq, shape, splits):
    d = make(*shape[:6], list(shape[6]), seed=sum(shape[:6]))
    out, lse = run(gq, d, num_splits=splits)
    assert gq.gqa_device_status() == 0
    check(d, out, lse, what=f"{shape} splits {splits}")


@pytest.mark.parametrize("splits", [0, 2, 9])
def test_same_splits_same_bits(gq, splits):
    d = make(6, 2, 32, 8, 128, 16, [700, 0, 15, 1200, 64, 333], seed=5)
    first = run(gq, d, num_splits=splits)
    for _ in range(5):
        again = run(gq, d, num_splits=splits)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("D", [64, 128])
def test_more_workers_than_steps(gq, D):
    d = make(2, 1, 8, 2, D, 16, [40, 3], seed=6)
    out, lse = run(gq, d, num_splits=64)
    check(d, out, lse)


def test_bad_pages_and_lengths_are_flagged(gq):
    """An out-of-range page inside a request: its tokens are skipped and the device error word says so; a length past
    the table's capacity or below zero is clamped, and flagged."""
    d = make(3, 1, 16, 4, 128, 16, [100, 64, 90], seed=7)
    d["table"][0, 2] = 10 ** 6
    d["table"][2, 0] = -1
    out, lse = run(gq, d)
    assert gq.gqa_device_status() == 7

    def skip(b, n):
        keep = torch.ones(n, dtype=torch.bool)
        if b == 0:
            keep[32:48] = False
        if b == 2:
            keep[0:16] = False
        return keep

    safe = {**d, "table": d["table"].clamp(0, d["k_pool"].shape[0] - 1)}
    check(safe, out, lse, skip=skip)
    d = make(3, 1, 16, 4, 128, 16, [96, 64, 0], seed=8)
    over = {**d, "lens": torch.tensor([97, 64, -5], dtype=torch.int32)}
    out, lse = run(gq, over)
    assert gq.gqa_device_status() == 7
    check(d, out, lse)


@pytest.mark.parametrize("splits", [0, 1, 5])
def test_requests_that_share_pages(gq, splits):
    """Requests with the same pages (a common prefix), one of them with the same page more than once."""
    d = make(4, 1, 16, 4, 128, 16, [200, 200, 200, 200], seed=23)
    d["table"][1] = d["table"][0]
    d["table"][2, :9] = d["table"][0, :9]
    d["table"][3] = d["table"][3, 2]
    out, lse = run(gq, d, num_splits=splits)
    assert gq.gqa_device_status() == 0
    check(d, out, lse)


def test_all_pages_bad(gq):
    d = make(1, 2, 8, 2, 64, 16, [100], seed=9)
    d["table"][:] = -1
    out, lse = run(gq, d, num_splits=3)
    assert gq.gqa_device_status() == 7
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("gain", [2.0 ** -20, 1e-3, 300.0, 2e4])
def test_value_magnitudes(gq, gain):
    """V scales from the subnormal end of fp16 to its top."""
    d = make(2, 1, 16, 2, 128, 16, [400, 1000], seed=10, v_gain=gain)
    out, lse = run(gq, d, num_splits=5)
    assert gq.gqa_device_status() == 0
    check(d, out, lse, what=f"gain {gain}")


def test_mixed_value_scales(gq):
    """Tokens whose V scales differ by 2^20, constant rows (scale 0) among them."""
    d = make(2, 1, 16, 2, 128, 16, [600, 900], seed=11)
    g = torch.Generator().manual_seed(12)
    e = torch.randint(-14, 7, d["params"].shape[:-1], generator=g).float()
    p = d["params"].float()
    p[..., 2:] = p[..., 2:] * (2.0 ** e)[..., None]
    zero = torch.rand(d["params"].shape[:-1], generator=g) < 0.2
    p[..., 2][zero] = 0.0
    d["params"] = p.half()
    d["v_pool"][zero] = 0
    out, lse = run(gq, d)
    check(d, out, lse)


def test_peaked_and_growing_scores(gq):
    """Scores that grow along the request by hundreds (the running maximum moves at every step), and one token far
    above all others."""
    d = make(2, 1, 8, 1, 64, 16, [800, 800], seed=13)
    p = d["params"].float()
    for b, f in ((0, lambda t: 1.0 + t.float() / 8), (1, lambda t: torch.where(t == 417, 200.0, 1.0))):
        t = torch.arange(800)
        at = ref.slots(d["table"][b], 16, t)
        p.view(-1, 1, 4)[at, :, :2] *= f(t)[:, None, None]
    d["params"] = p.half()
    for splits in (0, 1, 4):
        out, lse = run(gq, d, num_splits=splits)
        check(d, out, lse, what=f"splits {splits}")


def test_large_and_small_queries(gq):
    d = make(1, 1, 8, 2, 128, 16, [300], seed=14)
    scale = torch.tensor([2.0 ** -60, 2.0 ** -20, 1.0, 2.0 ** 6, 1.0, 2.0 ** -100, 0.0, 1.0]).view(1, 1, 8, 1)
    d["q"] = (d["q"].float() * scale).to(torch.bfloat16)
    out, lse = run(gq, d)
    check(d, out, lse)


def test_nan_rows_stay_their_own(gq):
    """A query row with NaN or infinity gives NaN; the other rows keep every bit."""
    d = make(2, 2, 16, 2, 128, 16, [300, 500], seed=15)
    clean = run(gq, d, num_splits=3)
    bad = {**d, "q": d["q"].clone()}
    bad["q"][0, 1, 3, 17] = float("nan")
    bad["q"][1, 0, 9, 100] = float("inf")
    out, lse = run(gq, bad, num_splits=3)
    hit = torch.zeros(2, 2, 16, dtype=torch.bool)
    hit[0, 1, 3] = hit[1, 0, 9] = True
    assert torch.all(torch.isnan(out[hit])) and torch.all(torch.isnan(lse.permute(0, 2, 1)[hit]))
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse.permute(0, 2, 1)[~hit], clean[1].permute(0, 2, 1)[~hit])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_parameters_that_are_not_finite(gq, value, which):
    """A token's K scale or zero, or V scale or zero, NaN or infinite (a scale below zero has no meaning): the rows that
    see it have no finite result, the rows and heads that do not keep every bit."""
    if which % 2 == 0 and value < 0:
        value = float("nan")
    d = make(2, 3, 16, 2, 128, 16, [300, 500], seed=21)
    clean = run(gq, d, num_splits=3)
    bad = {**d, "params": d["params"].clone()}
    at = lambda b, t: int(ref.slots(d["table"][b], 16, [t])[0])  # noqa: E731
    flat = bad["params"].view(-1, 2, 4)
    flat[at(0, 299), 1, which] = value  # seen by the last row of request 0 only
    flat[at(1, 498), 0, which] = value  # by the last two of request 1
    flat[at(1, 100), 1, which] = value  # by all
    out, lse = run(gq, bad, num_splits=3)
    hit = torch.zeros(2, 3, 16, dtype=torch.bool)
    hit[0, 2, 8:] = hit[1, 1:, :8] = hit[1, :, 8:] = True
    assert torch.equal(out[~hit], clean[0][~hit])
    assert torch.equal(lse.permute(0, 2, 1)[~hit], clean[1].permute(0, 2, 1)[~hit])
    if which >= 2 or value != value:  # a K parameter of infinity may give scores of -inf alone, which weigh nothing
        assert not torch.any(torch.isfinite(out[hit]).all(-1))


def test_codes_beyond_four_gib(gq):
    """Pools of more than 4 GiB each, the request's pages at their far end."""
    num_pages, ps, Hkv, D = 540_000, 16, 8, 128
    assert num_pages * ps * Hkv * D // 2 > 2 ** 32
    small = make(2, 1, 16, Hkv, D, ps, [130, 50], seed=16)
    n = small["k_pool"].shape[0]
    big = {k: v.cuda() for k, v in small.items()}
    for name in ("k_pool", "v_pool", "params"):
        t = torch.empty((num_pages,) + tuple(small[name].shape[1:]), dtype=small[name].dtype, device="cuda")
        t[num_pages - n:] = big[name]
        big[name] = t
    far = torch.where((small["table"] >= 0) & (small["table"] < n), small["table"] + (num_pages - n), small["table"])
    out, lse = gq.gqa_decode_paged_int4(big["q"], big["k_pool"], big["v_pool"], big["params"], far.cuda(), big["lens"])
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
    check(small, out.cpu(), lse.cpu())


def test_long_request(gq):
    d = make(2, 1, 8, 1, 64, 64, [200_000, 1], seed=17)
    out, lse = run(gq, d)
    check(d, out, lse)


def test_outputs_given_and_without_lse(gq):
    d = make(2, 1, 16, 2, 64, 16, [90, 200], seed=18)
    want = run(gq, d, num_splits=4)
    c = {n: t.cuda() for n, t in d.items()}
    a = (c["q"], c["k_pool"], c["v_pool"], c["params"], c["table"], c["lens"])
    out = torch.full_like(c["q"], 7.0)
    got, lse = gq.gqa_decode_paged_int4(*a, out=out, with_lse=False, num_splits=4)
    assert got is out and lse is None
    ws = torch.empty(max(256, gq.gqa_decode_paged_int4_workspace_bytes(2, 1, 16, 2, 64, 16, c["table"].shape[1], 4)),
                     dtype=torch.uint8, device="cuda")
    o2, l2 = gq.gqa_decode_paged_int4(*a, workspace=ws, num_splits=4)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(o2.cpu(), want[0]) and torch.equal(l2.cpu(), want[1])
    scaled, _ = gq.gqa_decode_paged_int4(*a, scale=1 / math.sqrt(64), num_splits=4)
    assert torch.equal(scaled.cpu(), want[0])


def test_other_streams_and_graphs(gq):
    """Two captured graphs and eager calls on streams of their own, run at once and again with new lengths: each call's
    partial results are its own."""
    ds = [make(4, 1, 32, 8, 128, 16, [600, 200, 0, 900], seed=19), make(3, 2, 16, 2, 64, 16, [1000, 10, 350], seed=20)]
    cs = [{n: t.cuda() for n, t in d.items()} for d in ds]
    call = lambda c, **kw: gq.gqa_decode_paged_int4(c["q"], c["k_pool"], c["v_pool"], c["params"], c["table"], c["lens"], **kw)  # noqa: E731
    want = [tuple(t.cpu() for t in call(c)) for c in cs]
    graphs, outs = [], []
    for c in cs:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(call(c))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for c, s in zip(cs, streams[2:]):
            eager.append(call(c, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o[0].cpu(), want[i][0]) and torch.equal(o[1].cpu(), want[i][1])
    for n, o in enumerate(eager):
        assert torch.equal(o[0].cpu(), want[n % 2][0]) and torch.equal(o[1].cpu(), want[n % 2][1])
    cs[0]["lens"].copy_(torch.tensor([10, 0, 0, 33], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    check({**ds[0], "lens": cs[0]["lens"].cpu()}, outs[0][0].cpu(), outs[0][1].cpu(), what="replayed with other lengths")


def test_allocated_outputs_of_a_given_stream(gq):
    """Outputs that a call on another stream allocates do not take memory that work queued on the current stream still
    reads."""
    d = make(64, 1, 32, 8, 128, 16, [40] * 64, seed=22)
    c = {n: t.cuda() for n, t in d.items()}
    args = (c["q"], c["k_pool"], c["v_pool"], c["params"], c["table"], c["lens"])
    want = gq.gqa_decode_paged_int4(*args)
    side = torch.cuda.Stream()
    busy = torch.zeros(256 << 20, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        x = torch.full_like(c["q"], 3.0)
        y = torch.empty_like(x)
        for _ in range(20):
            busy.add_(1.0)
        y.copy_(x)
        del x  # its memory may be handed out again, behind the copy on this stream
        got = gq.gqa_decode_paged_int4(*args, stream=side)
        torch.cuda.synchronize()
        assert torch.all(y == 3.0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("shape", [(2, 1, 8, 2, 128, 4, (300, 77)), (2, 2, 8, 8, 64, 12, (300, 5)), (1, 1, 8, 2, 128, 48, (1000,)),
                                   (3, 1, 40, 10, 128, 2, (90, 33, 64)), (2, 3, 12, 3, 64, 4, (200, 1)), (2, 1, 2, 1, 128, 32, (1500, 900)),
                                   (2, 1, 4, 2, 64, 6, (700, 31)), (1, 5, 10, 5, 64, 20, (444,))],
                         ids=lambda s: "b%d_sq%d_h%dx%d_d%d_ps%d" % s[:6])
@pytest.mark.parametrize("splits", [0, 1, 2, 700])
def test_page_sizes_and_head_counts(gq, shape, splits):
    d = make(*shape[:6], list(shape[6]), seed=100 + sum(shape[:6]))
    out, lse = run(gq, d, num_splits=splits)
    assert gq.gqa_device_status() == 0
    check(d, out, lse, what=f"{shape} splits {splits}")


@pytest.mark.parametrize("B", [255, 256, 257, 900])
def test_many_requests(gq, B):
    """Around and past the number of requests up to which each warp works out the schedule for itself; a third empty."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 70, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.33] = 0
    lens[-1] = 0
    d = make(B, 1, 8, 2, 64, 16, lens.tolist(), seed=B, ppr=5)
    for splits in (0, 1, 7):
        out, lse = run(gq, d, num_splits=splits)
        assert gq.gqa_device_status() == 0
        check(d, out, lse, what=f"splits {splits}")


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0] * 300, [1] + [0] * 40, [0] * 40 + [1], [33] * 40, [0, 32] * 20])
def test_empty_requests(gq, lens):
    d = make(len(lens), 2, 8, 2, 64, 16, lens, seed=3, ppr=3)
    for splits in (0, 1, 5):
        out, lse = run(gq, d, num_splits=splits)
        assert gq.gqa_device_status() == 0
        check(d, out, lse, what=f"splits {splits}")


@pytest.mark.parametrize("shape", [(1, 1, 8, 2, 64, 16, 500), (3, 1, 32, 8, 128, 16, 130), (2, 4, 32, 8, 128, 32, 64), (7, 2, 16, 1, 64, 8, 250),
                                   (170, 1, 16, 8, 128, 16, 90), (400, 1, 8, 2, 64, 16, 100), (700, 1, 3, 1, 64, 16, 70), (320, 3, 8, 2, 128, 16, 40),
                                   (1300, 1, 4, 2, 64, 5, 33), (5, 1, 8, 8, 64, 5, 96), (900, 1, 2, 1, 128, 4, 32),
                                   (4, 5, 8, 2, 128, 16, 60), (3, 1, 30, 1, 64, 16, 90), (200, 2, 24, 3, 128, 8, 30), (6, 8, 16, 4, 64, 3, 50)],
                         ids=lambda s: "b%d_sq%d_h%dx%d_d%d_ps%d_kv%d" % s)
def test_short_requests_whole(gq, shape):
    """Short requests, which the automatic choice leaves to one worker each: no workspace, as many requests as CTAs and
    more, and several of them after one another on a worker; the same bits at any number of requests around them."""
    B, Sq, Hq, Hkv, D, ps, hi = shape
    g = torch.Generator().manual_seed(sum(shape))
    lens = torch.randint(0, hi + 1, (B,), generator=g)
    lens[B // 2] = hi
    lens[torch.rand(B, generator=g) < 0.1] = 0
    d = make(B, Sq, Hq, Hkv, D, ps, lens.tolist(), seed=B, ppr=-(-hi // ps))
    ppr = d["table"].shape[1]
    assert gq.gqa_decode_paged_int4_workspace_bytes(B, Sq, Hq, Hkv, D, ps, ppr) == 0
    out, lse = run(gq, d)
    assert gq.gqa_device_status() == 0
    check(d, out, lse)
    n = gq.gqa_decode_paged_int4_num_splits(B, Sq, Hq, Hkv, D, ps, ppr)
    again = run(gq, d, num_splits=n)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    bad = {**d, "lens": d["lens"].clone()}
    bad["lens"][B - 1] = ppr * ps + 1
    run(gq, bad)
    assert gq.gqa_device_status() == 7


def test_largest_batch(gq):
    """65535 requests of 0 to 2 tokens, every result against 64 bits at once."""
    B, Hq, Hkv, D = 65535, 2, 1, 64
    g = torch.Generator(device="cuda").manual_seed(30)
    q = torch.randn(B, 1, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    k_pool, v_pool = (torch.randint(0, 256, (B, 2, Hkv, D // 2), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    params = (torch.rand(B, 2, Hkv, 4, generator=g, device="cuda") * torch.tensor([0.3, -4.0, 0.3, -4.0], device="cuda")).half()
    table = torch.randperm(B, generator=g, device="cuda").view(B, 1).to(torch.int32)
    lens = torch.randint(0, 3, (B,), generator=g, device="cuda", dtype=torch.int32)
    out, lse = gq.gqa_decode_paged_int4(q, k_pool, v_pool, params, table, lens)
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
    at = table[:, 0].long()
    k = ref.value_int4(k_pool[at], params[at][..., :2])[:, :, 0]
    v = ref.value_int4(v_pool[at], params[at][..., 2:])[:, :, 0]
    x = torch.einsum("bhd,btd->bht", q[:, 0].double(), k) / 8
    x = x.masked_fill(torch.arange(2, device="cuda") >= lens[:, None, None], -math.inf)
    some = lens > 0
    want = torch.einsum("bht,btd->bhd", torch.softmax(x[some], -1), v[some])
    assert torch.all(out[~some] == 0) and torch.all(torch.isneginf(lse[~some]))
    # scores of at most sum |q| (15 * 0.3 + 4) / 8 and V of at most 8.5, by the bounds of cache_ref.int4_bounds
    ds = (D + 8) * 2.0 ** -23 * 8.5 * q.double().abs().sum(-1).max() / 8
    assert torch.all((out[some][:, 0].double() - want).abs() <= 2 * ds * 8.5 + 2.0 ** -11 * 4.5 + 2.0 ** -8 * want.abs())
    assert torch.all((lse[some][..., 0].double() - torch.logsumexp(x[some], -1)).abs() <= ds + 2.0 ** -17)


@pytest.mark.parametrize("shape", [(3, 1, 32, 8, 128, 16), (2, 1, 8, 1, 64, 16), (2, 4, 16, 2, 128, 16), (2, 1, 6, 3, 64, 5)],
                         ids=["rings", "lanes", "16rows", "copies"])
def test_wait_that_runs_out(gq, shape):
    """A first stage that is never loaded: the wait for it ends at its limit, the call reports it, and the next call on
    the same stream is as it should be."""
    B = shape[0]
    d = make(*shape, [900] * B, seed=40)
    want = run(gq, d, num_splits=3)
    gq.gqa_set_wait_limit_ns(2_000_000)
    gq.gqa_debug_set_fault_mode(1)
    try:
        run(gq, d, num_splits=3)
        assert gq.gqa_device_status() == 6
    finally:
        gq.gqa_debug_set_fault_mode(0)
        gq.gqa_set_wait_limit_ns(0)
    again = run(gq, d, num_splits=3)
    assert gq.gqa_device_status() == 0
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])


@pytest.mark.parametrize("shape", [(3, 1, 8, 2, 64, 16), (2, 4, 16, 2, 128, 16), (160, 1, 16, 8, 128, 16), (2, 1, 6, 3, 64, 5)],
                         ids=["lanes", "16rows", "rings", "copies"])
def test_wait_that_runs_out_on_whole_requests(gq, shape):
    B = shape[0]
    d = make(*shape, [90] * B, seed=41)
    assert gq.gqa_decode_paged_int4_workspace_bytes(*shape, d["table"].shape[1]) == 0
    want = run(gq, d)
    gq.gqa_set_wait_limit_ns(2_000_000)
    gq.gqa_debug_set_fault_mode(1)
    try:
        run(gq, d)
        assert gq.gqa_device_status() == 6
    finally:
        gq.gqa_debug_set_fault_mode(0)
        gq.gqa_set_wait_limit_ns(0)
    again = run(gq, d)
    assert gq.gqa_device_status() == 0
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])


def test_weight_roundings_cancel_in_a_flat_value(gq):
    """V's codes all 8 with a zero of -8 scales: every element is 0 whatever the weights are.  A weight's fp16 rounding
    (2^-11) counts by the code's distance from 8, here 0; what is left are fp32 sums, within 2^-17 of the largest
    magnitude that they could hold, 15 scales and the zero."""
    for shape in ((3, 1, 32, 8, 128, 16, [4, 9, 300]), (2, 4, 16, 2, 64, 16, [70, 7])):
        d = make(*shape[:6], shape[6], seed=41)
        p = d["params"]
        d["v_pool"].fill_(0x88)
        p[..., 3] = -8 * p[..., 2]
        for splits in (0, 1, 4):
            out, lse = run(gq, d, num_splits=splits)
            for b, n in enumerate(shape[6]):
                at = ref.slots(d["table"][b], shape[5], range(n))
                top = float(p.flatten(0, 1)[at][..., 2].double().max())
                assert float(out[b].double().abs().max()) <= 2.0 ** -17 * 23 * top, (shape, splits, b)


def test_error_is_the_outputs_rounding(gq):
    """Root mean square error against 64 bits on N(0, 1) entries, beside that of the 64-bit result rounded to bf16.  A
    weight's rounding is at most 2^-11, 2^-11 / sqrt(3) in the mean square; a row of 128 normal values spans at most 7.5
    of its deviations, so that a code's distance from 8 is in the mean square at most 1.25 deviations (codes spread
    as the values do, their middle off by up to 0.75).  Against an output of one deviation's scale that is 1.25 x
    2.82e-4 = 3.53e-4 beside the rounding's 1.6e-3 or more: at most sqrt(1 + 0.22^2) = 1.024 of it."""
    d = make(4, 1, 32, 8, 128, 16, [300, 900, 2000, 500], seed=42)
    out, _ = run(gq, d)
    want = torch.zeros(out.shape, dtype=torch.float64)
    for b in range(4):
        n = int(d["lens"][b])
        at = ref.slots(d["table"][b], 16, range(n))
        p = d["params"].flatten(0, 1)[at]
        want[b, 0], _ = ref.attend(d["q"][b, 0], ref.value_int4(d["k_pool"].flatten(0, 1)[at], p[..., :2]),
                                   ref.value_int4(d["v_pool"].flatten(0, 1)[at], p[..., 2:]), n)
    own = float((out.double() - want).square().mean().sqrt())
    rounding = float((want.to(torch.bfloat16).double() - want).square().mean().sqrt())
    assert own <= 1.03 * rounding, (own, rounding)


@pytest.mark.parametrize("e,gain", [(18, 1.0), (21, 2.0 ** -9), (22, 2.0 ** -9), (23, 2.0 ** -9), (24, 1.0), (27, 1.0), (60, 1.0), (101, 1.0)])
def test_large_scores(gq, e, gain):
    """Scores of 2^e to 2^(e + 7) leave the weight to one token, however far below the next one is in fp32's steps.  The
    LSE is the largest score within (D + 8) 2^-23 of the magnitudes summed, the output that token's V, rounded to bf16
    (2^-8 of itself; the weight's rounding 2^-11 of 8 scales, fp32 sums 2^-17 of 15 scales and the zero).  (At 2^28 fp32
    has steps of 32, while an fp16 weight has room for 2^15 above 1: small V scales are where they could leave it.)"""
    D, n = 128, 200
    d = make(1, 1, 4, 2, D, 16, [n], seed=45, v_gain=gain)
    d["q"] = torch.randint(1, 4, d["q"].shape, generator=torch.Generator().manual_seed(46)).float().to(torch.bfloat16) * 2.0 ** e
    scale = 1.0
    out, lse = run(gq, d, scale=scale, num_splits=3)
    assert gq.gqa_device_status() == 0
    at = ref.slots(d["table"][0], 16, range(n))
    p = d["params"].flatten(0, 1)[at]
    k, v = ref.value_int4(d["k_pool"].flatten(0, 1)[at], p[..., :2]), ref.value_int4(d["v_pool"].flatten(0, 1)[at], p[..., 2:])
    mag = float((15 * p[..., 0].double() + p[..., 1].double().abs()).max())
    for h in range(4):
        q = d["q"][0, 0, h].double()
        s = k[:, h // 2] @ q * scale
        best = int(s.argmax())
        bound = (D + 8) * 2.0 ** -23 * mag * float(q.sum()) * scale
        second = float(s.sort().values[-2])
        assert float(s[best]) - second > 4 * bound  # the data: one token stands alone
        assert abs(float(lse[0, h, 0]) - float(s[best])) <= bound
        want = v[best, h // 2]
        vs = float(p[best, h // 2, 2])
        v_mag = 15 * vs + abs(float(p[best, h // 2, 3]))
        assert torch.all((out[0, 0, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * 8 * vs + 2.0 ** -17 * v_mag)


def test_queries_past_the_range_give_nan(gq):
    """A row with an infinite query element, or one whose scale times its largest element passes 2^104, is NaN where it
    sees a token and empty where it does not; finite rows up to there are right.  (All K values are below 0 or all
    above, so that no score is NaN by itself.)"""
    for sign in (1.0, -1.0):
        d = make(2, 2, 8, 2, 128, 16, [300, 1], seed=44)
        d["params"][..., 0] = 0.25
        d["params"][..., 1] = 0.5 if sign > 0 else -4.5
        d["q"] = d["q"].abs()
        clean = run(gq, d, num_splits=3)
        bad = {**d, "q": d["q"].clone()}
        bad["q"][0, 0, 3, 17] = float("inf")
        bad["q"][0, 1, 4, 9] = -float("inf")
        bad["q"][0, 1, 6, 9] = 3e38
        bad["q"][1, :, 2, 64] = float("inf")  # the first row of request 1 sees nothing
        out, lse = run(gq, bad, num_splits=3)
        hit = torch.zeros(2, 2, 8, dtype=torch.bool)
        hit[0, 0, 3] = hit[0, 1, 4] = hit[0, 1, 6] = hit[1, 1, 2] = True
        lse, was = lse.permute(0, 2, 1), clean[1].permute(0, 2, 1)
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], was[~hit])


@pytest.mark.parametrize("splits", [0, 1, 3, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_parameters_that_are_not_finite_give_nan(gq, which, value, splits):
    """A row that sees a token with a NaN or infinite parameter is NaN, its LSE too, whatever that token weighs: the
    query sums are positive and the token's K is -30, hundreds of nats below the others, unless its own K parameter is the
    one.  Early in the request (a step that all rows see whole) and in its last step; any number of workers."""
    d = make(2, 3, 16, 2, 128, 16, [900, 500], seed=43)
    d["q"] = d["q"].abs()
    at = lambda b, t: int(ref.slots(d["table"][b], 16, [t])[0])  # noqa: E731
    flat = d["params"].view(-1, 2, 4)
    places = [(0, 100, 0), (1, 499, 1)]  # seen by all rows of request 0; by the last one of request 1
    for b, t, g in places:
        flat[at(b, t), g, :2] = torch.tensor([0.0, -30.0]).half()
    clean = run(gq, d, num_splits=splits)
    assert torch.isfinite(clean[0]).all() and torch.isfinite(clean[1]).all()
    for b, t, g in places:
        flat[at(b, t), g, which] = value
    out, lse = run(gq, d, num_splits=splits)
    assert gq.gqa_device_status() == 0
    hit = torch.zeros(2, 3, 16, dtype=torch.bool)
    hit[0, :, :8] = hit[1, 2, 8:] = True
    lse, was = lse.permute(0, 2, 1), clean[1].permute(0, 2, 1)
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], was[~hit])
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()


@pytest.mark.parametrize("shape", [(1, 1, 24, 1, 64, 16, (3001,)), (2, 1, 20, 1, 128, 5, (900, 33)), (2, 1, 24, 1, 128, 16, (5000, 2047)),
                                   (1, 6, 3, 1, 64, 8, (2500,))],
                         ids=lambda s: "b%d_sq%d_h%dx%d_d%d_ps%d" % s[:6])
def test_five_groups_on_one_ring(gq, shape):
    """One KV head of 17 to 24 rows, 8 rows a warp: three warps a group, five groups that take turns at one ring of 15
    stages, and one warp without work; shares of all steps (there is a workspace)."""
    d = make(*shape[:6], list(shape[6]), seed=200 + sum(shape[:6]))
    assert gq.gqa_decode_paged_int4_workspace_bytes(*shape[:6], d["table"].shape[1]) > 0
    first = run(gq, d)
    assert gq.gqa_device_status() == 0
    check(d, *first, what=str(shape))
    for _ in range(3):
        again = run(gq, d)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("D", [64, 128])
def test_least_scores(gq, D):
    """All K at fp16's lowest value and queries as large as they may be: scores near fp32's lowest are scores, past the
    limit NaN, never a row without tokens.  Queries of zero take any scale.  (Workers' results are joined by their LSEs,
    which at -65504 x 64 and below have steps of 0.25 and more: how many of the 100 equal tokens a worker had is lost in
    them, by any factor from there on, so that several workers give some mean of the tokens.)"""
    d = make(1, 1, 8, 2, D, 16, [100], seed=47)
    d["params"][..., 0] = 0.0
    d["params"][..., 1] = -65504.0
    at = ref.slots(d["table"][0], 16, range(100))
    each = ref.value_int4(d["v_pool"].flatten(0, 1)[at], d["params"].flatten(0, 1)[at][..., 2:])
    v = each.mean(0)  # equal weights
    tops = [2.0 ** 60, 1.5 * 2.0 ** 103, 2.0 ** 104, 2.0 ** 120, 2.0 ** 127, 0.0, 1.0, 2.0 ** 102]
    d["q"] = torch.tensor(tops).view(1, 1, 8, 1).expand(1, 1, 8, D).to(torch.bfloat16).contiguous()
    for splits in (0, 3):
        out, lse = run(gq, d, scale=1.0, num_splits=splits)
        for h, x in enumerate(tops):
            if x >= 2.0 ** 104:
                assert torch.isnan(out[0, 0, h]).all() and torch.isnan(lse[0, h, 0]), h
                continue
            s = -65504.0 * D * x + math.log(100)
            # 64 fp32 terms and their scale; V: 15 scales and the zero as in check()
            assert abs(float(lse[0, h, 0]) - s) <= (D + 8) * 2.0 ** -23 * abs(s) + 2.0 ** -17, h
            want = v[h // 4]
            if splits > 1 and x > 0:
                low, high = each[:, h // 4].amin(0), each[:, h // 4].amax(0)
                want = torch.minimum(torch.maximum(out[0, 0, h].double(), low), high)
            assert torch.all((out[0, 0, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * 3 + 2.0 ** -17 * 10), h
    d["q"].zero_()
    for scale in (2.0 ** 60, 2.0 ** 120):
        out, lse = run(gq, d, scale=scale)
        assert torch.all((lse.double() - math.log(100)).abs() <= 2.0 ** -17)
        assert torch.all((out[0, 0].double().view(2, 4, D) - v[:, None]).abs() <= 2.0 ** -8 * v.abs()[:, None] + 2.0 ** -11 * 3 + 2.0 ** -17 * 10)
