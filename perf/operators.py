"""Cases of the paged cache's operators: appending to the cache, decoding over a cache held in 4 bits, and gathering
from the cache into dense tensors.

Each case is a dict of plain values; ``prepare`` makes its inputs, ``run`` makes one pass through the operator (the
library's entry points where ``own`` is true, elementary torch operations in fp32 where it is false), ``exact`` gives
the same outputs from the definitions in 64 bits.

The cache, as in the paged decode calls: K and V pools [num_pages, page_size, Hkv, D] (bf16, uint8 E4M3FN codes or
int8 codes; 4-bit pools hold D/2 bytes a row, element 2i in the low half of byte i), a page table [B, pages_per_req],
seq_lens [B].  A 4-bit pool keeps fp16 [num_pages, page_size, Hkv, 4] beside it: K scale, K zero, V scale, V zero of
every token and head; a code u (0..15) stands for u * scale + zero.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
F16_MAX = 65504.0


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # -- decode over a 4-bit cache
        # the serving shape of the benchmark's paged workloads: 32 requests of 16K-32K tokens
        dict(name="attend_b32_h64x8_d128_kv32k_ps16", op="attend", B=32, Sq=1, Hq=64, Hkv=8, D=128, ps=16, lo=16384, hi=32768),
        # one long document, answered alone: the split over the long axis, pages of 64
        dict(name="attend_b1_h64x8_d128_kv128k_ps64", op="attend", B=1, Sq=1, Hq=64, Hkv=8, D=128, ps=64, lo=131072, hi=131072),
        # a full batch of short chats, some slots of the batch empty
        dict(name="attend_b256_h32x8_d128_kv1k_ps16", op="attend", B=256, Sq=1, Hq=32, Hkv=8, D=128, ps=16, lo=0, hi=1024),
        # four draft tokens verified in one call, 16 rows per KV head
        dict(name="attend_b16_h32x8_d128_sq4_kv8k_ps32", op="attend", B=16, Sq=4, Hq=32, Hkv=8, D=128, ps=32, lo=5, hi=8192),
        # one KV head for all query heads, head size 64
        dict(name="attend_b8_h32x1_d64_kv8k_ps16", op="attend", B=8, Sq=1, Hq=32, Hkv=1, D=64, ps=16, lo=3000, hi=8192),
        # the smallest call: a small model's single request, an odd page size; latency counts
        dict(name="attend_b1_h8x2_d64_kv1k_ps5", op="attend", B=1, Sq=1, Hq=8, Hkv=2, D=64, ps=5, lo=1000, hi=1000),
        # -- appending to the cache, the rotation applied on the way (queries rotated in the same call)
        # one decode step of a batch, bf16 cache
        dict(name="append_bf16_b32_h64x8_d128_step", op="append", kv="bf16", B=32, n_lo=1, n_hi=1, Hq=64, Hkv=8, D=128, ps=16, lo=1, hi=512, rot=128, inter=False),
        # one decode step of a large batch into the 4-bit cache; the new entries read back
        dict(name="append_int4_b256_h32x8_d128_step", op="append", kv="int4", B=256, n_lo=1, n_hi=1, Hq=32, Hkv=8, D=128, ps=16, lo=1, hi=256, rot=128, inter=False),
        # a batch of prompts of ragged lengths into the FP8 cache
        dict(name="append_fp8_b16_h64x8_d128_prompts", op="append", kv="fp8", B=16, n_lo=1, n_hi=4096, Hq=64, Hkv=8, D=128, ps=16, lo=4096, hi=4096, rot=128, inter=False),
        # prompts into the 4-bit cache, head size 64, neighbouring pairs rotated in the first half of the head only;
        # the entries read back dense, as prompt attention wants them
        dict(name="append_int4_b24_h16x4_d64_prompts", op="append", kv="int4", B=24, n_lo=1, n_hi=2000, Hq=16, Hkv=4, D=64, ps=16, lo=2048, hi=4096, rot=32, inter=True),
        # -- gathering requests from the cache into dense bf16
        # the cached prefixes of a few requests, for a prompt chunk's dense attention
        dict(name="gather_int4_b8_h8_d128_kv16k", op="gather", kv="int4", B=8, Hkv=8, D=128, ps=16, lo=9000, hi=16384, part=False),
        # the newest part of each of many int8 requests, short
        dict(name="gather_int8_b64_h4_d64_kv512_ps7", op="gather", kv="int8", B=64, Hkv=4, D=64, ps=7, lo=0, hi=512, part=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "gather"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    ps = rng.choice([1, 5, 8, 16, 16, 16, 24, 32, 64, 128])
    if op == "attend":
        group, Sq = rng.choice([(1, 1), (2, 1), (3, 1), (4, 1), (4, 2), (4, 4), (5, 3), (8, 1), (8, 2), (16, 1), (32, 1)])
        hi = _log_int(rng, Sq, 131072)
        B = _log_int(rng, 1, max(1, min(256, (1 << 29) // (hi * Hkv * D))))
        return dict(op=op, B=B, Sq=Sq, Hq=group * Hkv, Hkv=Hkv, D=D, ps=ps, lo=rng.choice([0, Sq, (hi + 1) // 2, hi]), hi=hi)
    kv = rng.choice(["bf16", "fp8", "int8", "int4", "int4"])
    if op == "append":
        n_hi = rng.choice([1, 1, _log_int(rng, 2, 4096)])
        B = _log_int(rng, 1, max(1, min(256, (1 << 15) // n_hi)))
        hi = n_hi + rng.randint(0, 512)
        inter = rng.random() < 0.4
        return dict(op=op, kv=kv, B=B, n_lo=rng.choice([0, 1, n_hi]) if n_hi > 1 else 1, n_hi=n_hi, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]),
                    Hkv=Hkv, D=D, ps=ps, lo=n_hi, hi=hi, rot=rng.choice([16, D // 2, D, D]), inter=inter)
    hi = _log_int(rng, 1, 32768)
    B = _log_int(rng, 1, max(1, min(256, (1 << 27) // (hi * Hkv * D))))
    return dict(op=op, kv=kv, B=B, Hkv=Hkv, D=D, ps=ps, lo=rng.choice([0, 1, hi]), hi=hi, part=rng.random() < 0.5)


def _lens(c):
    """The requests' lengths, and the tokens that each brings (append) or that are asked for (gather, its newest): the
    same for every seed, so that a case's work is its own."""
    r = random.Random("%s %s %s %s %s" % (c["op"], c["B"], c["lo"], c["hi"], c["ps"]))
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    longest = r.randrange(c["B"])
    lens[longest] = c["hi"]
    if c["op"] == "append":
        new = [min(n, r.randint(c["n_lo"], c["n_hi"])) for n in lens]
        new[longest] = max(1, new[longest])
    elif c["op"] == "gather" and c["part"]:
        new = [r.randint(min(1, n), n) for n in lens]
    else:
        new = list(lens)
    return lens, new


# ------------------------------------------------------------------------------------------------ inputs
def _encode(x, kv, scale):
    """Codes of fp32 x [..., D] and, for 4 bits, each row's fp16 (scale, zero)."""
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    if kv in ("fp8", "int8"):
        y = x * float(torch.tensor(1.0) / torch.tensor(scale, dtype=torch.float32))
        if kv == "fp8":
            return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), None
        return y.round().clamp(-127, 127).to(torch.int8), None
    x = x.clamp(-F16_MAX, F16_MAX)
    zero = x.amin(-1, keepdim=True).half()
    step = ((x.amax(-1, keepdim=True) - zero.float()) * (1.0 / 15.0)).clamp(min=0).half()
    inv = torch.where(step > 0, 1.0 / step.float(), 0.0)
    u = ((x - zero.float()) * inv).round().clamp(0, 15).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), torch.cat([step, zero], -1)


def _pool(c, num_pages, gen, dev):
    """Pools of a cache in use: quantised N(0, 1) with a spread of its own for each channel, as keys and values have."""
    kv, Hkv, D, ps = c.get("kv", "int4"), c["Hkv"], c["D"], c["ps"]
    scale = 6.0 / {"bf16": 6.0, "fp8": E4M3_MAX, "int8": 127.0, "int4": 6.0}[kv]
    width = D // 2 if kv == "int4" else D
    kind = {"bf16": torch.bfloat16, "fp8": torch.uint8, "int8": torch.int8, "int4": torch.uint8}[kv]
    pools = [torch.empty(num_pages, ps, Hkv, width, dtype=kind, device=dev) for _ in range(2)]
    params = torch.empty(num_pages, ps, Hkv, 4, dtype=torch.float16, device=dev) if kv == "int4" else None
    chunk = max(1, (1 << 27) // (ps * Hkv * D))
    for i, pool in enumerate(pools):
        spread = 0.5 + torch.rand(Hkv, D, generator=gen, device=dev)
        for a in range(0, num_pages, chunk):
            b = min(num_pages, a + chunk)
            pool[a:b], p = _encode(torch.randn(b - a, ps, Hkv, D, generator=gen, device=dev) * spread, kv, scale)
            if p is not None:
                params[a:b, ..., 2 * i:2 * i + 2] = p
    return pools[0], pools[1], params, scale


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _lens(c)
    B, ps, D, Hkv = c["B"], c["ps"], c["D"], c["Hkv"]
    ppr = max(1, -(-max(c["hi"], 1) // ps))
    num_pages = B * ppr + 3
    s = dict(c=c, lens=torch.tensor(lens, dtype=torch.int32, device=dev), new=torch.tensor(new, dtype=torch.int32, device=dev))
    s["table"] = torch.randperm(num_pages, generator=gen, device=dev)[:B * ppr].view(B, ppr).to(torch.int32).contiguous()
    s["k_pool"], s["v_pool"], s["params"], s["scale"] = _pool(c, num_pages, gen, dev)
    if c["op"] == "attend":
        s["q"] = torch.randn(B, c["Sq"], c["Hq"], D, generator=gen, device=dev).to(torch.bfloat16)
        return s
    if c["op"] == "gather":
        s["starts"] = s["lens"] - s["new"] if c["part"] else None
        s["k_out"], s["v_out"] = (torch.zeros(B, max(1, max(new)), Hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        return s
    T = sum(new)
    # q, k and v as a fused projection leaves them: one row a token, padded behind the last request
    qkv = torch.randn(T + 2, c["Hq"] + 2 * Hkv, D, generator=gen, device=dev).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = qkv[:, :c["Hq"]], qkv[:, c["Hq"]:c["Hq"] + Hkv], qkv[:, c["Hq"] + Hkv:]
    s["cu"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
    s["T"] = T
    s["q_out"] = torch.zeros(T + 2, c["Hq"], D, dtype=torch.bfloat16, device=dev)
    # the rotation's angles in 64 bits, kept as fp32 cosines and sines by a user's program
    freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
    angle = torch.arange(max(c["hi"], 1), dtype=torch.float64, device=dev)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float().contiguous()
    s["starts"] = s["lens"] - s["new"]
    if c["kv"] in ("int8", "int4"):
        s["k_back"], s["v_back"] = (torch.zeros(B, max(1, max(new)), Hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _decode(codes, kv, scale, params):
    """fp32 values of gathered codes [..., Hkv, D or D/2]; params [..., Hkv, 2] for 4 bits."""
    if kv == "bf16":
        return codes.float()
    if kv == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scale
    if kv == "int8":
        return codes.float() * scale
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return u * params[..., 0:1].float() + params[..., 1:2].float()


def _rows(s, pos):
    """Pool rows of the positions pos [B, n]."""
    ps = s["c"]["ps"]
    pos = pos.clamp(0, s["table"].shape[1] * ps - 1)
    return s["table"].gather(1, pos // ps).long() * ps + pos % ps


def _read(s, rows):
    """fp32 K and V at pool rows [B, n]: [B, n, Hkv, D]."""
    kv, p = s["c"].get("kv", "int4"), s["params"]
    p = None if p is None else p.flatten(0, 1)[rows]
    return tuple(_decode(s[n].flatten(0, 1)[rows], kv, s["scale"], None if p is None else p[..., 2 * i:2 * i + 2])
                 for i, n in enumerate(("k_pool", "v_pool")))


def _plain_attend(s):
    c, q = s["c"], s["q"].float()
    B, Sq, Hq, D = q.shape
    Hkv, hi = c["Hkv"], max(c["hi"], 1)
    at = torch.arange(hi, device=q.device)
    k, v = _read(s, _rows(s, at.expand(B, hi)))
    q = q.view(B, Sq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)  # rows: head of the group, then query row
    x = (q @ k.permute(0, 2, 3, 1)).view(B, Hkv, Hq // Hkv, Sq, hi) * (1.0 / math.sqrt(D))
    seen = at <= (s["lens"][:, None] - Sq + torch.arange(Sq, device=q.device))[..., None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).view(B, Hkv, Hq // Hkv, Sq, D) / total.clamp(min=1e-37)
    lse = (total.log() + top)[..., 0]
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D).to(torch.bfloat16), "lse": lse.reshape(B, Hq, Sq)}


def _rotate(x, cos, sin, rot, inter):
    """x [T, H, D] fp32, cos and sin [T, rot/2]: the first rot elements of each head rotated in pairs (neighbours, or i
    and i + rot/2)."""
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _new_positions(s):
    """(request, position) of each appended token."""
    t = torch.arange(s["T"], device=s["cu"].device)
    req = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return req, s["starts"][req].long() + t - s["cu"][req].long()


def _plain_append(s):
    c, T = s["c"], s["T"]
    req, pos = _new_positions(s)
    cos, sin = s["cos_sin"][pos].chunk(2, -1)
    turn = lambda x: _rotate(x[:T].float(), cos, sin, c["rot"], c["inter"])  # noqa: E731
    s["q_out"][:T] = turn(s["q"]).to(torch.bfloat16)
    row = s["table"][req, pos // c["ps"]].long() * c["ps"] + pos % c["ps"]
    for i, (name, x) in enumerate((("k_pool", turn(s["k"])), ("v_pool", s["v"][:T].float()))):
        codes, p = _encode(x, c["kv"], s["scale"])
        s[name].flatten(0, 1)[row] = codes
        if p is not None:
            s["params"].flatten(0, 1)[..., 2 * i:2 * i + 2][row] = p


def _plain_gather(s, k_out, v_out):
    n = k_out.shape[1]
    at = torch.arange(n, device=k_out.device).expand(k_out.shape[0], n)
    first = 0 if s["starts"] is None else s["starts"][:, None].long()
    there = (at < s["new"][:, None])[..., None, None]
    for out, x in zip((k_out, v_out), _read(s, _rows(s, at + first))):
        out.copy_(torch.where(there, x.to(torch.bfloat16), out))


def run(state):
    s, c = state, state["c"]
    if own:
        import gqa_decode_attention_gb300 as gq
    if c["op"] == "attend":
        if own:
            out, lse = gq.gqa_decode_paged_int4(s["q"], s["k_pool"], s["v_pool"], s["params"], s["table"], s["lens"])
            return {"out": out, "lse": lse}
        return _plain_attend(s)
    scales = {"k_scale": s["scale"], "v_scale": s["scale"]}
    if c["op"] == "gather":
        if own:
            gq.gqa_paged_gather(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["k_out"], s["v_out"], starts=s["starts"],
                                kv_params=s["params"], **scales)
        else:
            _plain_gather(s, s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if own:
        gq.gqa_paged_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["lens"], cu_tokens=s["cu"], q=s["q"],
                            q_out=s["q_out"], cos_sin=s["cos_sin"], interleaved=c["inter"], kv_params=s["params"], **scales)
    else:
        _plain_append(s)
    if c["kv"] in ("int8", "int4"):  # the values that the new codes stand for, read back from the cache
        if own:
            gq.gqa_paged_gather(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["k_back"], s["v_back"], starts=s["starts"],
                                kv_params=s["params"], **scales)
        else:
            _plain_gather(s, s["k_back"], s["v_back"])
        return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}
    kind = torch.float8_e4m3fn if c["kv"] == "fp8" else torch.bfloat16
    return {"q": s["q_out"], "k": s["k_pool"].view(kind), "v": s["v_pool"].view(kind)}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    lens, new = _lens(c)
    kv = c.get("kv", "int4")
    entry = 2 * c["Hkv"] * (c["D"] // 2 + 4 if kv == "int4" else c["D"] * (2 if kv == "bf16" else 1))  # a token's K and V
    dense = 2 * c["Hkv"] * c["D"] * 2
    pages = 4 * sum(-(-n // c["ps"]) for n in lens)
    if c["op"] == "attend":
        rows = c["B"] * c["Sq"] * c["Hq"]
        return {"bytes": sum(lens) * entry + pages + rows * (4 * c["D"] + 4) + 4 * c["B"], "flops": 4 * sum(lens) * c["Sq"] * c["Hq"] * c["D"]}
    if c["op"] == "gather":
        return {"bytes": sum(new) * (entry + dense) + 4 * sum(-(-n // c["ps"]) for n in new) + 8 * c["B"], "flops": 2 * sum(new) * c["Hkv"] * c["D"]}
    T = sum(new)
    q = 2 * 2 * c["Hq"] * c["D"]
    back = entry + dense if kv in ("int8", "int4") else 0  # the read-back reads the entries and writes them dense
    return {"bytes": T * (q + dense + entry + back + 4 * c["rot"]) + 4 * sum(-(-n // c["ps"]) for n in new) + 8 * c["B"],
            "flops": T * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}


# ------------------------------------------------------------------------------------------------ 64 bits
def _slots(s, b, pos):
    """Pool rows of request b's positions."""
    pos = torch.as_tensor(pos, device=s["table"].device)
    return s["table"][b].long()[torch.div(pos, s["c"]["ps"], rounding_mode="floor")] * s["c"]["ps"] + pos % s["c"]["ps"]


def _value64(s, which, rows):
    """Values in 64 bits of the pool's entries at `rows`: [n, Hkv, D]."""
    kv = s["c"].get("kv", "int4")
    x = s["%s_pool" % which].flatten(0, 1)[rows]
    if kv == "int4":
        p = s["params"].flatten(0, 1)[rows].double()
        i = 0 if which == "k" else 2
        y = torch.empty(*x.shape[:-1], 2 * x.shape[-1], dtype=torch.float64, device=x.device)
        y[..., 0::2] = (x % 16).double()
        y[..., 1::2] = torch.div(x, 16, rounding_mode="floor").double()
        return y * p[..., i, None] + p[..., i + 1, None]
    if kv == "fp8":
        return x.view(torch.float8_e4m3fn).double() * s["scale"]
    return x.double() * (s["scale"] if kv == "int8" else 1.0)


def _store64(s, x, which, rows):
    """x [n, Hkv, D] in 64 bits as the cache holds it, and back: what a reader of the entries sees."""
    kv, scale = s["c"]["kv"], s["scale"]
    if kv == "bf16":
        return x
    if kv == "fp8":
        return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
    if kv == "int8":
        return (x / scale).round().clamp(-127, 127) * scale
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    zero = low.half().double()
    step = ((high - zero) / 15).half().double()
    return ((x - zero) / step).round().clamp(0, 15) * step + zero


def exact(case, seed):
    c, s = case, prepare(case, seed)
    lens, new = _lens(c)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    if c["op"] == "attend":
        Sq, Hq = c["Sq"], c["Hq"]
        out = torch.zeros(B, Sq, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            if lens[b] == 0:
                continue
            rows = _slots(s, b, list(range(lens[b])))
            k, v = _value64(s, "k", rows), _value64(s, "v", rows)
            for i in range(Sq):
                n = lens[b] - Sq + i + 1
                if n <= 0:
                    continue
                x = torch.einsum("hgd,thd->hgt", s["q"][b, i].double().view(Hkv, Hq // Hkv, D), k[:n]) / math.sqrt(D)
                lse[b, :, i] = torch.logsumexp(x, -1).flatten()
                out[b, i] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v[:n]).reshape(Hq, D)
        return {"out": out, "lse": lse}
    if c["op"] == "gather":
        k, v = (torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        for b in range(B):
            if new[b]:
                rows = _slots(s, b, list(range(lens[b] - new[b] if c["part"] else 0, lens[b])))
                k[b, :new[b]], v[b, :new[b]] = _value64(s, "k", rows), _value64(s, "v", rows)
        return {"k": k, "v": v}
    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
    back = c["kv"] in ("int8", "int4")
    if back:
        k, v = (torch.zeros(s["k_back"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    else:
        kind = torch.float8_e4m3fn if c["kv"] == "fp8" else torch.bfloat16
        k, v = (s[n].view(kind).double().flatten(0, 1) for n in ("k_pool", "v_pool"))
    half, t = c["rot"] // 2, 0
    first = torch.arange(half, device="cuda") * (2 if c["inter"] else 1)
    second = first + (1 if c["inter"] else half)
    for b in range(B):
        if not new[b]:
            continue
        at = list(range(lens[b] - new[b], lens[b]))
        table = s["cos_sin"][at[0]:at[-1] + 1].double()[:, None]
        turned = []
        for name in ("q", "k"):
            x = s[name][t:t + new[b]].double()
            y = x.clone()
            y[..., first] = x[..., first] * table[..., :half] - x[..., second] * table[..., half:]
            y[..., second] = x[..., second] * table[..., :half] + x[..., first] * table[..., half:]
            turned.append(y)
        q[t:t + new[b]] = turned[0]
        rows = _slots(s, b, at)
        for to, which, x in ((k, "k", turned[1]), (v, "v", s["v"][t:t + new[b]].double())):
            x = _store64(s, x, which, rows)
            if back:
                to[b, :new[b]] = x
            else:
                to[rows] = x
        t += new[b]
    return {"q": q, "k": k if back else k.view(s["k_pool"].shape), "v": v if back else v.view(s["v_pool"].shape)}
