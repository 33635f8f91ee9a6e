"""Cases of prompt attention: attention over packed prompts, attention of new tokens over a paged cache, and the merge of
attentions over parts of the keys.

Each case is a dict of plain values; ``prepare`` makes its inputs, ``run`` makes one pass through the operator (the
library's entry points where ``own`` is true, elementary torch operations in fp32 where it is false), ``exact`` gives
the same outputs from the definitions in 64 bits.

Packed tokens: sequence b owns the rows cu[b] .. cu[b+1]-1 of q (and of k and v, whose offsets may be others); row i of
n over L keys sees the keys j <= L - n + i, or all of them where ``causal`` is false.  Query head h reads KV head
h // (Hq / Hkv).  The cache is that of the paged calls: pools [num_pages, page_size, Hkv, D] (bf16, uint8 E4M3FN codes
or int8 codes; 4-bit pools hold D/2 bytes a row beside fp16 [num_pages, page_size, Hkv, 4] of K scale, K zero, V scale
and V zero), a page table [B, pages_per_req], and seq_lens [B], which count the new tokens too.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EXACT_FLOPS = 4e12  # about four seconds in 64 bits


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # -- prompts, packed one after the other
        # one long document
        dict(name="prompt_b1_h64x8_d128_n16k", op="prompt", B=1, lo=16384, hi=16384, Hq=64, Hkv=8, D=128, Dv=128, x_lo=0, x_hi=0, causal=True),
        # a batch of prompts of ragged lengths
        dict(name="prompt_b16_h64x8_d128_n4k", op="prompt", B=16, lo=1, hi=4096, Hq=64, Hkv=8, D=128, Dv=128, x_lo=0, x_hi=0, causal=True),
        # a full batch of short chats
        dict(name="prompt_b256_h32x8_d128_n256", op="prompt", B=256, lo=1, hi=256, Hq=32, Hkv=8, D=128, Dv=128, x_lo=0, x_hi=0, causal=True),
        # the smallest call: a small model's one short prompt; latency counts
        dict(name="prompt_b1_h8x2_d64_n17", op="prompt", B=1, lo=17, hi=17, Hq=8, Hkv=2, D=64, Dv=64, x_lo=0, x_hi=0, causal=True),
        # -- new tokens of requests over the paged cache that holds them
        # a chunk of a long document's prompt, its last
        dict(name="chunk_bf16_b1_h64x8_d128_n2k_kv128k_ps64", op="chunk", kv="bf16", B=1, ones=0, n_lo=2048, n_hi=2048, lo=131072, hi=131072, Hq=64, Hkv=8, D=128, ps=64, causal=True),
        # a serving step: most requests decode one token, a few bring a piece of their prompt
        dict(name="chunk_fp8_b32_h64x8_d128_mixed_kv32k_ps16", op="chunk", kv="fp8", B=32, ones=28, n_lo=100, n_hi=512, lo=1024, hi=32768, Hq=64, Hkv=8, D=128, ps=16, causal=True),
        # eight draft tokens a request checked in one call, more rows than the paged decode calls take
        dict(name="chunk_bf16_b16_h64x8_d128_n8_kv32k_ps16", op="chunk", kv="bf16", B=16, ones=0, n_lo=8, n_hi=8, lo=8192, hi=32768, Hq=64, Hkv=8, D=128, ps=16, causal=True),
        # follow-up questions over a 4-bit cache
        dict(name="chunk_int4_b8_h32x8_d128_n300_kv16k_ps16", op="chunk", kv="int4", B=8, ones=0, n_lo=1, n_hi=300, lo=2048, hi=16384, Hq=32, Hkv=8, D=128, ps=16, causal=True),
        # a small model's batch over an int8 cache with an odd page size
        dict(name="chunk_int8_b24_h16x4_d64_n256_kv4k_ps7", op="chunk", kv="int8", B=24, ones=0, n_lo=1, n_hi=256, lo=256, hi=4096, Hq=16, Hkv=4, D=64, ps=7, causal=True),
        # the smallest call: a few draft tokens of a small model's single request; latency counts
        dict(name="chunk_bf16_b1_h8x2_d64_n5_kv1k_ps5", op="chunk", kv="bf16", B=1, ones=0, n_lo=5, n_hi=5, lo=1000, hi=1000, Hq=8, Hkv=2, D=64, ps=5, causal=True),
        # -- attentions over parts of the keys made one
        # a long prompt's cached prefix and its own tokens
        dict(name="merge_2_t16k_h64_d128", op="merge", N=2, T=16384, H=64, D=128),
        # a decode step's batch: a prefix that all share, a document, the request's own tokens
        dict(name="merge_3_t32_h64_d128", op="merge", N=3, T=32, H=64, D=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "chunk", "chunk", "chunk", "merge"])
    if op == "merge":
        T, H, D = _log_int(rng, 1, 16384), rng.choice([1, 6, 8, 16, 32, 64]), rng.choice([64, 128])
        return dict(op=op, N=rng.choice([2, 2, 3, 5, 8] if T <= 4096 else [2]), T=T, H=H, D=D)
    Hkv = rng.choice([1, 2, 3, 4, 8, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 12, 16, 32])
    causal = rng.random() < 0.8
    if op == "prompt":
        D, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
        hi = _log_int(rng, 1, 16384)
        # as much as the largest listed prompt at most, and 2^22 rows of queries
        most = min(256, 64 * (1 << 28) // (Hq * hi * hi), (1 << 22) // (Hq * hi))
        B = _log_int(rng, 1, max(1, most))
        while Hq * hi * hi * B > 64 << 28:
            hi -= hi // 4
        x_lo, x_hi = rng.choice([(0, 0), (0, 0), (0, 0), (0, 700), (-9, 9)])  # keys beside a sequence's own
        return dict(op=op, B=B, lo=rng.choice([0, 1, (hi + 1) // 2, hi]), hi=hi, Hq=Hq, Hkv=Hkv, D=D, Dv=Dv, x_lo=x_lo,
                    x_hi=x_hi, causal=causal)
    D = rng.choice([64, 128, 128])
    n_hi = rng.choice([1, _log_int(rng, 2, 2048), _log_int(rng, 2, 2048)])
    hi = _log_int(rng, n_hi, 65536)
    most = min(256, (64 << 27) // (Hq * n_hi * hi), (1 << 20) // (Hkv * hi) + 1, (1 << 20) // (Hq * n_hi))
    B = _log_int(rng, 1, max(1, most))
    return dict(op=op, kv=rng.choice(["bf16", "bf16", "fp8", "int8", "int4"]), B=B, ones=rng.choice([0, 0, B // 2]),
                n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, lo=rng.choice([0, min(n_hi, hi), (hi + 1) // 2, hi]), hi=hi, Hq=Hq,
                Hkv=Hkv, D=D, ps=rng.choice([1, 5, 8, 16, 16, 16, 24, 32, 64, 128]), causal=causal)


def _lens(c):
    """Query rows and keys of each sequence: the same for every seed, so that a case's work is its own."""
    r = random.Random("%s %s %s %s %s" % (c["op"], c["B"], c["lo"], c["hi"], c["Hq"]))
    if c["op"] == "prompt":
        n = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
        n[r.randrange(c["B"])] = c["hi"]
        return n, [max(0, x + r.randint(c["x_lo"], c["x_hi"])) for x in n]
    n = [1 if b < c["ones"] else r.randint(c["n_lo"], c["n_hi"]) for b in range(c["B"])]
    n[-1] = c["n_hi"]
    L = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    L[-1] = c["hi"]
    return n, L


def _pairs(c):
    """Pairs of a query row and a key that it sees."""
    total = 0
    for n, L in zip(*_lens(c)):
        if not c["causal"]:
            total += n * L
        elif n and L:
            seen = min(n, L)  # rows that see a key: the last sees L, each before it one less
            total += seen * L - seen * (seen - 1) // 2
    return total


# ------------------------------------------------------------------------------------------------ inputs
def _encode(x, kv, scale):
    """Codes of fp32 x [..., D] and, for 4 bits, each row's fp16 (scale, zero)."""
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    if kv == "fp8":
        return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), None
    if kv == "int8":
        return (x / scale).round().clamp(-127, 127).to(torch.int8), None
    zero = x.amin(-1, keepdim=True).half()
    step = ((x.amax(-1, keepdim=True) - zero.float()) / 15).clamp(min=0).half()
    u = ((x - zero.float()) / step.float().clamp(min=2.0 ** -24)).round().clamp(0, 15).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), torch.cat([step, zero], -1)


def _pool(c, num_pages, gen, dev):
    """Pools of a cache in use: quantised N(0, 1) with a spread of its own for each channel, as keys and values have."""
    kv, Hkv, D, ps = c["kv"], c["Hkv"], c["D"], c["ps"]
    scale = 6.0 / {"bf16": 6.0, "fp8": E4M3_MAX, "int8": 127.0, "int4": 6.0}[kv]
    kind = {"bf16": torch.bfloat16, "fp8": torch.uint8, "int8": torch.int8, "int4": torch.uint8}[kv]
    pools = [torch.empty(num_pages, ps, Hkv, D // 2 if kv == "int4" else D, dtype=kind, device=dev) for _ in range(2)]
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


def _offsets(n, dev):
    return torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    s = dict(c=c)
    if c["op"] == "merge":
        # attentions over parts of different lengths; a part may hold no key that a row sees
        s["lses"] = [normal(c["T"], c["H"]) + float(i) for i in range(c["N"])]
        s["outs"] = [normal(c["T"], c["H"], c["D"]) for _ in range(c["N"])]
        for i in range(c["N"]):
            none = torch.rand(c["T"], c["H"], generator=gen, device=dev) < 0.05
            s["lses"][i][none] = -math.inf
            s["outs"][i] = s["outs"][i].masked_fill(none[..., None], 0.0).to(torch.bfloat16)
        return s
    n, L = _lens(c)
    Hq, Hkv, D, Dv = c["Hq"], c["Hkv"], c["D"], c.get("Dv", c["D"])
    T = sum(n)
    s["n"], s["L"], s["cu"] = n, L, _offsets(n, dev)
    # rows behind the last sequence, as a padded batch has them
    s["out"] = torch.zeros(T + 2, Hq, Dv, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(T + 2, Hq, device=dev)
    if c["op"] == "prompt":
        s["cu_k"] = _offsets(L, dev)
        if n == L and D == Dv:  # q, k and v as a fused projection leaves them
            x = normal(T + 2, Hq + 2 * Hkv, D).to(torch.bfloat16)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"] = normal(T + 2, Hq, D).to(torch.bfloat16)
            s["k"], s["v"] = (normal(sum(L) + 2, Hkv, d).to(torch.bfloat16) for d in (D, Dv))
        return s
    ppr = max(1, -(-c["hi"] // c["ps"]))
    num_pages = c["B"] * ppr + 3
    s["table"] = torch.randperm(num_pages, generator=gen, device=dev)[:c["B"] * ppr].view(c["B"], ppr).to(torch.int32).contiguous()
    s["lens"] = torch.tensor(L, dtype=torch.int32, device=dev)
    s["k_pool"], s["v_pool"], s["params"], s["scale"] = _pool(c, num_pages, gen, dev)
    s["q"] = normal(T + 2, Hq, D).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _attend(out, lse, q, k, v, causal):
    """One sequence in fp32: q [n, Hq, D], k and v [L, Hkv, D]; writes out [n, Hq, Dv] and lse [n, Hq]."""
    n, Hq, D = q.shape
    L, Hkv, Dv = v.shape
    G = Hq // Hkv
    if n == 0:
        return
    q, k, v = q.float(), k.float().permute(1, 2, 0), v.float().transpose(0, 1)
    rows = max(1, (1 << 28) // (Hq * max(L, 1)))
    for a in range(0, n, rows):
        x = q[a:a + rows]
        m = x.shape[0]
        x = x.view(m, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * m, D)  # a KV head's rows: head of the group, then token
        x = (x @ k).mul_(1.0 / math.sqrt(D))
        if causal:
            last = (L - n + a + torch.arange(m, device=x.device))[:, None]
            x.view(Hkv, G, m, L).masked_fill_(torch.arange(L, device=x.device) > last, -math.inf)
        top = x.amax(-1, keepdim=True) if L else x.new_full((*x.shape[:-1], 1), -math.inf)
        top = torch.where(top == -math.inf, 0.0, top)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p @ v) / total.clamp(min=1e-37)
        out[a:a + m] = o.view(Hkv, G, m, Dv).permute(2, 0, 1, 3).reshape(m, Hq, Dv).to(out.dtype)
        lse[a:a + m] = (total.log() + top).view(Hkv, G, m).permute(2, 0, 1).reshape(m, Hq)


def _read(s, b):
    """fp32 K and V of request b from the cache: [L, Hkv, D]."""
    ps, kv = s["c"]["ps"], s["c"]["kv"]
    at = torch.arange(s["L"][b], device=s["table"].device)
    rows = s["table"][b][at // ps].long() * ps + at % ps
    both = []
    for i, name in enumerate(("k_pool", "v_pool")):
        x = s[name].flatten(0, 1)[rows]
        if kv == "int4":
            p = s["params"].flatten(0, 1)[rows].float()[..., 2 * i:2 * i + 2]
            x = torch.stack([x & 15, x >> 4], -1).flatten(-2).float() * p[..., 0:1] + p[..., 1:2]
        elif kv == "fp8":
            x = x.view(torch.float8_e4m3fn).float() * s["scale"]
        elif kv == "int8":
            x = x.float() * s["scale"]
        both.append(x)
    return both


def _plain(s):
    c = s["c"]
    if c["op"] == "merge":
        lse = torch.stack(s["lses"])
        top = lse.amax(0)
        top = torch.where(top == -math.inf, 0.0, top)
        w = (lse - top).exp()
        total = w.sum(0)
        out = sum(x[..., None] * o.float() for x, o in zip(w, s["outs"])) / total.clamp(min=1e-37)[..., None]
        return {"out": out.to(torch.bfloat16), "lse": total.log() + top}
    t = u = 0
    for b, (n, L) in enumerate(zip(s["n"], s["L"])):
        k, v = (s["k"][u:u + L], s["v"][u:u + L]) if c["op"] == "prompt" else _read(s, b)
        _attend(s["out"][t:t + n], s["lse"][t:t + n], s["q"][t:t + n], k, v, c["causal"])
        t, u = t + n, u + L
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    s, c = state, state["c"]
    if not own:
        return _plain(s)
    import gqa_decode_attention_gb300 as gq
    if c["op"] == "merge":
        out, lse = gq.gqa_merge(s["outs"], s["lses"])
    elif c["op"] == "prompt":
        out, lse = gq.gqa_prefill(s["q"], s["k"], s["v"], s["cu"], None if s["n"] == s["L"] else s["cu_k"], out=s["out"],
                                  lse=s["lse"], causal=c["causal"])
    else:
        out, lse = gq.gqa_prefill_paged(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["cu"], out=s["out"],
                                        lse=s["lse"], causal=c["causal"], kv_params=s["params"], k_scale=s["scale"],
                                        v_scale=s["scale"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "merge":
        rows = c["T"] * c["H"]
        return {"bytes": (c["N"] + 1) * rows * (2 * c["D"] + 4), "flops": 2 * c["N"] * rows * c["D"]}
    n, L = _lens(c)
    Hkv, D, Dv = c["Hkv"], c["D"], c.get("Dv", c["D"])
    rows = sum(n) * c["Hq"]
    kv = c.get("kv", "bf16")
    entry = Hkv * (D + Dv) * 2 if kv == "bf16" else 2 * Hkv * (D // 2 + 4 if kv == "int4" else D)  # a token's K and V
    pages = 0 if c["op"] == "prompt" else 4 * sum(-(-x // c["ps"]) for x in L) + 4 * c["B"]
    return {"bytes": rows * (2 * D + 2 * Dv + 4) + sum(x for x, m in zip(L, n) if m) * entry + pages + 4 * c["B"],
            "flops": 2 * _pairs(c) * c["Hq"] * (D + Dv)}


# ------------------------------------------------------------------------------------------------ 64 bits
def _values64(s, which, b):
    """Request b's K or V in 64 bits from its pages, one page after the other: [L, Hkv, D]."""
    ps, L = s["c"]["ps"], s["L"][b]
    kv, pages = s["c"]["kv"], s["table"][b, :-(-L // ps)].long()
    x = s["%s_pool" % which].index_select(0, pages).flatten(0, 1)[:L]
    if kv == "int4":
        p = s["params"].index_select(0, pages).flatten(0, 1)[:L].double()
        i = 0 if which == "k" else 2
        y = torch.empty(*x.shape[:-1], 2 * x.shape[-1], dtype=torch.float64, device=x.device)
        y[..., 0::2] = (x % 16).double()
        y[..., 1::2] = torch.div(x, 16, rounding_mode="floor").double()
        return y * p[..., i, None] + p[..., i + 1, None]
    if kv == "fp8":
        return x.view(torch.float8_e4m3fn).double() * s["scale"]
    return x.double() * (s["scale"] if kv == "int8" else 1.0)


def exact(case, seed):
    c = case
    if c["op"] != "merge":
        n, L = _lens(c)
        if sum(x * y for x, y in zip(n, L)) * 2 * c["Hq"] * (c["D"] + c.get("Dv", c["D"])) > EXACT_FLOPS:
            return None
    s = prepare(case, seed)
    if c["op"] == "merge":
        lses = torch.stack([x.double() for x in s["lses"]], -1)
        lse = torch.logsumexp(lses, -1)
        share = torch.where(lses == -math.inf, 0.0, torch.exp(lses - lse[..., None]))
        out = torch.zeros(s["outs"][0].shape, dtype=torch.float64, device="cuda")
        for i, o in enumerate(s["outs"]):
            out += share[..., i:i + 1] * o.double()
        return {"out": out, "lse": lse}
    out, lse = (torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in ("out", "lse"))
    G = c["Hq"] // c["Hkv"]
    t = u = 0
    for b in range(c["B"]):
        if c["op"] == "prompt":
            k, v = s["k"][u:u + L[b]].double(), s["v"][u:u + L[b]].double()
        else:
            k, v = _values64(s, "k", b), _values64(s, "v", b)
        step = max(1, (1 << 25) // max(1, L[b]))
        for h in range(c["Hq"]):
            kh, vh = k[:, h // G], v[:, h // G]
            for a in range(0, n[b], step):
                e = min(n[b], a + step)
                x = (s["q"][t + a:t + e, h].double() @ kh.T) / math.sqrt(c["D"])
                if c["causal"]:
                    x += torch.full_like(x, -math.inf).triu(L[b] - n[b] + a + 1)
                total = torch.logsumexp(x, -1) if L[b] else torch.full((e - a,), -math.inf, dtype=torch.float64, device="cuda")
                lse[t + a:t + e, h] = total
                out[t + a:t + e, h] = torch.exp(x - torch.where(total == -math.inf, 0.0, total)[:, None]) @ vh
        t, u = t + n[b], u + L[b]
    return {"out": out, "lse": lse}
