"""Plain 64-bit form of prompt attention, for the tests, with the bounds that its roundings give.  Nothing here uses the
library."""
from __future__ import annotations

import math

import torch

import cache_ref as ref

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative


def attend(q, k, v, causal, scale=None):
    """q [n, Hq, D] over k [L, Hkv, D], v [L, Hkv, Dv], all double.  Returns out [n, Hq, Dv], lse [n, Hq], and for the
    bounds the weighted sum of |v| (mag), the largest sum of |q_d k_d| * scale of a row's keys (s_mag) and the largest |v|."""
    n, Hq, D = q.shape
    L, Hkv, Dv = v.shape
    dev = q.device
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    if n == 0 or L == 0:
        return z(n, Hq, Dv), torch.full((n, Hq), -math.inf, dtype=torch.float64, device=dev), z(n, Hq, Dv), z(n, Hq), z(n, Hq)
    q = q.view(n, Hkv, Hq // Hkv, D)
    x = torch.einsum("nhgd,lhd->nhgl", q, k) * scale
    s_mag = torch.einsum("nhgd,lhd->nhgl", q.abs(), k.abs()) * scale
    seen = torch.ones(n, L, dtype=torch.bool, device=dev)
    if causal:
        seen = torch.arange(L, device=dev) <= (L - n + torch.arange(n, device=dev))[:, None]
    hide = ~seen[:, None, None]
    x, s_mag = x.masked_fill(hide, -math.inf), s_mag.masked_fill(hide, 0.0).amax(-1)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    out, mag = torch.einsum("nhgl,lhd->nhgd", p, v), torch.einsum("nhgl,lhd->nhgd", p, v.abs())
    v_max = torch.where(hide, 0.0, v.abs().amax(-1).T[None, :, None]).amax(-1)
    return out.reshape(n, Hq, Dv), lse.reshape(n, Hq), mag.reshape(n, Hq, Dv), s_mag.reshape(n, Hq), v_max.expand(n, Hkv, Hq // Hkv).reshape(n, Hq)


def bounds(out, lse, mag, s_mag, v_max, D, L, kind):
    """Largest |error| of out and lse.

    Scores: D products, exact in fp32, summed in fp32 with at most 2^-23 of the sum of magnitudes an addition (a tensor
    core may truncate), then the scale and the reference: ds = (D + 8) 2^-23 s_mag.  4-bit and 8-bit codes enter as they
    are (a 4-bit scale and zero add four roundings, counted in the 8; s_mag then is of the magnitudes u ks + |kz|, which a
    factor of 3 covers: |k| can be as small as their difference, so 4-bit bounds take them by themselves).
    Weights: exp2 to 2^-21, rounded to the values' type (bf16; fp16 for codes, with 2^-25 of the row's reference, which is
    at most the largest weight, where they are subnormal: L 2^-25 v_max).  4-bit values are rounded to fp16 as well.  The
    sum of the weights and the weighted sum: L / 128 steps and 128 terms in a step, each addition within 2^-23, and at most
    2^-23 a rescale.  out is rounded to bf16.  lse: ds, the sum's error, exp2's and the logarithm's."""
    steps = (L / 128 + 160) * 2.0 ** -23
    ds = (D + 8) * 2.0 ** -23 * s_mag
    half = 2.0 ** -8 if kind in ("dense", "bf16") else 2.0 ** -11 * (2 if kind == "int4" else 1)
    rel = half + 2 * ds + 2.0 ** -20 + 2 * steps
    tiny = 0.0 if kind in ("dense", "bf16") else L * 2.0 ** -25
    d_out = 2.0 ** -8 * out.abs() * 1.01 + rel[..., None] * mag * 1.01 + tiny * v_max[..., None] + 1e-30
    d_lse = ds + steps + 2.0 ** -20 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)
    return d_out, d_lse


def make(n, L, Hq, Hkv, D, seed, kind="dense", Dv=None, ps=16, fused=False, pad=3, gain=1.0, dev="cuda"):
    """Inputs of sequences of n[b] queries over L[b] keys.  What belongs to no sequence is NaN (rows behind the last one,
    slots and parameters past a request's length), table entries past a request's pages are out of range: neither may
    reach a result."""
    g = torch.Generator().manual_seed(seed)
    Dv = D if Dv is None else Dv
    T, nan = sum(n), float("nan")
    cu = torch.tensor([0] + list(n)).cumsum(0).int()
    d = dict(n=list(n), L=list(L), kind=kind, cu=cu.to(dev), D=D, Dv=Dv, Hq=Hq, Hkv=Hkv)
    tail = lambda x: torch.cat([x, x.new_full((pad, *x.shape[1:]), nan)])  # noqa: E731
    if kind == "dense":
        S = sum(L)
        d["cu_k"] = torch.tensor([0] + list(L)).cumsum(0).int().to(dev)
        if fused:
            assert list(n) == list(L) and D == Dv
            x = tail(torch.randn(T, Hq + 2 * Hkv, D, generator=g) * gain).to(torch.bfloat16).to(dev)
            d["q"], d["k"], d["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            d["q"] = tail(torch.randn(T, Hq, D, generator=g) * gain).to(torch.bfloat16).to(dev)
            d["k"] = tail(torch.randn(S, Hkv, D, generator=g)).to(torch.bfloat16).to(dev)
            d["v"] = tail(torch.randn(S, Hkv, Dv, generator=g)).to(torch.bfloat16).to(dev)
        at = 0
        d["kv"] = []
        for x in L:
            d["kv"].append((d["k"][at:at + x].double(), d["v"][at:at + x].double()))
            at += x
        return d
    B = len(n)
    ppr = max(1, -(-max(L) // ps))
    pages = B * ppr + pad
    d["q"] = tail(torch.randn(T, Hq, D, generator=g) * gain).to(torch.bfloat16).to(dev)
    d["scale"] = 1.0 if kind in ("bf16", "int4") else 5.0 / (448.0 if kind == "fp8" else 127.0)
    x = torch.randn(2, pages, ps, Hkv, D, generator=g)
    (kc, kp), (vc, vp) = (ref.encode(kind, x[i], d["scale"]) for i in range(2))
    table = torch.randperm(pages, generator=g)[:B * ppr].view(B, ppr).int()
    used = torch.zeros(pages * ps, dtype=torch.bool)
    rows = []
    for b, l in enumerate(L):
        rows.append(ref.slots(table[b], ps, range(l)) if l else torch.zeros(0, dtype=torch.long))
        used[rows[b]] = True
        table[b, -(-l // ps):] = 2 ** 31 - 1 if b % 2 else -7
    for c in (kc, vc):
        c.view(pages * ps, -1)[~used] = {"bf16": nan, "fp8": 127, "int8": -128, "int4": 255}[kind]
    params = None
    if kind == "int4":
        params = torch.cat([kp, vp], -1)
        params.view(pages * ps, Hkv, 4)[~used] = torch.tensor([nan, math.inf, math.inf, nan]).half()
    d.update(k_pool=kc.to(dev), v_pool=vc.to(dev), params=None if params is None else params.to(dev), table=table.to(dev),
             lens=torch.tensor(L, dtype=torch.int32).to(dev), rows=[r.to(dev) for r in rows], ps=ps)
    d["kv"] = [held(d, r) for r in d["rows"]]
    return d


def held(d, rows):
    """64-bit K and V [len(rows), Hkv, D] of the pools' slots `rows`."""
    got = []
    for i, name in enumerate(("k_pool", "v_pool")):
        p = None if d["params"] is None else d["params"].flatten(0, 1)[rows][..., 2 * i:2 * i + 2]
        got.append(ref.values(d["kind"], d[name].flatten(0, 1)[rows], p, d["scale"]))
    return tuple(got)


def call(gq, d, causal=True, **kw):
    """The library's call on d: out, lse with rows of no sequence at -7 before it (unless given)."""
    T = d["q"].shape[0]
    if "out" not in kw:
        kw["out"] = torch.full((T, d["Hq"], d["Dv"]), -7.0, dtype=torch.bfloat16, device=d["q"].device)
        kw["lse"] = torch.full((T, d["Hq"]), -7.0, device=d["q"].device)
    if d["kind"] == "dense":
        return gq.gqa_prefill(d["q"], d["k"], d["v"], d["cu"], None if d["n"] == d["L"] and not d.get("own_k") else d["cu_k"],
                              causal=causal, **kw)
    return gq.gqa_prefill_paged(d["q"], d["k_pool"], d["v_pool"], d["table"], d["lens"], d["cu"], causal=causal,
                                kv_params=d["params"], k_scale=d["scale"], v_scale=d["scale"], **kw)


def check(d, out, lse, causal=True, scale=None, what="", untouched=True):
    """Every row against 64 bits, within bounds()."""
    t = 0
    for b, (n, L) in enumerate(zip(d["n"], d["L"])):
        k, v = d["kv"][b]
        got_o, got_l = out[t:t + n].double(), lse[t:t + n].double()
        for a in range(0, n, 512):
            q = d["q"][t + a:t + min(a + 512, n)].double()
            # rows a .. of n: as the last of a shorter sequence over the keys that they may see
            Lq = min(L, max(0, L - n + a + q.shape[0])) if causal else L
            want = attend(q, k[:Lq], v[:Lq], causal, scale) if (not causal or L - n + a + q.shape[0] >= 0) else attend(q, k[:0], v[:0], False)
            if causal and Lq > 0 and Lq - q.shape[0] != L - n + a:
                raise AssertionError("rows and keys out of step")
            if d["kind"] == "int4" and Lq:
                p = d["params"].flatten(0, 1)[d["rows"][b][:Lq]].double()
                mags = [(15 * p[..., 2 * i] + p[..., 2 * i + 1].abs()).amax(0) for i in range(2)]  # [Hkv]
                g = d["Hq"] // d["Hkv"]
                sc = 1.0 / math.sqrt(d["D"]) if scale is None else scale
                s_mag = q.abs().sum(-1) * mags[0].repeat_interleave(g) * sc
                want = (want[0], want[1], mags[1].repeat_interleave(g)[None, :, None].expand_as(want[0]), s_mag, want[4])
            d_out, d_lse = bounds(*want, d["D"], Lq, d["kind"])
            o, l = got_o[a:a + q.shape[0]], got_l[a:a + q.shape[0]]
            empty = want[1] == -math.inf
            assert torch.equal(l == -math.inf, empty), f"{what} request {b}: rows without a key"
            assert torch.all(o[empty] == 0), f"{what} request {b}: rows without a key"
            e = (o - want[0]).abs() - d_out
            assert bool((e <= 0).all()), f"{what} request {b} rows {a}..: out off by {float((o - want[0]).abs().nan_to_num(9e9).max())}, {float(e.nan_to_num(9e9).max())} past its bound"
            e = torch.where(empty, 0.0, (l - want[1]).abs() - d_lse)
            assert bool((e <= 0).all()), f"{what} request {b} rows {a}..: lse {float(e.nan_to_num(9e9).max())} past its bound"
        t += n
    if untouched:
        assert torch.all(out[t:] == -7) and torch.all(lse[t:] == -7), f"{what}: rows of no sequence were written"
