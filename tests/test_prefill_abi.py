"""Refusals of prompt attention and of the merge that need no GPU: bad arguments get the documented status, or a Python
error, before the device is touched."""
import ctypes

import pytest
import torch

import gqa_decode_attention_gb300 as gq
from gqa_decode_attention_gb300 import build as gbuild

A = 0x7F0000000000  # a never-dereferenced, aligned device address
BF16, FP8, INT8, INT4 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gq.load_library()


def prompt(lib, q=A, qs=1024, k=A, ks=256, v=A, vs=256, cq=A, ck=None, out=A, lse=A, Tq=6, Tk=6, B=2, Hq=8, Hkv=2, D=128, Dv=128,
           causal=1, scale=0.0, ws=None, ws_bytes=0):
    return lib.gqa_prefill(q, qs, k, ks, v, vs, cq, ck, out, lse, Tq, Tk, B, Hq, Hkv, D, Dv, causal, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(Tq=-1), 1), (dict(Tk=-1), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(Hq=6, Hkv=4), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(cq=None, Tq=5), 1), (dict(cq=None, Tk=5), 1), (dict(qs=1000), 1),
    (dict(ks=248), 1), (dict(vs=0), 1),
    (dict(D=96, Dv=96), 2), (dict(D=256, Dv=256, qs=4096, ks=4096, vs=4096), 2), (dict(D=128, Dv=64), 2), (dict(D=192, Dv=192, qs=1536, ks=384, vs=384), 2),
    (dict(B=65536), 2), (dict(Hq=8194, qs=8194 * 128), 2), (dict(Tq=1 << 28), 2),
    (dict(qs=1028), 3), (dict(ks=260), 3), (dict(vs=257), 3), (dict(q=A + 8), 3), (dict(k=A + 2), 3), (dict(v=A + 4), 3), (dict(out=A + 8), 3),
    (dict(lse=A + 2), 3), (dict(cq=A + 1), 3), (dict(ck=A + 2), 3),
    (dict(Tq=0, q=None, out=None), 0),  # nothing to do
])
def test_prompt_rejects(lib, kw, status):
    assert prompt(lib, **kw) == status


def chunk(lib, q=A, qs=1024, kvd=BF16, kp=A, vp=A, par=None, k_scale=1.0, v_scale=1.0, kss=None, vss=None, ns=0, pt=A, sl=A, cu=A,
          out=A, lse=A, T=6, B=2, Hq=8, Hkv=2, D=128, ps=16, ppr=4, num_pages=16, causal=1, scale=0.0, ws=None, ws_bytes=0):
    return lib.gqa_prefill_paged(q, qs, kvd, kp, vp, par, k_scale, v_scale, kss, vss, ns, pt, sl, cu, out, lse, T, B, Hq, Hkv, D, ps,
                                 ppr, num_pages, causal, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(Hq=6, Hkv=4), 1), (dict(q=None), 1), (dict(kp=None), 1),
    (dict(vp=None), 1), (dict(out=None), 1), (dict(pt=None), 1), (dict(sl=None), 1), (dict(cu=None, T=5), 1), (dict(kvd=4), 1),
    (dict(kvd=-1), 1), (dict(kvd=INT4), 1), (dict(par=A), 1), (dict(kvd=FP8, k_scale=float("nan")), 1),
    (dict(kvd=INT8, v_scale=float("inf")), 1), (dict(kvd=FP8, kss=A), 1), (dict(kvd=FP8, kss=A, vss=A, ns=3), 1),
    (dict(kss=A, vss=A, ns=1), 1), (dict(qs=1000), 1), (dict(ps=0), 1), (dict(ppr=0), 1), (dict(num_pages=0), 1),
    (dict(D=96), 2), (dict(D=192), 2), (dict(D=256), 2), (dict(B=65536), 2), (dict(Hq=8194, qs=8194 * 128), 2), (dict(T=1 << 28), 2),
    (dict(ps=1, ppr=(1 << 31) - 63), 2), (dict(num_pages=1 << 27), 2),
    (dict(qs=1028), 3), (dict(q=A + 8), 3), (dict(kp=A + 8), 3), (dict(vp=A + 4), 3), (dict(out=A + 2), 3), (dict(lse=A + 1), 3),
    (dict(pt=A + 2), 3), (dict(sl=A + 2), 3), (dict(cu=A + 1), 3), (dict(kvd=INT4, par=A + 4), 3), (dict(kvd=FP8, kss=A + 2, vss=A, ns=1), 3),
    (dict(T=0, q=None, out=None), 0),  # nothing to do
])
def test_chunk_rejects(lib, kw, status):
    assert chunk(lib, **kw) == status


def merge(lib, outs=(A, A), lses=(A, A), n=None, out=A, lse=A, rows=4, D=128):
    ptrs = ctypes.c_void_p * max(1, len(outs))
    return lib.gqa_merge(ptrs(*outs), ptrs(*lses), len(outs) if n is None else n, out, lse, rows, D, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 1), (dict(outs=(A,) * 9, lses=(A,) * 9), 1), (dict(rows=-1), 1), (dict(D=0), 1), (dict(outs=(A, None)), 1),
    (dict(lses=(None, A)), 1), (dict(out=None), 1), (dict(D=12), 2), (dict(D=264), 2), (dict(rows=1 << 31), 2),
    (dict(outs=(A, A + 8)), 3), (dict(lses=(A, A + 2)), 3), (dict(out=A + 8), 3), (dict(lse=A + 1), 3), (dict(rows=0), 0),
])
def test_merge_rejects(lib, kw, status):
    assert merge(lib, **kw) == status


def test_workspace_sizes_reject(lib):
    assert lib.gqa_prefill_workspace_bytes(6, 2, 8, 2, 96, 96) == 0
    assert lib.gqa_prefill_workspace_bytes(-1, 2, 8, 2, 128, 128) == 0
    assert lib.gqa_prefill_paged_workspace_bytes(6, 0, 8, 2, 128) == 0


def test_binding_rejects_host_tensors():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: gq.gqa_prefill(x, x, x), lambda: gq.gqa_prefill_paged(x, pool, pool, table, lens),
                 lambda: gq.gqa_merge([x], [x[..., 0].float()])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="one to 8"):
        gq.gqa_merge([], [])


@pytest.mark.gpu
def test_binding_rejects_mismatched_tensors():
    dev = "cuda"
    x = torch.zeros(6, 4, 64, dtype=torch.bfloat16, device=dev)
    cu = torch.tensor([0, 6], dtype=torch.int32, device=dev)
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    table, lens = torch.zeros(1, 4, dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev)
    lse = torch.zeros(6, 4, device=dev)
    bad = [
        lambda: gq.gqa_prefill(x, x, x[:5]),
        lambda: gq.gqa_prefill(x, x[:, :2], x),
        lambda: gq.gqa_prefill(x[0], x, x),
        lambda: gq.gqa_prefill(x.float(), x, x),
        lambda: gq.gqa_prefill(x, x.cpu(), x),
        lambda: gq.gqa_prefill(x, x, x, cu.long()),
        lambda: gq.gqa_prefill(x, x, x, cu, torch.zeros(3, dtype=torch.int32, device=dev)),
        lambda: gq.gqa_prefill(x, x, x, cu, out=x[:5]),
        lambda: gq.gqa_prefill(x, x, x, cu, lse=lse.half()),
        lambda: gq.gqa_prefill(x.transpose(0, 1), x, x),
        lambda: gq.gqa_prefill(x[..., ::2], x[..., ::2], x[..., ::2]),
        lambda: gq.gqa_prefill(x, x, x, workspace=torch.zeros(8, dtype=torch.uint8)),
        lambda: gq.gqa_prefill_paged(x, pool, pool, table, lens, lens),
        lambda: gq.gqa_prefill_paged(x, pool, pool[:2], table, lens),
        lambda: gq.gqa_prefill_paged(x[..., :32], pool, pool, table, lens),
        lambda: gq.gqa_prefill_paged(x, pool, pool, table.long(), lens),
        lambda: gq.gqa_prefill_paged(x, pool, pool, table, lens, k_scales=torch.ones(1, device=dev)),
        lambda: gq.gqa_prefill_paged(x, pool, pool, table, lens, kv_params=lse),
        lambda: gq.gqa_merge([x, x], [lse]),
        lambda: gq.gqa_merge([x, x[:5]], [lse, lse]),
        lambda: gq.gqa_merge([x], [lse.half()]),
        lambda: gq.gqa_merge([x], [lse], out=x[:3]),
        lambda: gq.gqa_merge([x.transpose(0, 1)], [lse.T]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, gq.GQAError)):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
    assert gq.gqa_device_status() == 0
