"""Refusals of the paged cache's entry points that need no GPU: bad arguments get the documented status, or a Python
error, before the device is touched."""
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


def attend(lib, q=A, kp=A, vp=A, par=A, pt=A, sl=A, out=A, lse=A, B=2, Sq=1, Hq=8, Hkv=2, D=128, ps=16, ppr=4, num_pages=16, scale=0.0,
           splits=0, ws=None, ws_bytes=0):
    return lib.gqa_decode_paged_int4(q, kp, vp, par, pt, sl, out, lse, B, Sq, Hq, Hkv, D, ps, ppr, num_pages, scale, splits, ws,
                                     ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=6, Hkv=4), 1), (dict(B=0), 1), (dict(Sq=0), 1), (dict(ps=0), 1), (dict(ppr=0), 1), (dict(num_pages=0), 1),
    (dict(splits=-1), 1), (dict(q=None), 1), (dict(par=None), 1), (dict(pt=None), 1), (dict(sl=None), 1), (dict(out=None), 1),
    (dict(D=96), 2), (dict(D=256), 2), (dict(Hq=258, Hkv=2), 2), (dict(Sq=33), 2), (dict(B=65536), 2),
    (dict(ps=1 << 16, ppr=1 << 15), 2), (dict(ps=1, ppr=(1 << 31) - 63), 2), (dict(ps=1 << 16, num_pages=1 << 15), 2),
    (dict(q=A + 2), 3), (dict(kp=A + 8), 3), (dict(vp=A + 4), 3), (dict(par=A + 8), 3), (dict(out=A + 2), 3), (dict(lse=A + 2), 3),
    (dict(pt=A + 1), 3), (dict(sl=A + 2), 3),
])
def test_int4_decode_rejects(lib, kw, status):
    assert attend(lib, **kw) == status


def test_int4_sizes_reject(lib):
    assert lib.gqa_decode_paged_int4_num_splits(2, 1, 8, 2, 96, 16, 4) == -2
    assert lib.gqa_decode_paged_int4_num_splits(2, 1, 6, 4, 128, 16, 4) == -1
    assert lib.gqa_decode_paged_int4_workspace_bytes(2, 1, 8, 2, 96, 16, 4, 3) == 0
    assert lib.gqa_decode_paged_int4_workspace_bytes(2, 1, 32, 8, 128, 16, 4, 1) == 0  # one worker writes all
    assert lib.gqa_decode_paged_int4_workspace_bytes(2, 1, 8, 2, 128, 16, 4, -1) == 0


def append(lib, q=A, qs=1024, qo=A, k=A, ks=256, v=A, vs=256, kvd=BF16, kp=A, vp=A, par=None, k_scale=1.0, v_scale=1.0, kss=None,
           vss=None, ns=0, pt=A, sl=A, cu=A, cos=A, rot=128, max_pos=64, inter=0, T=4, B=2, Hq=8, Hkv=2, D=128, ps=16, ppr=4,
           num_pages=16):
    return lib.gqa_paged_append(q, qs, qo, k, ks, v, vs, kvd, kp, vp, par, k_scale, v_scale, kss, vss, ns, pt, sl, cu, cos, rot,
                                max_pos, inter, T, B, Hq, Hkv, D, ps, ppr, num_pages, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(qo=None), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(kp=None), 1), (dict(pt=None), 1), (dict(sl=None), 1), (dict(cu=None, T=5), 1), (dict(kvd=4), 1), (dict(kvd=-1), 1),
    (dict(kvd=INT4), 1), (dict(kvd=BF16, par=A), 1), (dict(kvd=FP8, k_scale=0.0), 1), (dict(kvd=INT8, v_scale=-1.0), 1),
    (dict(kvd=INT8, v_scale=float("nan")), 1), (dict(kvd=FP8, kss=A), 1), (dict(kvd=FP8, kss=A, vss=A, ns=3), 1),
    (dict(kvd=BF16, kss=A, vss=A, ns=1), 1), (dict(rot=8), 1), (dict(rot=144), 1), (dict(rot=-16), 1), (dict(cos=None), 1),
    (dict(max_pos=0), 1), (dict(ks=248), 1), (dict(vs=0), 1), (dict(qs=1000), 1),
    (dict(D=96), 2), (dict(D=256), 2), (dict(B=65536, T=0), 2),
    (dict(ks=260), 3), (dict(qs=1028), 3), (dict(k=A + 2), 3), (dict(q=A + 8), 3), (dict(qo=A + 8), 3), (dict(cos=A + 4), 3),
    (dict(kvd=INT4, par=A + 4), 3), (dict(cu=A + 1), 3), (dict(kvd=FP8, kss=A + 2, vss=A, ns=1), 3), (dict(vp=A + 8), 3),
    (dict(T=0, k=None, v=None), 0),  # nothing to do
])
def test_append_rejects(lib, kw, status):
    assert append(lib, **kw) == status


def gather(lib, kvd=BF16, kp=A, vp=A, par=None, k_scale=1.0, v_scale=1.0, kss=None, vss=None, ns=0, pt=A, sl=A, st=None, ko=A, vo=A,
           B=2, rows=8, Hkv=2, D=128, ps=16, ppr=4, num_pages=16):
    return lib.gqa_paged_gather(kvd, kp, vp, par, k_scale, v_scale, kss, vss, ns, pt, sl, st, ko, vo, B, rows, Hkv, D, ps, ppr,
                                num_pages, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(rows=-1), 1), (dict(kvd=7), 1), (dict(kvd=INT4), 1), (dict(kvd=INT8, par=A), 1), (dict(kp=None), 1),
    (dict(ko=None), 1), (dict(vo=None), 1), (dict(pt=None), 1), (dict(kvd=FP8, vss=A, ns=1), 1),
    (dict(kvd=INT8, k_scale=float("inf")), 1), (dict(D=32), 2), (dict(D=256), 2), (dict(num_pages=1 << 27), 2),
    (dict(ko=A + 8), 3), (dict(kp=A + 4), 3), (dict(st=A + 2), 3), (dict(kvd=INT4, par=A + 4), 3),
    (dict(rows=0, ko=None, vo=None), 0),
])
def test_gather_rejects(lib, kw, status):
    assert gather(lib, **kw) == status


def test_binding_rejects_host_tensors():
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: gq.gqa_paged_append(x, x, pool, pool, table, lens),
                 lambda: gq.gqa_paged_gather(pool, pool, table, lens, rows=1),
                 lambda: gq.gqa_decode_paged_int4(x[None], pool, pool, pool, table, lens)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_binding_rejects_mismatched_tensors():
    dev = "cuda"
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    pool4 = torch.zeros(4, 16, 2, 32, dtype=torch.uint8, device=dev)
    params = torch.zeros(4, 16, 2, 4, dtype=torch.float16, device=dev)
    table, lens = torch.zeros(1, 4, dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device=dev)
    bad = [
        lambda: gq.gqa_paged_append(x, x[:2], pool, pool, table, lens),                       # k and v of different lengths
        lambda: gq.gqa_paged_append(x.transpose(0, 1), x.transpose(0, 1), pool, pool, table, lens),
        lambda: gq.gqa_paged_append(x[..., ::2], x[..., ::2], pool, pool, table, lens),
        lambda: gq.gqa_paged_append(x, x, pool, pool[:2], table, lens),
        lambda: gq.gqa_paged_append(x, x, pool, pool, table.long(), lens),
        lambda: gq.gqa_paged_append(x, x, pool, pool, table, lens.repeat(2)),
        lambda: gq.gqa_paged_append(x, x, pool, pool, table, lens, q_out=x),
        lambda: gq.gqa_paged_append(x, x, pool, pool, table, lens, q=x, q_out=x[:2]),
        lambda: gq.gqa_paged_append(x, x, pool, pool, table, lens, cu_tokens=lens),
        lambda: gq.gqa_paged_append(x, x, pool, pool, table, lens, cos_sin=torch.zeros(4, 64, device=dev).half()),
        lambda: gq.gqa_paged_append(x, x, pool4, pool4, table, lens, kv_params=params[:2]),
        lambda: gq.gqa_paged_append(x.cpu(), x, pool, pool, table, lens),
        lambda: gq.gqa_paged_append(x, x, pool, pool, table, lens, k_scales=torch.ones(1, device=dev)),
        lambda: gq.gqa_paged_gather(pool, pool, table, lens),
        lambda: gq.gqa_paged_gather(pool, pool, table, lens, k_out=pool, v_out=pool),
        lambda: gq.gqa_paged_gather(pool, pool, table, lens, rows=2, starts=lens.long()),
        lambda: gq.gqa_decode_paged_int4(q, pool4, pool4, None, table, lens),
        lambda: gq.gqa_decode_paged_int4(q, pool4, pool4, params.float(), table, lens),
        lambda: gq.gqa_decode_paged_int4(q[..., :32], pool4, pool4, params, table, lens),
        lambda: gq.gqa_decode_paged_int4(q, pool4, pool4, params, table, lens, out=q[:, :, :2]),
        lambda: gq.gqa_decode_paged_int4(q, pool4, pool4, params, table, lens, lse=torch.zeros(1, 4, 2, device=dev)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            raise AssertionError(f"call {i} went through")
    with pytest.raises(gq.GQAError):
        gq.gqa_decode_paged_int4(q.repeat(1, 65, 1, 1), pool4, pool4, params, table, lens)  # 130 rows a KV head
