"""GPU tests of prompt attention at its edges, against plain 64-bit computations."""
import pytest
import torch

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
