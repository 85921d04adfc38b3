"""The memory of the outputs that the helpers on heads make: large ones have
their own, so that one that is kept alone does not keep the other's."""
import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import gen, heads, rates_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def calls(q, k, w, p, rates):
    return {"rope_fwd": lambda **kw: nf.rope_fwd(q, k, p, rates, **kw), "rope_bwd": lambda **kw: nf.rope_bwd(q, k, p, rates, **kw),
            "qk_rmsnorm_rope_fwd": lambda **kw: nf.qk_rmsnorm_rope_fwd(q, k, w, w, p, rates, **kw),
            "qk_rmsnorm_rope_bwd": lambda **kw: nf.qk_rmsnorm_rope_bwd(q, k, q, k, w, w, p, rates, **kw)}


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["rope_fwd", "rope_bwd", "qk_rmsnorm_rope_fwd", "qk_rmsnorm_rope_bwd"])
def test_keys_kept_alone(name, kind):
    g = gen(31)
    for tokens, hq, hk, dim in ((4096, 64, 8, 128), (16, 8, 2, 64), (1500, 64, 2, 128), (2000, 64, 8, 20)):
        q, k, w = heads(g, tokens, hq, dim, kind=kind), heads(g, tokens, hk, dim, kind=kind), heads(g, dim, kind=kind)
        p, rates = torch.arange(tokens, device="cuda"), rates_of(dim)
        call = calls(q, k, w, p, rates)[name]
        got = call()[:2]
        if q.nbytes + k.nbytes > 32 << 20:
            rooms = [(t.untyped_storage().nbytes(), t.storage_offset()) for t in got]
            assert rooms == [(t.nbytes, 0) for t in got]
            torch.cuda.synchronize()
            held = torch.cuda.memory_allocated()
            want = [t.clone() for t in got]
            kept = call()[1]
            more = torch.cuda.memory_allocated() - held
            assert more <= q.nbytes + 2 * k.nbytes + (6 << 20)  # the clones, the kept keys; blocks are up to 2 MB larger
            assert torch.equal(kept, want[1])
        assert not set(range(got[0].data_ptr(), got[0].data_ptr() + got[0].nbytes, 512)) & set(range(got[1].data_ptr(), got[1].data_ptr() + got[1].nbytes, 512))
        # into the caller's own: the same bits
        names = ("dq", "dk") if name.endswith("bwd") else ("q_out", "k_out")
        own = {n: torch.empty_like(t) for n, t in zip(names, got)}
        given = call(**own)
        assert all(a is b and torch.equal(a, c) for a, b, c in zip(given, own.values(), got))
        one = call(**{names[0]: own[names[0]]})
        room = one[1].untyped_storage().nbytes()
        assert one[0] is own[names[0]] and torch.equal(one[1], got[1]) and room <= got[1].nbytes + 256
