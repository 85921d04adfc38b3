"""Host-side tests of the token-side operators' entry points (no GPU needed):
every argument is checked before anything is launched."""
import pytest
import torch

import row_normalization_inner_gb300 as nf

# Fake, never dereferenced addresses, far enough apart for the sizes below;
# every call returns from argument validation.
A, B, C, D, E = (k << 36 for k in range(1, 6))
BIG = 1 << 62


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


# ---------------------------------------------------------------- 8-bit RMSNorm

def q8(q=A, scale=B, x=C, w=D, rows=4, hidden=256, eps=1e-6, fmt=0, group=0):
    return nf.nf_rmsnorm_q8(q, scale, x, w, rows, hidden, eps, fmt, group, None)


def fused_q8(q=A, scale=B, x=C, res=E, w=D, rows=4, hidden=256, eps=1e-6, fmt=0, group=0):
    return nf.nf_fused_add_rmsnorm_q8(q, scale, x, res, w, rows, hidden, eps, fmt, group, None)


@pytest.mark.parametrize("call", [q8, fused_q8])
def test_q8_refusals(call):
    for hidden in (0, 4, 12, -8, 4095, nf.Q8_MAX_HIDDEN + 8):
        assert call(hidden=hidden) == nf.NF_ERR_UNSUPPORTED_HIDDEN
    for bad in ({"rows": -1}, {"rows": BIG}, {"eps": 0.0}, {"eps": -1.0}, {"eps": float("nan")},
                {"eps": float("inf")}, {"fmt": 2}, {"fmt": -1}, {"group": 64}, {"group": -128},
                {"q": None}, {"scale": None}, {"x": None}, {"w": None}):
        assert call(**bad) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"q": A + 4}, {"scale": B + 2}, {"x": C + 8}, {"w": D + 2}):
        assert call(**bad) == nf.NF_ERR_MISALIGNED, bad
    # nothing may overlap
    for bad in ({"q": C}, {"q": C + 4 * 256 * 2 - 8}, {"scale": C + 16}, {"scale": A + 4 * 256 - 4},
                {"q": D}, {"scale": D + 8}):
        assert call(**bad) == nf.NF_ERR_INVALID_ARG, bad
    # group scales: 2 per row
    assert call(scale=A - 4 * 2 * 4 + 4, group=128) == nf.NF_ERR_INVALID_ARG
    assert call(rows=0, q=None, scale=None, x=None, w=None) == nf.NF_OK


def test_q8_fused_residual_refusals():
    assert fused_q8(res=None) == nf.NF_ERR_INVALID_ARG
    assert fused_q8(res=E + 2) == nf.NF_ERR_MISALIGNED
    for res in (C, C + 16, A, D, B):
        assert fused_q8(res=res) == nf.NF_ERR_INVALID_ARG


def test_q8_helper_refusals():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nf.rmsnorm_q8(x, w)
    with pytest.raises(TypeError):
        nf.rmsnorm_q8(x.float(), w)
    with pytest.raises(TypeError):
        nf.fused_add_rmsnorm_q8(None, x, w)


# ---------------------------------------------------------------- embedding

def embed(y=A, ids=B, id_bytes=8, table=C, tokens=4, vocab=100, hidden=64, scale=1.0):
    return nf.nf_embedding_fwd(y, ids, id_bytes, table, tokens, vocab, hidden, scale, None)


def embed_grad(grad=A, kind=nf.NF_F32, add=0, dy=B, ids=C, id_bytes=8, tokens=4, vocab=100, hidden=64,
               scale=1.0, ws=D, ws_bytes=1 << 34):
    return nf.nf_embedding_bwd(grad, kind, add, dy, ids, id_bytes, tokens, vocab, hidden, scale, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("call", [embed, embed_grad])
def test_embedding_refusals(call):
    for hidden in (0, 4, 12, -8, (1 << 20) + 8):
        assert call(hidden=hidden) == nf.NF_ERR_UNSUPPORTED_HIDDEN
    for bad in ({"tokens": -1}, {"tokens": 1 << 31}, {"vocab": 0}, {"vocab": -5}, {"vocab": (1 << 30) + 1},
                {"scale": float("nan")}, {"scale": float("inf")}, {"id_bytes": 2}, {"id_bytes": 0}, {"ids": None}):
        assert call(**bad) == nf.NF_ERR_INVALID_ARG, bad


def test_embedding_fwd_pointers():
    for bad in ({"y": None}, {"table": None}, {"y": B}, {"y": B + 16}, {"y": C}, {"y": C + 100 * 64 * 2 - 16}):
        assert embed(**bad) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"y": A + 8}, {"table": C + 2}, {"ids": B + 4}, {"ids": B + 2, "id_bytes": 4}):
        assert embed(**bad) == nf.NF_ERR_MISALIGNED, bad
    assert embed(tokens=0, y=None, ids=None, table=None) == nf.NF_OK


def test_embedding_bwd_arguments():
    for bad in ({"grad": None}, {"dy": None}, {"ws": None}, {"kind": 2}, {"kind": -1}, {"add": 2}, {"add": -1}):
        assert embed_grad(**bad) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"grad": A + 8}, {"dy": B + 2}, {"ids": C + 4}, {"ws": D + 8}):
        assert embed_grad(**bad) == nf.NF_ERR_MISALIGNED, bad
    assert embed_grad(tokens=0, add=1, grad=None, dy=None, ids=None, ws=None) == nf.NF_OK
    assert embed_grad(tokens=0, grad=None) == nf.NF_ERR_INVALID_ARG
    for tokens, hidden in ((0, 64), (-1, 64), (1 << 31, 64), (4, 12), (4, 0), (4, (1 << 20) + 8)):
        assert nf.nf_embedding_bwd_workspace_size(tokens, hidden) == 0


def test_embedding_helper_refusals():
    ids = torch.zeros(3, dtype=torch.int64)
    table = torch.zeros(10, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nf.embedding_fwd(ids.float(), table)
    with pytest.raises(ValueError, match="CUDA"):
        nf.embedding_fwd(ids, table)
    with pytest.raises(TypeError):
        nf.embedding_bwd(table[:3], [0, 1, 2], 10)


# ---------------------------------------------------------------- token log probabilities

F = 7 << 36
G = 8 << 36
H = 9 << 36


def logprob(lp=A, ent=B, stats=C, top_lp=D, top_ids=E, logits=F, kind=nf.NF_BF16, stride=100, targets=G,
            id_bytes=8, rows=4, vocab=100, temperature=1.0, top=5):
    return nf.nf_token_logprob_fwd(lp, ent, stats, top_lp, top_ids, logits, kind, stride, targets, id_bytes,
                                   rows, vocab, temperature, top, None)


def logprob_grad(out=A, dstride=100, logits=F, kind=nf.NF_BF16, stride=100, targets=G, id_bytes=8, stats=C,
                 ent=B, d_lp=D, d_ent=E, rows=4, vocab=100, temperature=1.0):
    return nf.nf_token_logprob_bwd(out, dstride, logits, kind, stride, targets, id_bytes, stats, ent, d_lp,
                                   d_ent, rows, vocab, temperature, None)


@pytest.mark.parametrize("call", [logprob, logprob_grad])
def test_logprob_refusals(call):
    nan, inf = float("nan"), float("inf")
    for bad in ({"kind": 2}, {"kind": -1}, {"id_bytes": 2}, {"rows": -1}, {"rows": BIG}, {"vocab": 0}, {"vocab": -1},
                {"vocab": (1 << 30) + 1, "stride": 1 << 31}, {"stride": 99}, {"stride": BIG}, {"stride": -100},
                {"temperature": 0.0}, {"temperature": -1.0}, {"temperature": nan}, {"temperature": inf},
                {"temperature": 1e-30}, {"temperature": 1e30}, {"logits": None}, {"targets": None}, {"stats": None}):
        assert call(**bad) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"logits": F + 1}, {"logits": F + 2, "kind": nf.NF_F32}, {"targets": G + 4}, {"stats": C + 4}):
        assert call(**bad) == nf.NF_ERR_MISALIGNED, bad
    assert call(rows=0, logits=None, targets=None, stats=None) == nf.NF_OK


def test_logprob_fwd_outputs():
    for bad in ({"lp": None}, {"ent": None}, {"top_lp": None}, {"top_ids": None}, {"top": -1}, {"top": 33},
                {"lp": B}, {"lp": F}, {"lp": F + 3 * 200 + 196}, {"ent": G + 8}, {"stats": F + 8}, {"top_lp": F},
                {"top_ids": D + 16}, {"top_ids": G}, {"top_lp": A + 8}):
        assert logprob(**bad) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"lp": A + 2}, {"ent": B + 1}, {"top_lp": D + 2}, {"top_ids": E + 4}):
        assert logprob(**bad) == nf.NF_ERR_MISALIGNED, bad


def test_logprob_bwd_outputs():
    for bad in ({"out": None}, {"d_lp": None}, {"ent": None}, {"dstride": 99}, {"out": F + 2}, {"out": F + 790},
                {"out": F, "dstride": 108}, {"out": G}, {"out": C}, {"out": B}, {"out": D}, {"out": E}):
        assert logprob_grad(**bad) == nf.NF_ERR_INVALID_ARG, bad
    for bad in ({"out": A + 1}, {"d_lp": D + 2}, {"d_ent": E + 2}, {"ent": B + 2}):
        assert logprob_grad(**bad) == nf.NF_ERR_MISALIGNED, bad


def test_logprob_helper_refusals():
    logits = torch.zeros(3, 10)
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        nf.token_logprob_fwd(logits, ids)
    with pytest.raises(TypeError):
        nf.token_logprob_fwd(logits.double(), ids)
    with pytest.raises(TypeError):
        nf.token_logprob_bwd(None, ids, None, None, None)
