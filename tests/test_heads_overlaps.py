"""Sets of heads that share no byte are let through, however their rows lie
between one another's, and sets that do are refused (no GPU needed: the calls
end at an argument that is checked behind the overlaps).
"""
import random

import pytest

import row_normalization_inner_gb300 as nf
from test_heads_host import A, B, C, D, E, F, G, H, J, K, L

# a workspace of no bytes is refused behind the overlaps; without a GPU its size is not known, which comes before
LATE = (nf.NF_ERR_WORKSPACE_TOO_SMALL, nf.NF_ERR_CUDA)


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def back(q, k, dim, batch, tokens, dq=None, dk=None):
    """The gradient's status for inputs q and k and their gradients (in their own place unless given)."""
    far = [nf.Heads(x << 36, 10 ** 8, 10 ** 6, 10 ** 3, h.heads) for x, h in ((20, q), (24, k))]
    return nf.nf_qk_rmsnorm_rope_bwd(dq or q, K, far[0], q, E, dk or k, K + 4096, far[1], k, F, nf.NF_BF16, batch, tokens, dim, 1e-6, None, L, 0, None)


def test_heads_in_turn_under_a_padded_token():
    # [tokens, heads, 3, dim]: a query, a key and a value in turn, tokens 8 elements further apart than the heads fill
    for heads, dim, pad in ((4, 64, 8), (7, 80, 16), (1, 128, 24), (16, 64, 3 * 64 + 8)):
        token = heads * 3 * dim + pad
        q, k = (nf.Heads(B + 2 * dim * i, 10 * token + 8, token, 3 * dim, heads) for i in range(2))
        assert back(q, k, dim, 3, 10) in LATE
        near = nf.Heads(B + 2 * dim - 2, 10 * token + 8, token, 3 * dim, heads)
        assert back(q, near, dim, 3, 10) == nf.NF_ERR_INVALID_ARG


def test_orders_of_one_buffer():
    # queries and keys side by side in each place of a buffer of any order
    for heads, dim, tokens, batch in ((4, 64, 10, 3), (2, 80, 7, 1), (1, 64, 5, 2)):
        orders = {"bthsd": lambda b, t, h, s: ((b * tokens + t) * heads + h) * 2 + s, "btshd": lambda b, t, h, s: ((b * tokens + t) * 2 + s) * heads + h,
                  "bhtsd": lambda b, t, h, s: ((b * heads + h) * tokens + t) * 2 + s, "bhstd": lambda b, t, h, s: ((b * heads + h) * 2 + s) * tokens + t,
                  "tbhsd": lambda b, t, h, s: ((t * batch + b) * heads + h) * 2 + s, "hbstd": lambda b, t, h, s: ((h * batch + b) * 2 + s) * tokens + t,
                  "sbthd": lambda b, t, h, s: ((s * batch + b) * tokens + t) * heads + h, "thbsd": lambda b, t, h, s: ((t * heads + h) * batch + b) * 2 + s,
                  "htsbd": lambda b, t, h, s: ((h * tokens + t) * 2 + s) * batch + b}
        for name, at in orders.items():
            strides = [dim * at(*x) for x in ((1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0))]
            q, k = nf.Heads(B, *strides, heads), nf.Heads(B + 2 * dim * at(0, 0, 0, 1), *strides, heads)
            assert back(q, k, dim, batch, tokens) in LATE, name
            assert back(q, nf.Heads(k.data + 2, *strides, heads), dim, batch, tokens) == (
                nf.NF_ERR_INVALID_ARG if name != "sbthd" else back(q, k, dim, batch, tokens)), name


@pytest.mark.parametrize("cell", [nf.NF_CACHE_SAME, nf.NF_CACHE_INT8])
def test_keys_and_values_between_one_another_in_a_cache(cell):
    # pages of [heads, 2, page_size, dim]: a head's keys, then its values; the scales likewise
    pages, page, heads, dim, size = 20, 16, 4, 64, 1 if cell else 2
    q = nf.Heads(C, 0, heads * dim, dim, heads)

    def cache(at, scale_at):
        return nf.Pages(A + at * size, heads * 2 * page * dim, dim, 2 * page * dim, G + 4 * scale_at, heads * 2 * page, 1, 2 * page)

    def append(k, v):
        return nf.nf_kv_append(k, v, cell, pages, page, q, nf.Heads(D, 0, heads * dim, dim, heads), None, None, None, None, nf.NF_BF16, 10, 3, dim, H, H + 4096,
                               H + 8192, 7, 7, 1e-6, nf.Rope(J, dim, 0, 1.0, None, 0, 0), None)
    import torch
    if torch.cuda.is_available():
        pytest.skip("what is let through would be launched")
    assert append(cache(0, 0), cache(page * dim, page)) == nf.NF_ERR_CUDA
    assert append(cache(0, 0), cache(page * dim - 1, page)) == nf.NF_ERR_INVALID_ARG
    if cell:
        assert append(cache(0, 0), cache(page * dim, page - 1)) == nf.NF_ERR_INVALID_ARG


def test_random_views_are_decided_exactly():
    # against the bytes that they cover; an output's own rows have to be in order, each stride over what the smaller ones cover
    rng = random.Random(11)
    dim, let, refused = 4, 0, 0

    def covered(base, n, strides):
        return {base + 2 * (b * strides[0] + t * strides[1] + h * strides[2] + e) for b in range(n[0]) for t in range(n[1]) for h in range(n[2])
                for e in range(dim)}

    def in_order(n, strides):
        held = dim
        for s, count in sorted(zip(strides, n)):
            if count > 1:
                if s < held:
                    return False
                held += (count - 1) * s
        return True
    for _ in range(6000):
        n = (rng.choice([1, 2, 3]), rng.choice([1, 2, 4]))
        views = []
        for heads in (rng.choice([1, 2, 3]), rng.choice([1, 2, 5])):
            sizes, strides, step = (*n, heads), [0, 0, 0], dim * rng.choice([1, 1, 2, 3])
            for d in rng.sample(range(3), 3):
                strides[d] = step
                step = step * sizes[d] * rng.choice([1, 1, 2]) + rng.choice([0, 0, 0, 1, dim, 3 * dim])
            if views and rng.random() < 0.6:  # the same steps as the other
                strides = views[0][2]
            views.append((sizes, A + 2 * rng.choice([0, 1, 4, 8, 12, 16, 24, 32, 48, 64, 100, 203]), strides))
        (n1, b1, s1), (n2, b2, s2) = views
        q, k = nf.Heads(b1, *s1, n1[2]), nf.Heads(b2, *s2, n2[2])
        shared = bool(covered(b1, n1, s1) & covered(b2, n2, s2))
        far = nf.Heads(30 << 36, 10 ** 6, 10 ** 4, 100, k.heads)
        for dk in (k, far):  # both as outputs; k as an input beside the output q
            st = back(q, k, dim, n1[0], n1[1], dk=dk)
            good = not shared and in_order(n1, s1) and (dk is far or in_order(n2, s2))
            assert (st in LATE) == good, (views, st)
            let += good
            refused += not good
    assert let > 2000 and refused > 2000


def test_large_sets_are_decided_at_once():
    import time
    rng = random.Random(3)
    start = time.perf_counter()
    for _ in range(300):
        heads, dim, batch = rng.choice([1, 8, 999]), 64, rng.choice([1, 7, 1000])
        tokens = 2 ** 31 // (batch * heads * 2) - 1
        token = heads * 2 * dim + 8 * rng.randrange(3)
        strides = (token * tokens + 8 * rng.randrange(5), token, 2 * dim)
        q, k = nf.Heads(1 << 50, *strides, heads), nf.Heads((1 << 50) + 2 * dim, *strides, heads)
        far = [nf.Heads(x << 50, *strides, heads) for x in (3, 5)]
        st = nf.nf_qk_rmsnorm_rope_bwd(q, K, far[0], q, E, k, K + 4096, far[1], k, F, nf.NF_BF16, batch, tokens, dim, 1e-6, None, L, 0, None)
        assert st in LATE
    assert time.perf_counter() - start < 3.0
