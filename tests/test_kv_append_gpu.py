"""The append to a paged cache against the definition in 64 bits (bounds:
heads_reference); every slot that no token of the call has is compared bit for
bit with what it held."""
import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import (NORM, TURN, check_quantized, close, frequencies, gen, heads, normed, rates_of, turn)

pytestmark = pytest.mark.gpu

BF, F32, E4M3, INT8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


def bits(t):
    return t.clone(memory_format=torch.contiguous_format).view(torch.uint8)


class Step:
    """A call's inputs: sequences of the given lengths before it and new tokens in it, pages in a shuffled order."""

    def __init__(self, g, past, new, page, hq, hk, dim, kind=BF, cell=None, spare=3, ids=None, order="slots first"):
        self.kind, self.dim, self.hk, self.page = kind, dim, hk, page
        seqs, tokens = len(past), sum(new)
        self.past, self.new = past, new
        whole = heads(g, tokens, hq + 2 * hk, dim, kind=kind, scale=2.0)
        self.q, self.k, self.v = torch.split(whole, [hq, hk, hk], 1)
        self.qw, self.kw = [(1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(kind) for _ in range(2)]
        held = [-(-(max(p, 0) + n) // page) for p, n in zip(past, new)]
        self.pages = sum(held) + spare
        order_of = torch.randperm(self.pages, generator=g, device="cuda").tolist()
        width = max(held, default=0) + 1
        table = torch.full((seqs, width), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(held):
            table[s, :n] = torch.tensor(order_of[at:at + n], dtype=torch.int32)
            at += n
        self.table = table.cuda()
        self.past_t = torch.tensor(past, dtype=torch.int32, device="cuda")
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self.starts = None if all(n == 1 for n in new) else torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.seq = torch.repeat_interleave(torch.arange(seqs), torch.tensor(new)).cuda()
        self.place = torch.cat([torch.arange(max(p, 0), max(p, 0) + n) for p, n in zip(past, new)] + [torch.empty(0, dtype=torch.int64)]).cuda()
        shape = (self.pages, page, hk, dim) if order == "slots first" else (self.pages, hk, page, dim)
        self.cell = cell or kind
        caches = [heads(g, *shape, scale=8.0).to(torch.float32).clamp(-120, 120).to(self.cell) for _ in range(2)]
        self.scales = [torch.rand(shape[:3], generator=g, device="cuda") if self.cell in (E4M3, INT8) else None for _ in range(2)]
        if order != "slots first":
            caches = [c.transpose(1, 2) for c in caches]
            self.scales = [s if s is None else s.transpose(1, 2) for s in self.scales]
        self.caches = caches

    def used(self):
        """Tokens that are stored."""
        return (self.past_t[self.seq] >= 0)

    def call(self, **kw):
        args = dict(starts=self.starts, k_scale=self.scales[0], v_scale=self.scales[1]) | kw
        return nf.kv_append(self.k, self.v, *self.caches, self.table, self.past_t, **args)

    def check(self, before, k_rows, k_error, stored=None):
        """The caches and scales against the rows, and against `before` elsewhere."""
        stored = self.used() if stored is None else stored
        page = self.table.long()[self.seq, self.place // self.page][stored]
        slot = (self.place % self.page)[stored]
        rest = torch.ones(self.pages, self.page, dtype=torch.bool, device="cuda")
        rest[page, slot] = False
        v = self.v.double()
        for cache, scale, old, old_scale, rows, error in ((self.caches[0], self.scales[0], before[0], before[2], k_rows, k_error),
                                                          (self.caches[1], self.scales[1], before[1], before[3], v, 0 * v)):
            assert torch.equal(bits(cache[rest]), bits(old[rest]))
            got = cache[page, slot]
            if scale is None:
                close(got, rows[stored], error[stored])
            else:
                assert torch.equal(scale[rest], old_scale[rest])
                check_quantized(got, scale[page, slot], rows[stored], error[stored])

    def copy(self):
        return [t if t is None else t.clone() for t in self.caches + self.scales]


STEPS = [  # past, new, page, query heads, key heads, head_dim, rotated
    ([0], [1], 16, 4, 1, 64, 64),
    ([100000], [1], 64, 32, 8, 128, 128),
    ([5, 0, 15, 16, 17, 31, 300], [1] * 7, 16, 8, 2, 128, 64),
    ([0, 0, 3, 40], [17, 1, 0, 30], 16, 4, 4, 64, 64),
    ([7, 0, 0, 5, 1], [0, 0, 50, 0, 0], 10, 3, 1, 80, 80),
    ([2, 9], [33, 64], 1, 5, 5, 96, 48),
    ([3] * 70, [k % 4 for k in range(70)], 7, 2, 2, 72, 48),
    ([1] * 1100, [1] * 500 + [2] * 600, 3, 1, 1, 64, 64),
    ([4, 8], [3, 5], 16, 2, 2, 20, 10),
    ([4, 8], [3, 5], 16, 2, 2, 256, 0),
    ([4, 8, 1], [3, 5, 1], 16, 2, 3, 7, 6),
    ([9, 500, 0], [2000, 1, 3003], 64, 17, 9, 64, 64),  # several rows to a warp
    ([0, 5], [1500, 1011], 128, 40, 8, 128, 64),
    ([3, 0, 100, 7] * 10, [100, 101, 1, 50] * 10, 16, 8, 2, 128, 128),  # several tokens to a warp
    ([7] * 40, [101] * 40, 10, 3, 1, 80, 80),
]


@pytest.mark.parametrize("cell", ["same", E4M3, INT8])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("past,new,page,hq,hk,dim,rot", STEPS)
def test_append(past, new, page, hq, hk, dim, rot, kind, cell):
    for layout, norm, order in (("half", True, "slots first"), ("interleaved", False, "heads first")):
        g = gen(dim + page)
        s = Step(g, past, new, page, hq, hk, dim, kind, None if cell == "same" else cell, order=order)
        before, keep = s.copy(), [t.clone() for t in (s.q, s.k, s.v)]
        kw = dict(q_weight=s.qw, k_weight=s.kw, eps=EPS) if norm else {}
        q_out = s.call(q=s.q, rates=rates_of(rot), layout=layout, magnitude=1.25 if rot else 1.0, **kw)

        def rows(x, w):
            n, error = (normed(x, w, EPS), NORM) if norm else (x.double(), 0.0)
            if not rot:
                return n, error * n.abs()
            y, size = turn(n, s.place, frequencies(rot), 1.25, layout)
            return y, (error + TURN) * size
        close(q_out, *rows(s.q, s.qw))
        s.check(before, *rows(s.k, s.kw))
        assert all(torch.equal(a, b) for a, b in zip(keep, (s.q, s.k, s.v)))
        # without queries: the same caches, bit for bit
        after = s.copy()
        for t, old in zip(s.caches + s.scales, before):
            if t is not None:
                t.copy_(old)
        assert s.call(rates=rates_of(rot), layout=layout, magnitude=1.25 if rot else 1.0, **({"k_weight": s.kw} if norm else {})) is None
        assert all(a is None or torch.equal(bits(a), bits(b)) for a, b in zip(after, s.copy()))


@pytest.mark.parametrize("cell", ["same", E4M3])
@pytest.mark.parametrize("dim", [128, 80])
def test_padding_among_many_tokens(cell, dim):
    # padded sequences and missing pages beside others in one warp
    g = gen(27)
    past = [(-1 if n % 5 == 3 else 3 * n) for n in range(300)]
    s = Step(g, past, [n % 17 for n in range(300)], 8, 8, 2, dim, BF, None if cell == "same" else cell)
    gone = torch.arange(0, 300, 7)
    s.table[gone.cuda(), 1] = s.pages + 5
    before = s.copy()
    q_out = torch.full_like(s.q, 9.0)
    s.call(q=s.q, rates=rates_of(dim), q_out=q_out)
    used = s.used()
    stored = used & ~((s.seq % 7 == 0) & (s.place // 8 == 1))
    assert torch.all(q_out[~used] == 9.0)
    y, size = turn(s.q, s.place, frequencies(dim))
    close(q_out[used], y[used], TURN * size[used])
    y, size = turn(s.k, s.place, frequencies(dim))
    s.check(before, y, TURN * size, stored)


@pytest.mark.parametrize("cell", ["same", E4M3])
@pytest.mark.parametrize("dim", [128, 20])
def test_padding_and_pages_that_are_not_there(cell, dim):
    g = gen(21)
    # sequences 1 and 4 are padding; tokens behind the last sequence too
    s = Step(g, [5, -1, 20, 0, -7], [4, 3, 9, 1, 2], 8, 4, 2, dim, BF, None if cell == "same" else cell)
    tokens = len(s.seq)
    more = heads(g, tokens + 6, 8, dim)
    s.q, s.k, s.v = [torch.cat([x, more[tokens:, a:b]]) for x, a, b in ((s.q, 0, 4), (s.k, 4, 6), (s.v, 6, 8))]
    # sequence 2 (places 20 to 28) has no page for places 24 to 28, or one out of range; sequence 3's only page is out of range
    s.table[2, 3] = s.pages
    s.table[3, 0] = -5
    before = s.copy()
    q_out = torch.full_like(s.q, 9.0)
    assert s.call(q=s.q, rates=rates_of(dim), q_out=q_out) is q_out
    used = torch.cat([s.used(), torch.zeros(6, dtype=torch.bool, device="cuda")])
    stored = used[:tokens] & ~((s.seq == 2) & (s.place >= 24)) & (s.seq != 3)
    assert torch.all(q_out[~used] == 9.0)
    y, size = turn(s.q[:tokens], s.place, frequencies(dim))
    close(q_out[used], y[used[:tokens]], TURN * size[used[:tokens]])
    k, v = s.k, s.v
    s.k, s.v = k[:tokens], v[:tokens]
    y, size = turn(s.k, s.place, frequencies(dim))
    s.check(before, y, TURN * size, stored)
    # a table too narrow for a place
    s.k, s.v, s.q = k, v, s.q
    wide, s.table = s.table, s.table[:, :3]
    after = s.copy()
    s.call(rates=rates_of(dim))
    s.table = wide
    assert all(a is None or torch.equal(bits(a), bits(b)) for a, b in zip(after, s.copy()))
    # decode steps: fewer sequences than tokens, and no cache at all
    d = Step(g, [3, -1, 9, 0], [1, 1, 1, 1], 8, 4, 2, dim, BF, None if cell == "same" else cell)
    before = d.copy()
    d.table, d.past_t = d.table[:3], d.past_t[:3]
    d.seq, d.place, k, v = d.seq[:3], d.place[:3], d.k, d.v
    d.call(rates=rates_of(dim))
    d.k, d.v = k[:3], v[:3]
    y, size = turn(d.k, d.place, frequencies(dim))
    d.check(before, y, TURN * size)
    d.caches = [c[:0] for c in d.caches]
    d.scales = [c if c is None else c[:0] for c in d.scales]
    assert d.call(q=d.q[:3], rates=rates_of(dim)).shape == d.q[:3].shape


def test_given_positions_and_neighbours_of_a_view():
    g = gen(22)
    s = Step(g, [5, 20], [4, 9], 8, 4, 2, 64)
    positions = torch.randint(0, 5000, (13,), generator=g, device="cuda")
    before = s.copy()
    q = s.call(q=s.q, rates=rates_of(64), positions=positions.int())
    y, size = turn(s.q, positions, frequencies(64))
    close(q, y, TURN * size)
    y, size = turn(s.k, positions, frequencies(64))
    s.check(before, y, TURN * size)
    # keys and values side by side in one buffer, half of its slots and heads
    both = heads(g, s.pages, 2, 16, 4, 64)
    keep = both.clone()
    s.caches = [both[:, 0, 4:12, 1:3], both[:, 1, 4:12, 1:3]]
    before = s.copy()
    y, size = turn(s.q, s.place, frequencies(64))
    assert s.call(q=s.q, rates=rates_of(64), q_out=s.q) is s.q
    close(s.q, y, TURN * size)
    y, size = turn(s.k, s.place, frequencies(64))
    s.check(before, y, TURN * size)
    both[:, :, 4:12, 1:3] = keep[:, :, 4:12, 1:3]
    assert torch.equal(both, keep)


@pytest.mark.parametrize("cell", ["same", E4M3, INT8])
@pytest.mark.parametrize("dim", [64, 20])
def test_rows_of_zeros_nan_and_infinity(cell, dim):
    g = gen(23)
    s = Step(g, [0, 0, 0, 0, 0], [1] * 5, 4, 1, 2, dim, BF, None if cell == "same" else cell)
    s.k[0], s.v[0] = 0, 0
    s.k[1, 1, 3] = float("nan")
    s.v[2, 0, dim - 1] = -float("inf")
    s.v[3, 1] = 3e38
    s.call()
    page = s.table[:, 0].long()
    rows, values = s.caches[0][page, 0], s.caches[1][page, 0]
    if cell == "same":
        assert torch.equal(bits(rows), bits(s.k)) and torch.equal(bits(values), bits(s.v))
        return
    ks, vs = s.scales[0][page, 0], s.scales[1][page, 0]
    assert torch.all(ks[0] == 2.0 ** -100) and torch.all(rows[0].float() == 0) and torch.all(vs[0] == 2.0 ** -100)
    assert torch.isnan(ks[1, 1]) and torch.all(rows[1, 1].float() == 0) and torch.isfinite(ks[1, 0])
    assert torch.isnan(vs[2, 0]) and torch.all(values[2, 0].float() == 0) and torch.isfinite(vs[2, 1])
    check_quantized(values[3, 1:], vs[3, 1:], s.v[3, 1:].double(), 0 * s.v[3, 1:].double())


def test_far_pages_of_a_large_cache():
    # offsets beyond 32 bits: 2^31 and more elements before the last pages
    g = gen(24)
    pages, page, hk, dim = 2 ** 21 + 5, 8, 2, 64
    cache = torch.zeros(2, pages, page, hk, dim, dtype=E4M3, device="cuda")
    scale = torch.zeros(2, pages, page, hk, device="cuda")
    k, v = heads(g, 3, hk, dim), heads(g, 3, hk, dim)
    table = torch.tensor([[pages - 1], [0], [2 ** 21]], dtype=torch.int32, device="cuda")
    past = torch.tensor([7, 0, 3], dtype=torch.int32, device="cuda")
    nf.kv_append(k, v, cache[0], cache[1], table, past, k_scale=scale[0], v_scale=scale[1])
    at = (table[:, 0].long(), past.long())
    check_quantized(cache[0][at], scale[0][at], k.double(), 0 * k.double())
    check_quantized(cache[1][at], scale[1][at], v.double(), 0 * v.double())
    assert int((scale != 0).sum()) == 12


def test_a_sequence_by_chunks_and_by_tokens_streams_and_graphs():
    g = gen(25)
    lengths, page, hk, dim = [37, 5, 64], 16, 2, 128
    whole = [heads(g, n, 3 * hk, dim) for n in lengths]
    rates, pages = rates_of(dim), 12
    table = torch.randperm(pages, generator=g, device="cuda").int()[:12].view(3, 4)

    def fresh():
        return [torch.zeros(pages, page, hk, dim, dtype=BF, device="cuda") for _ in range(2)]

    def step(caches, past, new, **kw):
        rows = torch.cat([w[p:p + n] for w, p, n in zip(whole, past, new)])
        q, k, v = torch.split(rows, hk, 1)
        starts = torch.tensor([0, new[0], new[0] + new[1], sum(new)], dtype=torch.int32, device="cuda")
        return nf.kv_append(k, v, *caches, table, torch.tensor(past, dtype=torch.int32, device="cuda"), starts=starts, rates=rates, q=q, **kw)
    want = fresh()
    q_all = step(want, [0, 0, 0], lengths)
    chunks = fresh()
    q1 = step(chunks, [0, 0, 0], [20, 5, 1])
    q2 = step(chunks, [20, 5, 1], [17, 0, 63])
    assert all(torch.equal(a, b) for a, b in zip(want, chunks))
    assert torch.equal(torch.cat([q1[:20], q2[:17], q1[20:25], q1[25:], q2[17:]]), q_all)
    # token by token through a captured step, sequences that are done padded
    tokens = fresh()
    k, v = [torch.zeros(3, hk, dim, dtype=BF, device="cuda") for _ in range(2)]
    past = torch.zeros(3, dtype=torch.int32, device="cuda")
    nf.kv_append(k, v, *fresh(), table, past, rates=rates)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf.kv_append(k, v, *tokens, table, past, rates=rates)
    for t in range(max(lengths)):
        for s, n in enumerate(lengths):
            if t < n:
                k[s], v[s] = whole[s][t, hk:2 * hk], whole[s][t, 2 * hk:]
        past.copy_(torch.tensor([t if t < n else -1 for n in lengths], dtype=torch.int32))
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, tokens))
    other = fresh()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q = step(other, [0, 0, 0], lengths, stream=side)
    side.synchronize()
    assert torch.equal(q, q_all) and all(torch.equal(a, b) for a, b in zip(want, other))


def test_refusals():
    g = gen(26)
    s = Step(g, [5, 20], [4, 9], 8, 4, 2, 64)
    base = dict(k=s.k, v=s.v, k_cache=s.caches[0], v_cache=s.caches[1], table=s.table, past=s.past_t, starts=s.starts, rates=rates_of(64), q=s.q)
    before = s.copy()
    c = s.caches[0]
    e4, sc = c.to(E4M3), torch.zeros(c.shape[:3], device="cuda")
    bad = [(TypeError, dict(k=s.k.half())), (TypeError, dict(v=s.v.float())), (TypeError, dict(k_cache=c.float(), v_cache=c.float())),
           (TypeError, dict(v_cache=e4)), (ValueError, dict(k_cache=e4, v_cache=e4)), (ValueError, dict(k_scale=sc, v_scale=sc)),
           (TypeError, dict(k_cache=e4, v_cache=e4.clone(), k_scale=sc.double(), v_scale=sc)),
           (ValueError, dict(k_cache=e4, v_cache=e4.clone(), k_scale=sc[:1], v_scale=sc)), (ValueError, dict(k=s.k[:5])),
           (ValueError, dict(k_cache=c[:, :, :1], v_cache=c[:, :, :1])), (ValueError, dict(k_cache=c[..., :32], v_cache=c[..., :32])),
           (TypeError, dict(table=s.table.long())), (ValueError, dict(table=s.table[:1])), (TypeError, dict(past=s.past_t.long())),
           (ValueError, dict(past=s.past_t[:1])), (ValueError, dict(starts=s.starts[:2])), (TypeError, dict(starts=s.starts.long())),
           (ValueError, dict(q=None, q_weight=s.qw)), (ValueError, dict(q=None, q_out=s.q)), (ValueError, dict(q=s.q[:3])),
           (ValueError, dict(k=s.k[None], v=s.v[None])), (ValueError, dict(rates=None, positions=s.place)), (nf.NFError, dict(v_cache=c)),
           (nf.NFError, dict(k_weight=s.kw, eps=0.0)), (nf.NFError, dict(k_cache=c[:1].expand(c.shape))),
           (nf.NFError, dict(q_out=s.k.as_strided((13, 4, 64), s.k.stride())))]
    for error, change in bad:
        with pytest.raises(error):
            nf.kv_append(**(base | change))
    torch.cuda.synchronize()
    assert all(a is None or torch.equal(a, b) for a, b in zip(before, s.copy()))


TOGETHER = [  # shares with keys and values: tokens enough for four rows to a warp, past and new as below
    (32, 8, 128, 128), (40, 10, 128, 64), (32, 4, 80, 80), (6, 6, 72, 48), (3, 3, 112, 112), (1, 13, 64, 64), (32, 8, 256, 256),
]


@pytest.mark.parametrize("cell", ["same", E4M3, INT8])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("hq,hk,dim,rot", TOGETHER)
def test_keys_and_values_in_one_share(hq, hk, dim, rot, kind, cell):
    test_append([9, 500, 0], [700, 1, 803], 64, hq, hk, dim, rot, kind, cell)


@pytest.mark.parametrize("cell", ["same", E4M3])
@pytest.mark.parametrize("hq,hk,dim", [(32, 8, 128), (32, 4, 80), (40, 10, 128)])
def test_padding_beside_keys_and_values_in_one_share(hq, hk, dim, cell):
    g = gen(28)
    past = [(-1 if n % 5 == 3 else 3 * n) for n in range(170)]
    s = Step(g, past, [n % 17 for n in range(170)], 8, hq, hk, dim, BF, None if cell == "same" else cell)
    gone = torch.arange(0, 170, 7)
    s.table[gone.cuda(), 1] = s.pages + 5
    before = s.copy()
    q_out = torch.full_like(s.q, 9.0)
    s.call(q=s.q, rates=rates_of(dim), q_out=q_out)
    used = s.used()
    stored = used & ~((s.seq % 7 == 0) & (s.place // 8 == 1))
    assert torch.all(q_out[~used] == 9.0)
    y, size = turn(s.q, s.place, frequencies(dim))
    close(q_out[used], y[used], TURN * size[used])
    y, size = turn(s.k, s.place, frequencies(dim))
    s.check(before, y, TURN * size, stored)


@pytest.mark.parametrize("cell", ["same", E4M3, INT8])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("hq,hk,dim,rot", [(8, 1, 128, 128), (5, 1, 64, 64), (8, 2, 64, 32), (7, 1, 80, 80), (8, 2, 72, 48), (3, 1, 256, 256)])
def test_keys_and_values_of_several_tokens_in_one_share(hq, hk, dim, rot, kind, cell):
    # more warps than run at a time, padded sequences and missing pages among them
    g = gen(hq + dim)
    past = [(-1 if n % 5 == 3 else 7 * n) for n in range(200)]
    s = Step(g, past, [(n * 37) % 131 for n in range(200)], 16, hq, hk, dim, kind, None if cell == "same" else cell, order="heads first")
    gone = torch.arange(0, 200, 7)
    s.table[gone.cuda(), 1] = s.pages + 5
    before = s.copy()
    q_out = torch.full_like(s.q, 9.0)
    s.call(q=s.q, rates=rates_of(rot), q_weight=s.qw, k_weight=s.kw, eps=EPS, q_out=q_out)
    used = s.used()
    stored = used & ~((s.seq % 7 == 0) & (s.place // 16 == 1))
    assert torch.all(q_out[~used] == 9.0)

    def rows(x, w):
        y, size = turn(normed(x, w, EPS), s.place, frequencies(rot))
        return y, (NORM + TURN) * size
    y, error = rows(s.q, s.qw)
    close(q_out[used], y[used], error[used])
    s.check(before, *rows(s.k, s.kw), stored)
