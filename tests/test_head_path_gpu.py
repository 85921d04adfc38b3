"""The operators on attention heads together, as a model uses them: a block's
rows normalized, projected, cut into heads, normalized and rotated, attended
over, and back; and the serving side, where a prompt's chunks and then single
tokens go through a paged cache.

Tolerances.  As in test_token_path_gpu: with R roundings to bf16 on the way to a
result, each off by at most 2^-8 of its own tensor, a result is within R * 2^-8
of its norm times the gain of the stages behind, near 1 here; 4 R * 2^-8 is
asserted in the 2-norm against a 64-bit evaluation of the same model.
"""
import math

import pytest
import torch

import row_normalization_inner_gb300 as nf
from heads_reference import frequencies, gen, normed, turn

pytestmark = pytest.mark.gpu

EPS, HQ, HK, DIM = 1e-6, 8, 2, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_normalization_inner_gb300 import build
    build.build()
    yield


class Block:
    def __init__(self, hidden=256, seed=0):
        g = gen(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.norm = (1 + 0.1 * draw(hidden)).bfloat16()
        self.project = (draw(hidden, (HQ + 2 * HK) * DIM) / math.sqrt(hidden)).bfloat16()
        self.qw, self.kw = (1 + 0.1 * draw(DIM)).bfloat16(), (1 + 0.1 * draw(DIM)).bfloat16()
        self.rates, self.freq, self.hidden, self.g = nf.rope_rates(DIM), frequencies(DIM), hidden, g

    def heads(self, x):
        """Views of the projection's output."""
        h = (nf.rmsnorm_fwd(x, self.norm, EPS) @ self.project).view(*x.shape[:-1], HQ + 2 * HK, DIM)
        return torch.split(h, [HQ, HK, HK], -2)


def attend(q, k, v, first=0):
    """Causal attention of queries at places first, first + 1, ... over keys and values [length, HK, DIM], in 64 bits."""
    q, k, v = (t.double() for t in (q, k, v))
    k, v = (t.repeat_interleave(HQ // HK, 1) for t in (k, v))
    scores = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(DIM)
    places = first + torch.arange(len(q), device="cuda")
    scores = scores.masked_fill(torch.arange(len(k), device="cuda")[None] > places[:, None], -math.inf)
    return torch.einsum("hqk,khd->qhd", torch.softmax(scores, -1), v)


def off(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


def test_training_step():
    b = Block()
    x = torch.randn(2, 300, b.hidden, generator=b.g, device="cuda").bfloat16()
    positions = torch.stack([torch.arange(300), 1000 + torch.arange(300)]).cuda()
    q, k, v = b.heads(x)
    qr, kr = nf.qk_rmsnorm_rope_fwd(q, k, b.qw, b.kw, positions, b.rates, EPS)
    leaves = [t.detach().double().requires_grad_() for t in (q, k, b.qw, b.kw)]
    want = [turn(normed(t, w, EPS), positions, b.freq)[0] for t, w in zip(leaves[:2], leaves[2:])]
    assert off(qr, want[0].detach()) < 4 * 2.0 ** -8 and off(kr, want[1].detach()) < 4 * 2.0 ** -8
    out = torch.stack([attend(want[0][n], want[1][n], v[n]) for n in range(2)])
    d_out = torch.randn(out.shape, generator=b.g, device="cuda", dtype=torch.float64)
    # the attention's own gradients for the rotated heads, rounded as its backward pass leaves them
    dqr, dkr = torch.autograd.grad((out * d_out).sum(), want, retain_graph=True)
    ref = torch.autograd.grad((out * d_out).sum(), leaves)
    dh = torch.zeros(2, 300, HQ + 2 * HK, DIM, device="cuda", dtype=torch.bfloat16)  # the projection's gradient, in place
    dq, dk, _ = torch.split(dh, [HQ, HK, HK], 2)
    got = nf.qk_rmsnorm_rope_bwd(dqr.bfloat16(), dkr.bfloat16(), q, k, b.qw, b.kw, positions, b.rates, EPS, dq=dq, dk=dk)
    for a, r in zip(got, ref):
        assert off(a, r) < 4 * 2 * 2.0 ** -8
    # the rotation alone, forwards and back
    qr, kr = nf.rope_fwd(q, k, positions, b.rates)
    assert off(qr, turn(q, positions, b.freq)[0]) < 4 * 2.0 ** -8
    back = nf.rope_bwd(qr, kr, positions, b.rates)
    assert off(back[0], q.double()) < 4 * 2 * 2.0 ** -8 and off(back[1], k.double()) < 4 * 2 * 2.0 ** -8


@pytest.mark.parametrize("cell", ["same", "e4m3", "int8"])
def test_serving(cell):
    b = Block(seed=1)
    lengths, page = [90, 5, 33], 16
    x = [torch.randn(n, b.hidden, generator=b.g, device="cuda").bfloat16() for n in lengths]
    whole = []
    for t in x:  # the whole sequences at once, without a cache
        q, k, v = b.heads(t)
        p = torch.arange(len(t), device="cuda")
        whole.append(attend(*nf.qk_rmsnorm_rope_fwd(q, k, b.qw, b.kw, p, b.rates, EPS), v))
    pages, types = 12, {"same": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
    caches = [torch.zeros(pages, page, HK, DIM, dtype=types[cell], device="cuda") for _ in range(2)]
    scales = [None if cell == "same" else torch.zeros(pages, page, HK, device="cuda") for _ in range(2)]
    table = torch.full((3, 6), -1, dtype=torch.int32)
    order, at = torch.randperm(pages).int(), 0
    for s, n in enumerate(lengths):
        m = -(-n // page)
        table[s, :m], at = order[at:at + m], at + m
    table = table.cuda()

    def cached(s, n):
        """The first n keys and values of a sequence, from its pages."""
        at = torch.arange(n, device="cuda")
        where = (table[s].long()[at // page], at % page)
        return [c[where].float() * (1.0 if z is None else z[where][..., None]) for c, z in zip(caches, scales)]
    # prompts in chunks of all lengths, then the rest token by token, sequences that are done padded
    out = [[] for _ in lengths]
    past = [0, 0, 0]
    for chunk in ([60, 3, 0], [20, 0, 20], [3, 1, 1]):
        q, k, v = b.heads(torch.cat([t[p:p + n] for t, p, n in zip(x, past, chunk)]))
        starts = torch.tensor([0, *torch.tensor(chunk).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        qr = nf.kv_append(k, v, *caches, table, torch.tensor(past, dtype=torch.int32, device="cuda"), starts, b.rates, q=q, q_weight=b.qw,
                          k_weight=b.kw, eps=EPS, k_scale=scales[0], v_scale=scales[1])
        for s, n in enumerate(chunk):
            if n:
                out[s].append(attend(qr[starts[s]:starts[s + 1]], *cached(s, past[s] + n), past[s]))
        past = [p + n for p, n in zip(past, chunk)]
    while any(p < n for p, n in zip(past, lengths)):
        here = [p < n for p, n in zip(past, lengths)]
        q, k, v = b.heads(torch.stack([t[min(p, len(t) - 1)] for t, p in zip(x, past)]))
        lens = torch.tensor([p if h else -1 for p, h in zip(past, here)], dtype=torch.int32, device="cuda")
        qr = nf.kv_append(k, v, *caches, table, lens, rates=b.rates, q=q, q_weight=b.qw, k_weight=b.kw, eps=EPS, k_scale=scales[0], v_scale=scales[1])
        for s, h in enumerate(here):
            if h:
                out[s].append(attend(qr[s:s + 1], *cached(s, past[s] + 1), past[s]))
                past[s] += 1
    # int8 and e4m3 round keys and values to half a step of 2^-7 of a row's largest and of 2^-3 of a value
    bound = {"same": 2.0 ** -8, "int8": 2.0 ** -6, "e4m3": 2.0 ** -4}[cell]
    for got, want in zip(out, whole):
        assert off(torch.cat(got), want) < 4 * bound


FRESH = r"""
import torch
import row_normalization_inner_gb300 as nf
rates = nf.rope_rates(128)
# all kernels met for the first time inside a capture, but the helpers' own first call
x = torch.randn(2, 1, 1, 128, device="cuda").bfloat16()
nf.rope_fwd(x, None, torch.zeros(2, 1, dtype=torch.int64, device="cuda"), rates)
g = torch.Generator(device="cuda").manual_seed(1)
q, k = torch.randn(3000, 16, 128, generator=g, device="cuda").bfloat16(), torch.randn(3000, 4, 128, generator=g, device="cuda").bfloat16()
w, f = torch.randn(128, generator=g, device="cuda").bfloat16(), torch.randn(7, 3, 90, generator=g, device="cuda")
wf, p, rf = torch.randn(90, generator=g, device="cuda"), torch.arange(3000, device="cuda"), nf.rope_rates(90)
table = torch.arange(200, dtype=torch.int32, device="cuda").view(4, 50)
past, starts = torch.tensor([0, 5, 0, 1], dtype=torch.int32, device="cuda"), torch.tensor([0, 700, 1400, 2300, 2990], dtype=torch.int32, device="cuda")
cache = [torch.zeros(200, 16, 4, 128, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
scale = [torch.zeros(200, 16, 4, device="cuda") for _ in range(2)]

def step():
    out = list(nf.rope_fwd(q, k, p, rates)) + list(nf.rope_bwd(q[:9], k[:9], p[:9], rates, "interleaved"))
    out += list(nf.qk_rmsnorm_rope_fwd(q, k, w, w, p, rates)) + list(nf.qk_rmsnorm_rope_bwd(q, k, q, k, w, w, p, rates))
    out += [t for t in nf.qk_rmsnorm_rope_bwd(f, None, f, None, wf, None, p[:7], rf) if t is not None]
    qo = torch.zeros_like(q)
    out += [nf.kv_append(k, k, *cache, table, past, starts, rates, q=q, k_weight=w, k_scale=scale[0], v_scale=scale[1], q_out=qo)]
    return out + [t.view(torch.uint8).clone() for t in cache] + [t.clone() for t in scale]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("captured")
"""


def test_kernels_first_met_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def calls(seed):
    g = gen(seed)
    q, k = (torch.randn(700, n, DIM, generator=g, device="cuda").bfloat16() for n in (HQ, HK))
    w, p, rates = torch.ones(DIM, device="cuda").bfloat16(), torch.arange(700, device="cuda") + seed, nf.rope_rates(DIM)
    table, past = torch.arange(50, dtype=torch.int32, device="cuda")[None], torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 700], dtype=torch.int32, device="cuda")

    def run():
        cache = [torch.zeros(50, 16, HK, DIM, device="cuda").bfloat16() for _ in range(2)]
        qo = nf.kv_append(k, k, *cache, table, past, starts, rates, q=q, q_weight=w)
        return [*nf.rope_fwd(q, k, p, rates), *nf.qk_rmsnorm_rope_fwd(q, k, w, w, p, rates), *nf.qk_rmsnorm_rope_bwd(q, k, q, k, w, w, p, rates),
                qo, *cache]
    return run


def test_calls_at_once_on_two_streams():
    runs = [calls(1), calls(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        got = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(r())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_from_several_threads():
    from concurrent.futures import ThreadPoolExecutor
    runs = [calls(s) for s in range(4)]
    want = [r() for r in runs]
    torch.cuda.synchronize()

    def work(r):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                got = r()
            torch.cuda.current_stream().synchronize()
        return got

    with ThreadPoolExecutor(4) as pool:
        for got, ref in zip(pool.map(work, runs), want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_a_workspace_of_two_graphs():
    # two captured gradients that share a workspace, replayed one after the other on one stream
    runs, ws = [], torch.empty(nf.nf_qk_rmsnorm_rope_bwd_workspace_size(DIM), dtype=torch.uint8, device="cuda")
    for seed in (1, 2):
        g = gen(seed)
        q, d = (torch.randn(500, HQ, DIM, generator=g, device="cuda").bfloat16() for _ in range(2))
        w = torch.ones(DIM, device="cuda").bfloat16()
        want = nf.qk_rmsnorm_rope_bwd(d, None, q, None, w, None, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = nf.qk_rmsnorm_rope_bwd(d, None, q, None, w, None, workspace=ws)
        runs.append((graph, got, want, (q, d, w)))
    for _ in range(3):
        for graph, got, _, _ in runs:
            got[2].zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for _, got, want, _ in runs for a, b in zip(got, want) if a is not None)
