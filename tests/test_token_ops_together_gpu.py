"""The operators that lead from one token to the next used together, as examples/head_step.py uses them: a tied table's
gradient against 64-bit autograd, answers from a head in 4 bits, sampled answers, and all of it in captured graphs.

Tolerances.  Gradients are within the framework's bound for gradients (1e-2 relative Frobenius error); the loss within
4e-3, the bound for losses of bf16 hidden states.  What two ways of making the same calls give is equal, bit by bit.
"""
from __future__ import annotations

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F
import oracle
from examples.head_step import Head, decode, train_step
from linear_cross_entropy_tmem_gb300 import token_ops

from .test_token_ops_gpu import BF, HF, SP, gen, half_step, rand, sample_ref, skewed

pytestmark = pytest.mark.gpu


def same(a, b):
    a, b = a.contiguous().view(-1), b.contiguous().view(-1)
    return a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------------------------------------------
# Training
# ---------------------------------------------------------------------------------------------------
def tied_inputs(n, d, v, seed=3):
    ids = skewed(n, v, seed).clamp(0, v - 1)
    r = rand((n, d), BF, seed + 1)
    t = torch.randint(0, v, (n,), generator=gen(seed), device="cuda")
    t[::13] = -100
    return ids, r, t


def tied_ref(head, ids, r, t):
    """Loss and gradients (residual, norm, weight) of the composition in 64 bits."""
    ref = [a.detach().double().requires_grad_(True) for a in (r, head.norm, head.weight)]
    h = ref[2][ids] * head.weight.shape[1] ** 0.5 + ref[0]
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * ref[1]
    loss = torch.nn.functional.cross_entropy(y @ ref[2].t(), t, ignore_index=-100)
    loss.backward()
    return loss.detach(), [a.grad for a in ref]


@pytest.mark.parametrize("n,d,v", [(300, 200, 1000), (515, 1280, 3001)])
def test_tied_table_gradient(n, d, v):
    ids, r, t = tied_inputs(n, d, v)
    head = Head(d, v)
    lr = r.clone().requires_grad_(True)
    loss, _ = head.tied_loss(ids, lr, t)
    loss.backward()
    want, grads = tied_ref(head, ids, r, t)
    assert abs(float(loss.detach()) - float(want)) <= 4e-3
    for got, w in zip((lr.grad, head.norm.grad, head.weight.grad), grads):
        assert oracle.relative_frobenius(got.float().cpu(), w.cpu()) <= 1e-2


def test_tied_table_gradient_added_in_place():
    """The rows' sums added to what the head's backward left in dW: the same as autograd's sum up to its rounding."""
    n, d, v = 400, 256, 2000
    ids, r, t = tied_inputs(n, d, v)
    head = Head(d, v)
    scale = d ** 0.5
    x = F.flce_embedding(head.weight.detach(), ids, scale=scale).requires_grad_(True)
    loss, _ = head.loss(x, r, t)
    loss.backward()
    dw = head.weight.grad
    before = dw.clone()
    got = F.flce_embedding_backward(x.grad, ids, v, scale=scale, dweight=dw)
    assert got is dw
    untouched = torch.ones(v, dtype=torch.bool, device="cuda")
    untouched[ids] = False
    assert same(dw[untouched], before[untouched])
    rows = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, ids, x.grad.double() * scale)
    size = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, ids, x.grad.double().abs() * scale)
    want = rows + before.double()
    count = torch.bincount(ids, minlength=v)[:, None].double()
    tol = half_step(BF, want) * 1.01 + (count + 4) * 2.0 ** -24 * (size + before.double().abs())
    assert torch.all((dw.double() - want).abs() <= tol)
    _, grads = tied_ref(head, ids, r, t)
    assert oracle.relative_frobenius(dw.float().cpu(), grads[2].cpu()) <= 1e-2


def test_tied_training_steps_run():
    ids, r, t = tied_inputs(256, 128, 500)
    head = Head(128, 500)
    for _ in range(3):
        before = head.weight.detach().clone()
        loss, norm = train_step(head, ids, r, t, lr=0.5, max_norm=0.05)
        assert torch.isfinite(loss) and float(norm) > 0.05
        size = torch.cat([p.grad.flatten().float() for p in head.parameters()]).norm()
        assert float(size) <= 0.05 * (1 + 2.0 ** -7) and not same(before, head.weight.detach())


# ---------------------------------------------------------------------------------------------------
# Answers
# ---------------------------------------------------------------------------------------------------
def test_answer_of_a_head_in_four_bits():
    """Every step of an answer by itself, then the whole chain: lookup, norm, logits, penalties, sampling."""
    b, d, v = 9, 256, 3003
    head, embed = Head(d, v), rand((v, d), BF, 2)
    w4 = head.four_bits()
    ids = torch.randint(0, v, (b,), generator=gen(1), device="cuda")
    ids[4] = -1
    x = F.flce_embedding(embed, ids)
    stream = rand((b, d), SP, 5)
    tokens = torch.randint(0, v, (b, 20), generator=gen(2), device="cuda")
    kw = dict(tokens=tokens, repetition=torch.full((b,), 1.3, device="cuda"))
    got = head.answer(x, stream, weight4=w4, **kw)
    y = F.flce_add_rms_norm(x, head.norm.detach(), stream, need_rstd=False).y
    hv = F.mxfp4_dequantize(F.mxfp4_quantize(y)).double()
    z = hv @ F.mxfp4_dequantize(w4).double().t()
    seen = torch.zeros(b, v, dtype=torch.bool, device="cuda").scatter_(1, tokens, True)
    want = torch.where(seen, torch.where(z > 0, z / 1.3, z * 1.3), z)
    size = hv.abs() @ F.mxfp4_dequantize(w4).double().abs().t()
    # the product's fp32 sums (see test_token_ops_gpu.py), two roundings to bf16, and the penalty's steps between them
    tol = 1.3 * (2 * 4 + 2) * 2.0 ** -24 * size + want.abs() * (2 * 2.0 ** -8 + 2.0 ** -15) + 2.0 ** -20
    assert torch.all((got.logits.double() - want).abs() <= tol)
    u = torch.rand(b, generator=gen(7), device="cuda")
    k, p = torch.full((b,), 30, device="cuda"), torch.full((b,), 0.8, device="cuda")
    r = F.sample_tokens(got.logits, u, top_k=k, top_p=p)
    for i in range(b):
        tok, _, kept = sample_ref(got.logits[i].cpu(), u[i].cpu(), None, k[i].cpu(), p[i].cpu())
        assert (int(r.token[i]), int(r.kept[i])) == (tok, kept)
    again = F.flce_embedding(embed, r.token)
    assert same(again, embed[r.token])


@pytest.mark.parametrize("four", [False, True], ids=["bf16", "4bits"])
def test_sampled_answers(four):
    v, d, b = 3000, 256, 5
    head, embed = Head(d, v), rand((v, d), BF, 4)
    prompts = torch.randint(0, v, (b, 9), generator=gen(5), device="cuda")
    mask = torch.zeros(b, (v + 31) // 32, dtype=torch.int32, device="cuda")
    mask[:, 10] = -1
    w4 = head.four_bits() if four else None
    # one entry left: the greedy answer
    greedy = decode(head, embed, prompts, 6, mask=mask, weight4=w4)
    assert same(greedy, decode(head, embed, prompts, 6, mask=mask, weight4=w4, sampling=dict(top_k=1), generator=gen(1)))
    some = dict(temperature=5.0, top_k=20, top_p=0.99, min_p=1e-6)
    a = decode(head, embed, prompts, 10, mask=mask, weight4=w4, sampling=some, generator=gen(1))
    assert torch.all((a >= 320) & (a < 352))
    assert same(a, decode(head, embed, prompts, 10, mask=mask, weight4=w4, sampling=some, generator=gen(1)))
    assert not same(a, decode(head, embed, prompts, 10, mask=mask, weight4=w4, sampling=some, generator=gen(2)))
    # nothing allowed: -1, whose embedding is zeros
    out = decode(head, embed, prompts, 3, mask=torch.zeros_like(mask), weight4=w4, sampling=some, generator=gen(1))
    assert torch.all(out == -1)


# ---------------------------------------------------------------------------------------------------
# Streams, graphs, marshalling
# ---------------------------------------------------------------------------------------------------
class Step:
    """One step of an answer on buffers of its own, and the gradient of its embedding; `fill` gives new inputs."""

    def __init__(self, b=7, d=192, v=5003, seed=0, workspace=None):
        self.b, self.d, self.v, self.ws = b, d, v, workspace
        self.table, self.w4 = rand((v, d), BF, seed + 1), F.mxfp4_quantize(rand((v, d), BF, seed + 2))
        self.ids = torch.zeros(b, dtype=torch.int64, device="cuda")
        self.u = torch.zeros(b, device="cuda")
        self.p = torch.full((b,), 0.9, device="cuda")
        self.k = torch.full((b,), 2000, device="cuda")
        self.dout = torch.zeros(b, d, dtype=BF, device="cuda")
        self.dw = torch.zeros(v, d, dtype=BF, device="cuda")

    def fill(self, seed):
        self.ids.copy_(skewed(self.b, self.v, seed))
        self.u.copy_(torch.rand(self.b, generator=gen(seed), device="cuda"))
        self.dout.copy_(rand((self.b, self.d), BF, seed))
        self.dw.copy_(rand((self.v, self.d), BF, seed + 1))
        self.table.copy_(rand((self.v, self.d), BF, seed + 2))

    def __call__(self):
        x = F.flce_embedding(self.table, self.ids, scale=3.0)
        z = F.mxfp4_logits(x, self.w4, softcap=30.0, workspace=self.ws)
        r = F.sample_tokens(z, self.u, top_k=self.k, top_p=self.p)
        q = F.mxfp4_quantize(x)
        g = F.flce_embedding_backward(self.dout, self.ids, self.v, workspace=self.ws)
        F.flce_embedding_backward(self.dout, r.token, self.v, dweight=self.dw, workspace=self.ws)
        return [x, z, *r, q.codes, q.scales, F.mxfp4_dequantize(q, SP), g, self.dw.clone()]


def expected(step, seed):
    step.fill(seed)
    return [t.clone() for t in step()]


def captured(step):
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    return graph, out


@pytest.mark.parametrize("shape", [(7, 192, 5003), (1, 64, 300), (130, 1000, 1501), (300, 64, 70001)], ids=str)
def test_captured_steps_take_new_values(shape):
    step = Step(*shape)
    graph, out = captured(step)
    for seed in (11, 12, 13, 12):
        want = expected(step, seed)
        step.fill(seed)
        graph.replay()
        for a, b in zip(out, want):
            assert same(a, b)


def test_two_graphs_share_a_workspace():
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    steps = [Step(7, 192, 5003, 1, ws), Step(150, 100, 1200, 2, ws)]
    graphs = [captured(s) for s in steps]
    want = [expected(s, 21 + i) for i, s in enumerate(steps)]
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for i, s in enumerate(steps):
            s.fill(21 + i)
        for i in order:
            steps[i].fill(21 + i)
            graphs[i][0].replay()
        for i in set(order):
            for a, b in zip(graphs[i][1], want[i]):
                assert same(a, b)


def test_backward_captured_while_an_eager_graph_of_the_leaf_lives():
    """Both were recorded on the stream that captures, as autograd wants it of every function."""
    v, d = 300, 64
    w = rand((v, d), BF, 1).requires_grad_(True)
    ids, up = skewed(50, v, 2), rand((50, d), BF, 3)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        eager = F.embedding(w, ids, scale=2.0)
        want, = torch.autograd.grad(F.embedding(w, ids, scale=2.0), w, up)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got, = torch.autograd.grad(F.embedding(w, ids, scale=2.0), w, up)
    for seed in (4, 5):
        up.copy_(rand((50, d), BF, seed))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want, = torch.autograd.grad(F.embedding(w, ids, scale=2.0), w, up)
            graph.replay()
        side.synchronize()
        assert same(got, want)
    with torch.cuda.stream(side):
        eager.backward(up)
    side.synchronize()
    assert same(w.grad, want)


def test_other_streams():
    """The same calls on two streams at once, each with its own inputs and workspaces."""
    steps = [Step(9, 320, 4000, 1), Step(64, 128, 9001, 2)]
    want = [expected(s, 31 + i) for i, s in enumerate(steps)]
    for i, s in enumerate(steps):
        s.fill(31 + i)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None, None]
    for _ in range(3):
        for i, (s, st) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(st):
                s.fill(31 + i)
                got[i] = s()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert same(a, b)


def test_both_ways_of_marshalling_agree(monkeypatch):
    step = Step(12, 200, 3001, 4)
    wide = rand((12, 512), BF, 6)
    z = rand((12, 3001), HF, 7)
    bias = rand((3001,), SP, 8)

    def run():
        step.fill(41)
        out = step()
        big = torch.zeros(12, 4000, dtype=SP, device="cuda")
        o = F.mxfp4_logits(wide[:, 3:203], step.w4, bias, logit_scale=0.5, out=big[:, 8:3009])
        assert o.data_ptr() == big[:, 8:].data_ptr()
        t = F.sample_tokens(z, step.u, temperature=step.p, min_p=step.p / 100)
        e = F.flce_embedding(step.table, step.ids.to(torch.int32).view(3, 4), out_dtype=SP)
        g = F.flce_embedding_backward(wide[:, 5:205], step.ids, 3001, padding_idx=0, dtype=BF)
        q = F.mxfp4_quantize(wide[:, 1:100])
        return [*out, big, *t, e, g, q.codes, q.scales, F.mxfp4_dequantize(q, HF)]
    native = run()
    monkeypatch.setattr(token_ops, "_call", lambda *a: None)
    for a, b in zip(native, run()):
        assert a.shape == b.shape and a.stride() == b.stride() and same(a, b)


@pytest.mark.parametrize("path", ["native", "python"])
def test_counts_of_in_place_changes(path, monkeypatch):
    """What a call writes into a given tensor counts as changed; what it only reads does not."""
    if path == "python":
        monkeypatch.setattr(token_ops, "_call", lambda *a: None)
    step = Step(5, 64, 300, 1)
    step.fill(1)
    out = torch.empty(5, 300, dtype=BF, device="cuda")
    x = F.flce_embedding(step.table, step.ids)
    reads = [step.table, step.ids, step.dout, step.u, x, step.w4.codes, step.w4.scales]
    before = [t._version for t in reads]
    counts = out._version, step.dw._version
    F.mxfp4_logits(x, step.w4, out=out)
    F.flce_embedding_backward(step.dout, step.ids, 300, dweight=step.dw)
    F.sample_tokens(out, step.u)
    assert out._version == counts[0] + 1 and step.dw._version == counts[1] + 1
    assert [t._version for t in reads] == before
    # a saved tensor that a call wrote raises in backward
    a = rand((5, 300), BF, 3).requires_grad_(True)
    y = (a * out).sum()
    F.mxfp4_logits(x, step.w4, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


# ---------------------------------------------------------------------------------------------------
# Forms that larger or odder calls take
# ---------------------------------------------------------------------------------------------------
def grad_ref(dout, ids, v, scale):
    on = (ids >= 0) & (ids < v)
    x = dout.double()[on] * scale
    zero = torch.zeros(v, dout.shape[1], dtype=torch.float64, device="cuda")
    return zero.index_add(0, ids[on], x), zero.index_add(0, ids[on], x.abs()), torch.bincount(ids[on], minlength=v)


@pytest.mark.parametrize("cols", [8, 56, 64, 72, 200, 256, 264, 384, 512, 520, 776, 1032, 1536, 2040])
@pytest.mark.parametrize("n", [1, 33, 250, 4500])
def test_gradient_of_narrow_tables(n, cols):
    """Several chunks of tokens to a block: every number of threads for a chunk, last blocks with chunks of no tokens."""
    v = 2500
    ids, dout = skewed(n, v, cols), rand((n, cols), SP, n)
    want, size, count = grad_ref(dout, ids, v, 2.0)
    got = F.flce_embedding_backward(dout, ids, v, scale=2.0)
    assert torch.all((got.double() - want).abs() <= (count[:, None] + 5) * 2.0 ** -24 * size * 1.0001)
    assert torch.all(got[count == 0] == 0)
    # within a wider table whose other columns stay, and rows that start off 16-byte boundaries
    wide = torch.full((v, cols + 5), 7.0, device="cuda")
    F.flce_embedding_backward(dout, ids, v, scale=2.0, dweight=wide[:, 3:3 + cols])
    assert torch.all(wide[:, :3] == 7) and torch.all(wide[:, 3 + cols:] == 7)
    assert torch.all((wide[:, 3:3 + cols].double() - 7 - want).abs() <=
                     (count[:, None] + 6) * 2.0 ** -24 * (size + 7) * 1.0001)


@pytest.mark.parametrize("cols", [1, 8, 63, 64, 130, 1000])
@pytest.mark.parametrize("t", [BF, SP], ids=str)
def test_tables_of_many_rows_are_cleared(t, cols):
    v = 300007
    ids = torch.tensor([0, v - 1, 5, 4095, 4096, v, -1], device="cuda")
    dout = torch.ones(7, cols, dtype=t, device="cuda")
    got = F.flce_embedding_backward(dout, ids, v)
    want = torch.zeros(v, cols, dtype=t, device="cuda")
    want[ids[:5]] = 1
    assert torch.equal(got, want)


def test_rows_past_32_bits():
    """Row strides that put a table's or a matrix's last rows more than 2^32 elements behind its first."""
    d, stride, v = 24, (1 << 31) + 8, 3
    flat = torch.empty((v - 1) * stride + d + v, dtype=BF, device="cuda")
    table, beside = flat.as_strided((v, d), (stride, 1)), flat.as_strided((v, v), (stride, 1), d)
    values = rand((v, d), BF, 1)
    table.copy_(values)
    ids = torch.tensor([2, 0, 1, 2, -1], device="cuda")
    x = F.flce_embedding(table, ids)
    assert same(x[:4], values[ids[:4]])
    dout = rand((5, d), BF, 2)
    want = F.flce_embedding_backward(dout, ids, v, dweight=values.clone())
    F.flce_embedding_backward(dout, ids, v, dweight=table)
    assert same(table, want)
    q, p = F.mxfp4_quantize(table), F.mxfp4_quantize(want)
    assert same(q.codes, p.codes) and same(q.scales, p.scales)
    z = F.mxfp4_logits(table, F.mxfp4_quantize(values), out=beside)
    assert same(z, F.mxfp4_logits(want, F.mxfp4_quantize(values)))
    u = torch.rand(v, generator=gen(3), device="cuda")
    a, b = F.sample_tokens(table, u), F.sample_tokens(table.contiguous(), u)
    assert same(a.token, b.token) and same(a.logprob, b.logprob)


@pytest.mark.parametrize("t", [BF, HF, SP], ids=str)
@pytest.mark.parametrize("n,d", [(1, 33), (129, 257), (400, 255), (70, 513), (33, 1283)])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_four_bits_of_rows_off_16_byte_boundaries(t, n, d, shift):
    wide = rand((n, d + 40 + d % 2), t, d)
    x = wide[:, shift:shift + d]
    q, p = F.mxfp4_quantize(x), F.mxfp4_quantize(torch.nn.functional.pad(x, (0, -d % 32 + 32))[:, :d])
    own = F.mxfp4_quantize(x.contiguous())
    for a in (p, own):
        assert same(q.codes, a.codes) and same(q.scales, a.scales)
    # both ways back: rows of d elements, and the same padded to whole blocks of 32
    full = F.MxFp4(q.codes, q.scales, -(-d // 32) * 32)
    for o in (BF, SP):
        y = F.mxfp4_dequantize(full, o)
        assert same(F.mxfp4_dequantize(q, o), y[:, :d]) and torch.all(y[:, d:] == 0)


@pytest.mark.parametrize("t", [BF, SP], ids=str)
def test_samples_where_many_entries_stand_up_to_the_cuts(t):
    """Lists of 65 to 1024 entries, cut by top-k and top-p anywhere, with ties on the cuts."""
    b, v = 24, 6000
    z = (torch.randn(b, v, generator=gen(1), device="cuda") * 2).to(t)
    z[::3] = (z[::3].float() * 4).round().to(t) / 4  # many equal values
    u = torch.rand(b, generator=gen(2), device="cuda")
    for k in (64, 65, 100, 511, 1000, 1023, 1024, 1025, 2000):
        for p in (None, 0.05, 0.5, 0.93, 0.999):
            kk = torch.full((b,), k, device="cuda")
            pp = None if p is None else torch.full((b,), p, device="cuda")
            r = F.sample_tokens(z, u, top_k=kk, top_p=pp)
            for i in range(0, b, 5):
                tok, lp, kept = sample_ref(z[i].cpu(), u[i].cpu(), None, kk[i].cpu(), None if p is None else pp[i].cpu())
                got = int(r.token[i]), int(r.kept[i])
                assert got == (tok, kept), (k, p, i, got, tok, kept)
                assert abs(float(r.logprob[i]) - lp) <= abs(lp) * 2.0 ** -23 + 2.0 ** -29
