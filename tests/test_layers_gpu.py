"""Sampling, embedding and layer norm together with the head, as a drafter uses them: tokens are drawn, embedded and
normed into the rows that the head takes; the trunk trains with the head's distillation loss."""
import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding as dh
from speculative_decoding_draft_dh_gb300 import distill, inputs, layers

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def trunk(cfg, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    table = torch.randn(cfg.vocab, cfg.d, generator=g, device=DEV).to(dtype)
    weight = (3 + 0.3 * torch.randn(cfg.d, generator=g, device=DEV)).to(dtype)
    return table, weight, (0.1 * torch.randn(cfg.d, generator=g, device=DEV)).to(dtype), g


def test_drafting_steps():
    """Each step: the head's candidates, a token drawn from their exact logits, its row embedded, added to the state
    and normed for the head again; the draws are checked against plain 64-bit arithmetic."""
    cfg = inputs.head_config("tiny", B=4)
    x = inputs.make_head(cfg, seed=3, device=DEV)
    table, weight, bias, g = trunk(cfg, 3)
    state = x["h"].clone()
    for _ in range(5):
        h, _ = dh.layer_norm(state, weight, bias)
        idx, _, logits, _ = dh.draft_head(h, x["U"], x["V"], x["W"], cfg.K)
        u = torch.rand(cfg.B, generator=g, device=DEV)
        at, prob = dh.sample(logits, u, temperature=0.8, top_p=0.9)
        token = idx.gather(1, at.long()[:, None])[:, 0]
        state = state + dh.embed(table, token, scale=0.5)
        torch.cuda.synchronize()
        for b in range(cfg.B):
            z = logits[b].double()
            order = z.argsort(descending=True, stable=True)
            w = ((z[order] - z.max()) / float(torch.tensor(0.8))).softmax(0)
            kept = w[:int(torch.searchsorted(w.cumsum(0), float(torch.tensor(0.9)))) + 1]
            run = kept.cumsum(0) / kept.sum()
            at_ref = int(torch.searchsorted(run, float(u[b]), right=True))
            assert token[b] == idx[b, order[at_ref]]
            assert abs(prob[b] - kept[at_ref] / kept.sum()) <= 1e-6
        want = torch.nn.functional.layer_norm(state.double(), (cfg.d,), weight.double(), bias.double())
        got, _ = dh.layer_norm(state, weight, bias)
        assert (got - want).abs().max() <= 1e-5 * want.abs().max()


def test_norm_feeds_the_head_at_once():
    """The rescoring reads hidden rows that a norm or a lookup has just written."""
    cfg = inputs.head_config("batch1", B=1, d=512, vocab=8192, r=128, K=64)
    x = inputs.make_head(cfg, seed=1, device=DEV)
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    idx = torch.arange(64, dtype=torch.int32, device=DEV)[None].contiguous()
    h = x["h"].clone()
    rows = torch.randn(2, 1, 512, device=DEV).bfloat16()
    table = torch.randn(40, 512, device=DEV).bfloat16()
    for i in range(200):
        dh.layer_norm(rows[i % 2], w, out=h)
        got, _ = dh.exact_rescore(h, x["W"], idx, with_probs=False)
        keep = got.clone()
        torch.cuda.synchronize()
        want, _ = dh.exact_rescore(dh.layer_norm(rows[i % 2], w)[0].clone(), x["W"], idx, with_probs=False)
        torch.cuda.synchronize()
        assert torch.equal(keep, want)
        tok = torch.tensor([i % 40], dtype=torch.int32, device=DEV)
        dh.embed(table, tok, out=h)
        keep = dh.exact_rescore(h, x["W"], idx, with_probs=False)[0].clone()
        torch.cuda.synchronize()
        want, _ = dh.exact_rescore(table[i % 40][None].contiguous(), x["W"], idx, with_probs=False)
        assert torch.equal(keep, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_gradients(dtype):
    """Embedding, norm, the low-rank scores and the distillation loss: autograd's gradients against those of the
    same formulas in 64 bits."""
    cfg = inputs.head_config("tiny", B=4)
    x = inputs.make_head(cfg, seed=5, device=DEV)
    table, weight, bias, g = trunk(cfg, 5, dtype)
    tok = torch.randint(-1, 50, (6, 7), generator=g, device=DEV, dtype=torch.int32)
    idx = torch.randint(0, cfg.vocab, (6, 7, 8), generator=g, device=DEV, dtype=torch.int32)
    teacher = 3 * torch.randn(6, 7, 8, generator=g, device=DEV)
    U, V = x["U"].to(dtype), x["V"].to(dtype)

    def loss64(t, w, b):
        held = (tok >= 0)[..., None]
        h = torch.where(held, t[tok.clamp(min=0).long()], 0.0) * 0.7
        h = torch.nn.functional.layer_norm(h, (cfg.d,), w, b, eps=1e-3)
        q = torch.log_softmax((h @ U.double()) @ V.double() / 2, -1)
        p = torch.softmax(teacher.double() / 2, -1)
        return (4 * (p * (p.log() - q.gather(-1, idx.long()))).sum(-1)).mean()
    leaves = [t.clone().requires_grad_(True) for t in (table, weight, bias)]
    h = layers.layer_norm(layers.embedding(leaves[0], tok, scale=0.7), leaves[1], leaves[2], eps=1e-3)
    scores = (h @ U) @ V
    distill.distill_loss(scores, idx, teacher, temperature=2.0).mean().backward()
    exact = [t.double().requires_grad_(True) for t in (table, weight, bias)]
    loss64(*exact).backward()
    # the trunk's and the products' roundings; in bf16 each of the chain's seven is 2^-9 of its value on average
    tol = 1e-4 if dtype == torch.float32 else 0.03
    for got, want in zip(leaves, exact):
        assert got.grad.dtype == dtype
        assert (got.grad.double() - want.grad).norm() <= tol * want.grad.norm()


def test_autograd_shapes_and_broadcast():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(3, 4, 96, generator=g, device=DEV, requires_grad=True)
    w = torch.randn(96, generator=g, device=DEV, requires_grad=True)
    y = layers.layer_norm(x.transpose(0, 1), w)
    y.sum().backward()  # an expanded gradient
    X, W = x.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    torch.nn.functional.layer_norm(X.transpose(0, 1), (96,), W).sum().backward()
    assert (x.grad - X.grad).abs().max() <= 1e-5 and (w.grad - W.grad).abs().max() <= 1e-4
    # a broadcast input: the gradients of its copies add up
    row = torch.randn(1, 96, generator=g, device=DEV, requires_grad=True)
    k = torch.randn(5, 96, generator=g, device=DEV)
    (layers.layer_norm(row.expand(5, 96)) * k).sum().backward()
    R = row.detach().double().requires_grad_(True)
    (torch.nn.functional.layer_norm(R.expand(5, 96), (96,)) * k).sum().backward()
    assert (row.grad - R.grad).abs().max() <= 1e-5
    table = torch.randn(10, 16, generator=g, device=DEV, requires_grad=True)
    tok = torch.tensor([[1, -1], [9, 1]], dtype=torch.int32, device=DEV)
    rows = layers.embedding(table, tok, scale=2.0)
    assert rows.shape == (2, 2, 16) and not rows[0, 1].any()
    rows.sum().backward()
    want = torch.zeros(10, 16, device=DEV)
    want[1], want[9] = 4.0, 2.0
    assert torch.equal(table.grad, want)
    # bias alone; without gradients no graph
    b = torch.randn(96, generator=g, device=DEV, requires_grad=True)
    layers.layer_norm(x.detach(), None, b).sum().backward()
    assert (b.grad - 12).abs().max() == 0
    assert not layers.layer_norm(x.detach()).requires_grad and not layers.embedding(table.detach(), tok).requires_grad
    with torch.no_grad():
        assert not layers.layer_norm(x, w).requires_grad
    # a value that the backward pass needs and that is overwritten is noticed
    h = torch.randn(4, 96, generator=g, device=DEV)
    y = layers.layer_norm(h, w)
    dh.layer_norm(h, out=h)
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 61])
def test_columns_of_one_buffer(d, dtype):
    """What is read and what is written may be other columns of the same rows, with the bits of the same call between
    buffers of that layout (of another layout the order of a row's sums differs); rows that share elements are
    refused."""
    g = torch.Generator(device=DEV).manual_seed(d)
    whole = torch.randn(41, 4 * d + 3, generator=g, device=DEV).to(dtype)
    tok = torch.randint(-1, 40, (40,), generator=g, device=DEV, dtype=torch.int32)
    cols = lambda t: (t[:40, :d], t[:40, d:2 * d], t[:40, 2 * d + 1:3 * d + 1])  # noqa: E731
    x, y, dx = cols(whole)
    plain, want, want_dx = (cols(whole.clone())[i] for i in range(3))
    _, stats = dh.layer_norm(plain, out=want, with_stats=True)
    dh.layer_norm(x, out=y)
    assert torch.equal(y, want) and torch.equal(x, plain)
    grads = dh.layer_norm_backward(want, plain, stats, grad_x=want_dx)
    got = dh.layer_norm_backward(y, x, stats, grad_x=dx)
    assert all(torch.equal(a, b) for a, b in zip(got, grads)) and torch.equal(x, plain) and torch.equal(y, want)
    dh.embed(x, tok, out=y)
    assert torch.equal(y, dh.embed(plain, tok)) and torch.equal(x, plain)
    dh.embed_backward(x, tok, 40, grad_table=dx)
    assert torch.equal(dx, dh.embed_backward(plain, tok, 40, grad_table=want_dx)) and torch.equal(x, plain)
    for col in (d - 1, 1, 3 * d + 4):  # the last one's rows end in the next row's first column
        out = whole.as_strided(x.shape, x.stride(), col)
        with pytest.raises(dh.DhError, match="INVALID_ARG"):
            dh.embed(x, tok, out=out)
        with pytest.raises(dh.DhError, match="INVALID_ARG"):
            dh.layer_norm(x, out=out)


def test_gradients_are_not_captured():
    table = torch.randn(10, 16, device=DEV, requires_grad=True)
    tok = torch.tensor([1, 2], dtype=torch.int32, device=DEV)
    rows = layers.embedding(table, tok)  # an eager graph of the same leaf lives meanwhile
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(RuntimeError, match="captured"):
                layers.embedding(table, tok)
            with pytest.raises(RuntimeError, match="captured"):
                layers.layer_norm(table)
            with torch.no_grad():  # serving
                out = layers.layer_norm(layers.embedding(table, tok))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, layers.layer_norm(rows.detach()))
    rows.sum().backward()
    assert table.grad[1].eq(1).all()


def test_a_captured_training_step():
    """The step from the binding's own calls: lookup, norm, scores, loss and gradient, back to the table."""
    V, d, N, K = 5000, 256, 96, 8
    g = torch.Generator(device=DEV).manual_seed(2)
    table = torch.randn(V, d, generator=g, device=DEV)
    w = torch.ones(d, device=DEV)
    head = torch.randn(d, V, generator=g, device=DEV) * 0.05
    tok = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    idx = torch.randint(0, V, (N, K), generator=g, device=DEV, dtype=torch.int32)
    teacher = torch.randn(N, K, generator=g, device=DEV)
    weight = torch.full((N,), 1 / N, device=DEV)

    def step():
        rows = dh.embed(table, tok)
        h, stats = dh.layer_norm(rows, w, with_stats=True)
        loss, gz = dh.distill_topk_step(h @ head, idx, teacher, weight)
        gh = gz @ head.t()
        gx, gw, _ = dh.layer_norm_backward(gh, rows, stats, w, with_bias=False)
        return loss, gw, dh.embed_backward(gx, tok, V)
    for _ in range(2):
        step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    tok.copy_(torch.randint(0, 20, (N,), generator=g, device=DEV, dtype=torch.int32))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


def test_calls_on_two_streams_and_threads():
    import threading
    z = torch.randn(64, 20000, device=DEV) * 3
    u = torch.rand(64, device=DEV)
    table = torch.randn(3000, 512, device=DEV)
    tok = torch.randint(0, 3000, (5000,), device=DEV, dtype=torch.int32)
    g = torch.randn(5000, 512, device=DEV)

    def work():
        t, p = dh.sample(z, u, top_p=0.9)
        e = dh.embed(table, tok)
        y, st = dh.layer_norm(e, with_stats=True)
        return (t, p, e, y, dh.embed_backward(g, tok, 3000)) + dh.layer_norm_backward(g, e, st)
    want = work()
    torch.cuda.synchronize()
    bad = []

    def thread():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = work()
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(1)
    threads = [threading.Thread(target=thread) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_forward_mode_is_refused():
    """Tangents would be lost without a word: there is no forward-mode derivative."""
    from torch.autograd import forward_ad
    table, x = torch.randn(10, 16, device=DEV), torch.randn(4, 16, device=DEV)
    w, tok = torch.ones(16, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    calls = [lambda t: layers.embedding(t(table), tok), lambda t: layers.layer_norm(t(x)),
             lambda t: layers.layer_norm(x, t(w)), lambda t: layers.layer_norm(x, w, t(w)),
             lambda t: layers.layer_norm(t(x).t().contiguous().t(), w)]
    for call in calls:
        plain = call(lambda t: t)
        with forward_ad.dual_level():
            assert torch.equal(call(lambda t: t), plain)
            for grad in (False, True):
                for leaf in (False, True):
                    dual = lambda t: forward_ad.make_dual(t.clone().requires_grad_(leaf), torch.ones_like(t))  # noqa: E731
                    with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="forward"):
                        call(dual)
    with pytest.raises(NotImplementedError, match="forward"):
        torch.func.jvp(lambda t: layers.layer_norm(t, w), (x,), (x,))
