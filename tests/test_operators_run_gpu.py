"""The operators together, as a drafter uses them: beams are selected over the vocabulary, their states
follow, ended beams are carried along, and an accepted path is appended to the committed states; the
head is trained on the same rows.  Checked step by step against plain lists and 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_draft_dh_gb300 import binding as dh
from speculative_decoding_draft_dh_gb300 import distill, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_beam_search_with_states_that_follow():
    """Six steps of beam search of a toy drafter whose next logits depend on everything its state
    holds, against the same search over lists of tokens."""
    R, W, V, d, S, EOS = 3, 4, 2000, 32, 6, 7
    g = torch.Generator().manual_seed(5)
    emb = torch.randn(V, d, generator=g).to(DEV)
    head = (torch.randn(d, V, generator=g) * 0.7).to(DEV)
    head[:, EOS] += 0.4 * emb.mean(0) + 0.3          # ends now and then
    cache = torch.zeros(2, R, W, S + 1, d, device=DEV)  # two layers: positions hold what was fed
    start = torch.tensor([3, 11, 90], device=DEV)
    cache[:, :, :, 0] = emb[start][None, :, None, :]
    cache[1] *= 0.5
    score = torch.full((R, W), -float("inf"), device=DEV)
    score[:, 0] = 0.0                                # one beam at first
    finished = torch.zeros(R, W, dtype=torch.int32, device=DEV)
    # the plain search: per request a list of (tokens, score, finished), by beam
    plain = [[([int(start[r])], 0.0, False)] + [None] * (W - 1) for r in range(R)]

    def logits_of(tokens):
        return torch.tanh(torch.stack([emb[t] for t in tokens]).sum(0) * 0.3) @ head

    for step in range(S):
        held = step + 1
        h = torch.tanh((cache[0, :, :, :held].sum(2) + 2 * cache[1, :, :, :held].sum(2)) * 0.15)
        logits = torch.empty(R, W, V, device=DEV)
        for r in range(R):
            for w in range(W):
                logits[r, w] = h[r, w] @ head
        parent, token, best = dh.beam_select(logits, score, W, finished=finished, pad_token=EOS)
        dh.reorder_states(cache, parent, lengths=torch.full((R,), held, dtype=torch.int32, device=DEV), length_dim=3)
        torch.cuda.synchronize()
        for r in range(R):
            cands = []
            for w, beam in enumerate(plain[r]):
                if beam is None:
                    continue
                toks, sc, fin = beam
                if fin:
                    cands.append((sc, w, EOS, toks, True))
                    continue
                z = logits_of(toks).double().cpu().numpy()
                # the state that followed is the beam's own history
                assert np.allclose(z, logits[r, w].double().cpu().numpy(), rtol=1e-4, atol=1e-4)
                lp = z - z.max() - np.log(np.exp(z - z.max()).sum())
                for v in np.argsort(-lp, kind="stable")[:W]:
                    cands.append((sc + lp[v], w, int(v), toks, False))
            cands.sort(key=lambda c: (-c[0], c[1], c[2]))
            nxt = []
            for j, (sc, w, v, toks, fin) in enumerate(cands[:W]):
                # toy logits of two summation orders differ by 1e-4 at most; the seeds' gaps are wider
                assert int(parent[r, j]) == w and int(token[r, j]) == v
                assert abs(float(best[r, j]) - sc) <= 1e-3
                nxt.append((toks + [v], sc, fin or v == EOS) if not fin else (toks, sc, True))
            plain[r] = nxt + [None] * (W - len(nxt))
        was = finished.gather(1, parent.clamp(min=0).long())
        finished = ((was != 0) | (token == EOS)).int()
        score = best
        new = emb[token.clamp(min=0).long()]
        keep = (was == 0)[..., None].float()
        cache[0, :, :, held], cache[1, :, :, held] = new * keep, 0.5 * new * keep


def test_a_round_of_drafting_and_training():
    """The head drafts, the tree is accepted, its states are appended, and the rows train the head."""
    cfg = inputs.head_config("tiny", B=4)
    x = inputs.make_head(cfg, seed=9, device=DEV)
    idx, _, exact, probs = dh.draft_head(x["h"], x["U"], x["V"], x["W"], cfg.K)
    dh.expand_children(probs, idx, 4)
    t = inputs.make_tree(inputs.TREE_CONFIGS["tiny_tree"], seed=9, device=DEV)
    acc = dh.tree_accept(t["logits"], t["parent"], t["token"])
    tree = torch.randn(2, 4, 8, 2, 16, device=DEV, dtype=torch.bfloat16)
    cache = torch.zeros(2, 4, 2, 32, 16, device=DEV, dtype=torch.bfloat16)
    held = torch.tensor([0, 5, 9, 20], dtype=torch.int32, device=DEV)
    dh.reorder_states(tree, acc["path"], out=cache, dst_base=held, out_slot_dim=3)
    o = oracle.tree_accept(t["logits"].cpu(), t["parent"].cpu(), t["token"].cpu())
    torch.cuda.synchronize()
    for r in range(4):
        path = [p for p in o["path"][r] if p >= 0]
        for i, p in enumerate(path):
            assert torch.equal(cache[:, r, :, int(held[r]) + i], tree[:, r, p])
        rest = cache[:, r].clone()
        rest[:, :, int(held[r]):int(held[r]) + len(path)] = 0
        assert not rest.any()
    # one step of each form of training, and a selection over the trained scores
    U, V = x["U"].clone().requires_grad_(True), x["V"].clone().requires_grad_(True)
    scores = (x["h"] @ U) @ V
    loss = distill.distill_loss(scores, idx, exact, temperature=2.0)
    loss.mean().backward()
    w = torch.full((4,), 0.25, device=DEV)
    l2, grad = dh.distill_topk_step(scores.detach(), idx, exact, w, temperature=2.0)
    gV = (x["h"] @ U.detach()).t() @ grad
    assert torch.allclose(l2, loss.detach(), rtol=1e-5, atol=1e-5)
    assert (gV - V.grad).norm() <= 1e-4 * V.grad.norm()
    with torch.no_grad():
        U -= 0.1 * U.grad
        V -= 0.1 * V.grad
    parent, token, score = dh.beam_select(((x["h"] @ U) @ V).detach().view(2, 2, -1), torch.zeros(2, 2, device=DEV), 6)
    assert ((parent >= 0) & (parent < 2)).all() and ((token >= 0) & (token < cfg.vocab)).all()
    assert (score[:, :-1] >= score[:, 1:]).all()


@pytest.mark.parametrize("own_streams", [False, True])
def test_calls_from_two_threads(own_streams):
    """Calls that interleave on one stream, or run on two, give what they give alone."""
    import threading
    g = torch.Generator().manual_seed(3)
    z = torch.randn(40, 30001, generator=g).to(DEV).bfloat16()
    idx = torch.randint(0, 30001, (40, 12), generator=g).int().to(DEV)
    y, w = torch.randn(40, 12, generator=g).to(DEV), torch.rand(40, generator=g).to(DEV)
    score = -torch.rand(10, 4, generator=g).to(DEV)
    beams = z.view(10, 4, 30001)
    want_step, want_beam = dh.distill_topk_step(z, idx, y, w), dh.beam_select(beams, score, 8)
    want_loss = dh.distill_topk(z, idx, y)
    torch.cuda.synchronize()
    wrong = []

    def work(calls):
        stream = torch.cuda.Stream() if own_streams else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            got = [f() for _ in range(30) for f, _ in calls]
        stream.synchronize()
        for i, out in enumerate(got):
            for a, b in zip(out, calls[i % len(calls)][1]):
                if not torch.equal(a, b):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(calls,)) for calls in (
        [(lambda: dh.distill_topk_step(z, idx, y, w), want_step), (lambda: dh.beam_select(beams, score, 8), want_beam)],
        [(lambda: dh.beam_select(beams, score, 8), want_beam), (lambda: dh.distill_topk(z, idx, y), want_loss)])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


@pytest.mark.parametrize("in_place", [False, True])
def test_rescoring_of_states_that_just_moved(in_place):
    """The hidden rows that a reordering writes last, rescored by the next call on the stream: a kernel
    that starts under the reordering may not see rows that have not moved yet."""
    A, B, d, V, K = 2000, 64, 2048, 5000, 16
    g = torch.Generator(device=DEV).manual_seed(9)
    states = torch.randn(A, 1, B, d, generator=g, device=DEV).bfloat16()
    idx = torch.arange(B, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    W = torch.randn(V, d, generator=g, device=DEV).bfloat16()
    cand = torch.randint(0, V, (B, K), generator=g, device=DEV, dtype=torch.int32)
    want = dh.exact_rescore(states[-1, 0].flip(0).contiguous(), W, cand)
    for _ in range(5):
        out = states.clone() if in_place else torch.zeros_like(states)
        torch.cuda.synchronize()
        if in_place:
            dh.reorder_states(out, idx)
        else:
            dh.reorder_states(states, idx, out=out)
        got = dh.exact_rescore(out[-1, 0], W, cand)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rescoring_of_a_gradient():
    """The same for rows that a gradient call has just written."""
    N, d, V, K = 4096, 2048, 5000, 16
    g = torch.Generator(device=DEV).manual_seed(10)
    z = torch.randn(N, d, generator=g, device=DEV).bfloat16()
    idx = torch.randint(0, d, (N, 200), generator=g, device=DEV, dtype=torch.int32)
    y = torch.randn(N, 200, generator=g, device=DEV)
    gl = torch.full((N,), 1000.0, device=DEV)
    W = torch.randn(V, d, generator=g, device=DEV).bfloat16()
    cand = torch.randint(0, V, (64, K), generator=g, device=DEV, dtype=torch.int32)
    stats = dh.distill_topk(z, idx, y)[1]
    for call in (lambda out: dh.distill_topk_step(z, idx, y, gl, grad_out=out)[1],
                 lambda out: dh.distill_topk_backward(z, idx, y, stats, gl, grad_out=out)):
        out = torch.zeros_like(z)
        call(out)
        torch.cuda.synchronize()
        want = dh.exact_rescore(out[-64:], W, cand)
        for _ in range(5):
            out = torch.zeros_like(z)
            torch.cuda.synchronize()
            got = dh.exact_rescore(call(out)[-64:], W, cand)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_memory_that_is_written_counts_as_modified():
    """Autograd notices that what it saved was overwritten: outputs that the caller gives raise their version."""
    g = torch.Generator().manual_seed(13)
    z = torch.randn(4, 5000, generator=g).to(DEV)
    idx, y = torch.randint(0, 5000, (4, 6), generator=g).int().to(DEV), torch.randn(4, 6, generator=g).to(DEV)
    w, score = torch.ones(4, device=DEV), torch.zeros(2, 2, device=DEV)
    parents = torch.tensor([[1, 0], [0, 0], [1, 1], [0, 1]], dtype=torch.int32, device=DEV)
    loss, stats = dh.distill_topk(z, idx, y)
    out = dict(loss_out=torch.empty_like(loss), stats_out=torch.empty_like(stats))
    picks = dict(parent_out=torch.empty(2, 3, dtype=torch.int32, device=DEV),
                 token_out=torch.empty(2, 3, dtype=torch.int32, device=DEV), score_out=torch.empty(2, 3, device=DEV))
    grad, moved, side = torch.empty_like(z), torch.zeros(1, 4, 2, 8, device=DEV), torch.cuda.Stream()
    calls = [(lambda s: dh.distill_topk(z, idx, y, stream=s, **out), list(out.values())),
             (lambda s: dh.distill_topk_backward(z, idx, y, stats, w, grad_out=grad, stream=s), [grad]),
             (lambda s: dh.distill_topk_step(z, idx, y, w, loss_out=out["loss_out"], grad_out=grad, stream=s),
              [out["loss_out"], grad]),
             (lambda s: dh.beam_select(z.view(2, 2, 5000), score, 3, stream=s, **picks), list(picks.values())),
             (lambda s: dh.reorder_states(moved, parents, stream=s), [moved]),
             (lambda s: dh.reorder_states(moved.clone(), parents, out=moved, stream=s), [moved])]
    for call, written in calls:
        for stream in (None, side):
            side.wait_stream(torch.cuda.current_stream())
            before = [t._version for t in written], z._version
            call(stream)
            torch.cuda.current_stream().wait_stream(side)
            assert all(t._version > v for t, v in zip(written, before[0])) and z._version == before[1]

    # the gradient in the place of logits that a backward pass still needs
    for call in (lambda t: dh.distill_topk_step(t, idx, y, w, grad_out=t),
                 lambda t: dh.distill_topk_backward(t, idx, y, stats, w, grad_out=t)):
        capped = torch.tanh(z.clone().requires_grad_(True))
        loss = distill.distill_loss(capped, idx, y)
        call(capped.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.sum().backward()
    # states that moved under one
    held = torch.tanh(torch.randn(1, 4, 2, 8, device=DEV).requires_grad_(True))
    with torch.no_grad():
        dh.reorder_states(held, parents)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        held.sum().backward()
    # tensors of inference mode have no version
    with torch.inference_mode():
        free = z.clone()
        want = dh.distill_topk_step(z, idx, y, w)
    got = dh.distill_topk_step(free, idx, y, w, grad_out=free)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and got[1] is free
