"""Beam selection (dh_beam_select) against the definition in 64 bits.

Within a beam the order is the logits' own and must match exactly.  Between beams the order hangs on
the rows' normalisers, whose error is below 2^-20 (fp32 exponentials and sums): a candidate within
that of another beam's may come before or after it, and moves those of its own beam by a place with
it.  So every beam's candidates have to be the first of its own order, every place's score that of
the reference's place within 2^-20, and equal scores (equal rows at equal scores) tie exactly, to
the lowest beam and token.  Scores are within 2^-20 and half a step of fp32.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding as dh

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
CLOSE = 2.0 ** -20
NONE = -np.inf


def reference(logits, score, M, finished=None, pad=0, T=1.0):
    """(parent, token, score, all scores [R, W, V]) in 64 bits."""
    z = logits.double().cpu().numpy() / np.float64(np.float32(T))
    sc = score.double().cpu().numpy()
    R, W, V = z.shape
    full = np.full((R, W, V), NONE)
    for r in range(R):
        for w in range(W):
            if not np.isfinite(sc[r, w]):
                continue
            if finished is not None and int(finished[r, w]) != 0:
                full[r, w, 0] = sc[r, w]
                continue
            m = z[r, w].max()
            if not np.isfinite(m):
                continue
            full[r, w] = sc[r, w] - np.log(np.exp(z[r, w] - m).sum()) + (z[r, w] - m)
    par, tok = np.full((R, M), -1, np.int64), np.full((R, M), -1, np.int64)
    out = np.full((R, M), NONE)
    for r in range(R):
        flat = full[r].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:M]
        order = order[flat[order] > NONE]
        par[r, :len(order)], tok[r, :len(order)], out[r, :len(order)] = order // V, order % V, flat[order]
        if finished is not None:
            for j in range(len(order)):
                if int(finished[r, par[r, j]]) != 0:
                    tok[r, j] = pad
    return par, tok, out, full


def check(logits, score, M, finished=None, pad=0, T=1.0):
    par, tok, sc = dh.beam_select(logits, score, M, finished=finished, pad_token=pad, temperature=T)
    torch.cuda.synchronize()
    par, tok, sc = par.cpu().numpy(), tok.cpu().numpy(), sc.double().cpu().numpy()
    rp, rt, rs, full = reference(logits, score, M, finished, pad, T)
    assert np.array_equal(np.isfinite(sc), np.isfinite(rs))
    f = np.isfinite(rs)
    assert (np.abs(sc[f] - rs[f]) <= CLOSE + 2.0 ** -24 * np.abs(rs[f])).all()
    assert (par[~f] == -1).all() and (tok[~f] == -1).all()
    fin = np.zeros(score.shape, bool) if finished is None else finished.cpu().numpy() != 0
    V = logits.shape[2]
    for r in np.flatnonzero(((par != rp) | (tok != rt)).any(axis=1)):
        n = int(f[r].sum())
        at = np.where(fin[r, par[r, :n]], 0, tok[r, :n])
        s = full[r, par[r, :n], at]
        assert (np.abs(s - rs[r, :n]) <= CLOSE).all(), f"request {r}: {s} against {rs[r, :n]}"
        place = par[r, :n].astype(np.int64) * V + at
        level = s[1:] == s[:-1]
        assert (place[1:][level] > place[:-1][level]).all(), f"request {r}: order of equal scores"
        for w in range(logits.shape[1]):
            mine = at[par[r, :n] == w]
            order = np.argsort(-full[r, w], kind="stable")[:len(mine) + 1]
            assert np.array_equal(mine, order[:len(mine)]), f"request {r}: order of beam {w}"
            if len(mine) < V and full[r, w, order[-1]] > NONE:  # the beam's best that was left out
                behind = place[s == full[r, w, order[-1]]]
                assert (behind < w * V + order[-1]).all(), f"request {r}: a lower token of an equal score left out"
    return par, tok, sc


def make(R, W, V, dtype, seed=0, ld=None, base=0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    ld = ld or V
    buf = torch.zeros(base + R * W * ld, dtype=DT[dtype])
    z = buf[base:].view(R, W, ld)[:, :, :V]
    z.copy_(std * torch.randn(R, W, V, generator=g))
    hot = torch.randint(0, V, (R, W, 4), generator=g)
    z.scatter_(2, hot, (z.gather(2, hot).float() + 9.0).to(z.dtype))
    score = -10.0 * torch.rand(R, W, generator=g)
    buf = buf.to(DEV)
    return buf[base:].view(R, W, ld)[:, :, :V], score.to(DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,W,V,M,T", [(1, 1, 1, 1, 1.0), (2, 3, 5, 4, 1.0), (1, 1, 1000, 256, 1.0), (3, 4, 1024, 8, 0.7),
                                       (2, 2, 1025, 2, 2.0), (2, 8, 4096, 16, 1.0), (1, 16, 50257, 32, 1.0),
                                       (1, 4, 151936, 4, 1.0), (2, 128, 700, 256, 1.0), (5, 7, 33, 40, 1.0),
                                       (1, 2, 20000, 256, 1.0)])
def test_sizes(R, W, V, M, T, dtype):
    check(*make(R, W, V, dtype, seed=V + M), M, T=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,ld,base", [(1001, 1001, 0), (1001, 1008, 0), (1003, 1003, 1), (5000, 5003, 3), (9, 9, 5)])
def test_strides_and_alignment(V, ld, base, dtype):
    z, score = make(3, 5, V, dtype, seed=V, ld=ld, base=base)
    par, tok, sc = check(z, score, 10)
    again = dh.beam_select(z.contiguous(), score, 10)
    for a, b in zip((par, tok), again):
        np.testing.assert_array_equal(a, b.cpu().numpy())  # the rows' place in memory changes nothing
    np.testing.assert_array_equal(sc.astype(np.float32), again[2].cpu().numpy())
    wide = torch.zeros(3, 5, 2, V, dtype=z.dtype, device=DEV)
    wide[:, :, 1] = z
    other = dh.beam_select(wide[:, :, 1], score, 10)
    for a, b in zip(again, other):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_rows_tie_to_the_lowest_beam(dtype):
    """One row shared by all beams (stride 0), and copies of it at other alignments."""
    z, _ = make(1, 1, 9999, dtype, seed=7)
    score = torch.zeros(1, 6, device=DEV)
    par, tok, _ = check(z.expand(1, 6, 9999), score, 24)
    assert par[0, :6].tolist() == list(range(6)) and len(set(tok[0, :6])) == 1
    copies = z.expand(1, 6, 9999).contiguous()  # an odd row length: every row lies differently
    p2, t2, _ = check(copies, score, 24)
    np.testing.assert_array_equal(par, p2)
    np.testing.assert_array_equal(tok, t2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["constant", "two", "steps", "rising", "falling", "half"])
@pytest.mark.parametrize("W,V,M", [(1, 30000, 8), (3, 9000, 64), (2, 5000, 256), (4, 100, 16)])
def test_rows_of_few_values(kind, W, V, M, dtype):
    """Ties by the thousand: the lowest beams and tokens, whatever the list holds."""
    i = torch.arange(V, device=DEV)
    row = {"constant": i * 0.0, "two": (i % 2).float(), "steps": (i % 7).float(), "rising": i * (8.0 / V),
           "falling": -i * (8.0 / V), "half": (i >= V // 2).float()}[kind]
    z = row.to(DT[dtype]).expand(2, W, V).contiguous()
    check(z, torch.zeros(2, W, device=DEV), M)
    check(z, torch.linspace(-1, 0, 2 * W, device=DEV).view(2, W), M)
    fin = torch.zeros(2, W, dtype=torch.int32, device=DEV)
    fin[0, -1] = fin[1, 0] = 1
    lse = float(torch.logsumexp(z[0, 0].double(), 0))
    level = torch.zeros(2, W, device=DEV)
    level[fin != 0] = float(z[0, 0].max()) - lse  # finished at about the others' best score
    check(z, level, M, finished=fin, pad=5)


def test_unused_finished_and_broken_beams():
    z, score = make(6, 4, 3000, "f32", seed=9)
    inf = float("inf")
    score[0, 1:] = -inf                 # the first step: one beam
    score[1] = -inf                     # nothing
    score[2, 0], score[2, 1], score[2, 2] = float("nan"), inf, -1e9
    z[3, 0] = -inf                      # nothing left in the row
    z[3, 1, 5], z[3, 2, 7] = float("nan"), inf
    z[4, :, 100:] = -inf                # masked vocabulary
    z[4, 2, :] = torch.finfo(torch.float32).min
    fin = torch.zeros(6, 4, dtype=torch.int32, device=DEV)
    fin[5, 1], fin[5, 3] = 1, -7
    fin[0, 0] = 0
    rz, rsc = z.clone(), score.clone()
    rz[3, 1], rz[3, 2] = -inf, -inf     # no distribution: no candidate
    par, tok, sc = dh.beam_select(z, score, 12, finished=fin, pad_token=-3)
    rp, rt, rs, _ = reference(rz, torch.where(torch.isfinite(rsc), rsc, torch.full_like(rsc, -inf)), 12, fin, -3)
    np.testing.assert_array_equal(par.cpu().numpy(), rp)
    np.testing.assert_array_equal(tok.cpu().numpy(), rt)
    assert (par[1] == -1).all() and (par[3] == 3).all() and (par[0] == 0).all()
    f = np.isfinite(rs)
    assert np.array_equal(np.isfinite(sc.cpu().numpy()), f)
    assert (np.abs(sc.double().cpu().numpy()[f] - rs[f]) <= CLOSE + 2.0 ** -24 * np.abs(rs[f])).all()
    # every beam finished, with logits that must not matter
    junk = torch.full_like(z, float("nan"))
    par, tok, sc = dh.beam_select(junk, score[4:5].expand(6, 4).contiguous(), 6,
                                  finished=torch.ones(6, 4, dtype=torch.int32, device=DEV), pad_token=9)
    order = torch.argsort(score[4], descending=True, stable=True)
    assert torch.equal(par[0, :4].long(), order) and (tok[:, :4] == 9).all() and (par[:, 4:] == -1).all()
    assert torch.equal(sc[0, :4], score[4][order])


def test_far_scores_and_temperatures():
    """Scores of very different size beside each other, and extreme temperatures."""
    z, score = make(2, 4, 5000, "f32", seed=15)
    score[:, 1], score[:, 3] = -1e9, -1e30
    check(z, score, 6)
    for T in (0.01, 100.0):
        check(z, torch.zeros(2, 4, device=DEV), 6, T=T)
    par, tok, sc = dh.beam_select(z, score, 20000 // 100, temperature=1e-30)
    assert torch.isfinite(sc[:, 0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,W,V,M", [(1, 128, 60001, 200), (1, 2, 2 ** 21, 16), (40, 3, 1500, 6), (3000, 2, 64, 3), (2, 17, 151936, 20)])
def test_many_segments(R, W, V, M, dtype):
    """More segments than are staged, held in registers, or looked at in one round."""
    check(*make(R, W, V, dtype, seed=V), M)


def test_offsets_beyond_32_bits():
    z, score = make(2, 2, 3000, "bf16", seed=27)
    far = torch.empty(4 * 1_200_000_000, dtype=torch.bfloat16, device=DEV).view(2, 2, 1_200_000_000)[:, :, :3000]
    far.copy_(z)
    for a, b in zip(dh.beam_select(z, score, 6), dh.beam_select(far, score, 6)):
        assert torch.equal(a, b)


def test_m_of_a_single_row_is_its_log_probabilities():
    z, _ = make(3, 1, 20011, "bf16", seed=21)
    par, tok, sc = dh.beam_select(z, torch.zeros(3, 1, device=DEV), 64)
    logp = torch.log_softmax(z[:, 0].double(), dim=1)
    best = logp.sort(dim=1, descending=True, stable=True)
    assert torch.equal(tok.long(), best.indices[:, :64]) and (par == 0).all()
    assert ((sc.double() - best.values[:, :64]).abs() <= CLOSE + 2.0 ** -20).all()


def test_graph_capture_streams_and_workspace():
    a, b = make(4, 4, 30000, "bf16", seed=1), make(4, 4, 30000, "bf16", seed=2)
    want = [dh.beam_select(*x, 8) for x in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dh.beam_select(*x, 8))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    ws = dh.Workspace()
    streams[0].wait_stream(torch.cuda.current_stream())
    more = dh.beam_select(*a, 8, workspace=ws, stream=streams[0])
    streams[0].synchronize()
    for w, o in ((want[0], outs[0]), (want[1], outs[1]), (want[0], more)):
        for x, y in zip(w, o):
            assert torch.equal(x, y)


def test_refusals():
    z, score = make(2, 3, 50, "f32", seed=1)
    with pytest.raises(TypeError):
        dh.beam_select(z.half(), score, 2)
    for bad in (lambda: dh.beam_select(z[0], score, 2), lambda: dh.beam_select(z.transpose(1, 2), score, 2),
                lambda: dh.beam_select(z, score.double(), 2), lambda: dh.beam_select(z, score[:, :2], 2),
                lambda: dh.beam_select(z, score.cpu(), 2), lambda: dh.beam_select(z.cpu(), score, 2),
                lambda: dh.beam_select(z, score, 2, finished=score),
                lambda: dh.beam_select(z, score, 2, token_out=torch.empty(2, 3, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for M, status in ((0, 1), (-1, 1), (257, 2)):
        with pytest.raises(dh.DhError) as e:
            dh.beam_select(z, score, M)
        assert e.value.status == status
    with pytest.raises(dh.DhError):
        dh.beam_select(z, score, 2, temperature=0.0)
    with pytest.raises(dh.DhError):
        dh.beam_select(torch.zeros(1, 129, 4, device=DEV), torch.zeros(1, 129, device=DEV), 2)
    par, tok, sc = dh.beam_select(z[:0], score[:0], 2)
    same = dh.beam_select(z, score, np.int64(2), temperature=np.float32(1), pad_token=np.int32(3))
    for a, b in zip(same, dh.beam_select(z, score, 2)):
        assert torch.equal(a, b)
    assert par.shape == (0, 2) and sc.shape == (0, 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50257, 151936])
@pytest.mark.parametrize("std", [0.5, 1.0, 3.0])
def test_normalisers_at_their_stated_error(std, V, dtype):
    """The logarithm of a row's sum, by the score of its first token at a score of about its negative.

    With d = (max - z)/T and q the row's probabilities the error is at most, all of one sign, the rounding
    of log2(e)/T and 1/T to fp32, 2^-24 of the exponent: 2^-24 E_q[d]; the mean error of the 2^x unit,
    5.1e-8 over a range of exponents of one (1.5e-7 the largest); and, independent of each other, the
    terms' argument (2^-24 d) and 2^x, and the sums' roundings within a segment: its tree has 2^j additions
    of weight 2^-j at depth j, so their variance is below two of 2^-24 / sqrt 3.  Those count six
    deviations.  That is 1e-7 to 4e-7 here; scores are rounded once."""
    g = torch.Generator().manual_seed(71)
    z = (std * torch.randn(16, 1, V, generator=g)).to(DT[dtype])
    for T in (1.0, 0.7, 1.047, 1.27, 0.55, 4.0):
        d = (z.double().amax(2, keepdim=True) - z.double())[:, 0].numpy() / np.float64(np.float32(T))
        total = np.exp(-d).sum(1)
        q = np.exp(-d) / total[:, None]
        seg = 512 if dtype == "f32" else 1024
        share = np.add.reduceat(q, np.arange(0, V, seg), axis=1)
        u = 2.0 ** -24
        noise = np.sqrt((q * q * ((u * d) ** 2 / 3 + 1.5e-7 ** 2)).sum(1) + (share * share).sum(1) * 2 * u * u / 3)
        score = torch.from_numpy(np.log(total)).float()
        _, _, out = dh.beam_select(z.to(DEV), score[:, None].to(DEV), 1, temperature=T)
        err = out[:, 0].double().cpu().numpy() - (score.double().numpy() - np.log(total))
        assert (np.abs(err) <= u * (q * d).sum(1) + 5.1e-8 + 6 * noise + u * np.abs(out[:, 0].cpu().numpy())).all(), T
