"""Distillation from a teacher's top logits (dh_distill_topk and its gradient) against the formulas
in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding).  With x = (z - m)/T a term of the
sum has the relative error 3 u |x| (difference, constant and product) + 2^-22 (the 2^x unit), and the
sums at most 16 u: the row's sum is within 2^-20 (1 + |x|) of its terms, a probability within
2^-19 (1 + |x|), a logarithm within 2^-20 + 2 u |log|.  The loss adds p (log p - log q) with those
errors; the gradient g T (q - P) those of q and P and half a step of its own type.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding as dh
from speculative_decoding_draft_dh_gb300 import distill, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -19
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def reference(z, idx, y, T, n_valid=None, g=None):
    """Loss, stats and gradient of each row in 64 bits (numpy), with the bounds above."""
    z, y = z.double().cpu().numpy(), y.double().cpu().numpy()
    idx = idx.cpu().numpy()
    N, V = z.shape
    nv = np.full(N, idx.shape[1]) if n_valid is None else np.clip(n_valid.cpu().numpy(), 0, idx.shape[1])
    g = np.ones(N) if g is None else g.double().cpu().numpy()
    loss, ltol = np.zeros(N), np.zeros(N)
    grad, gtol = np.zeros((N, V)), np.zeros((N, V))
    m, s = z.max(axis=1), np.zeros(N)
    for n in range(N):
        with np.errstate(invalid="ignore", divide="ignore"):
            x = (z[n] - m[n]) / T if m[n] != -np.inf else np.full(V, -np.inf)
            e = np.exp(x)
            s[n] = e.sum()
            q = e / s[n] if s[n] > 0 else np.zeros(V)
            logq = x - np.log(s[n]) if s[n] > 0 else np.full(V, -np.inf)
        k = [j for j in range(nv[n]) if 0 <= idx[n, j] < V and y[n, j] > -np.inf]
        if not k:
            continue
        a = (y[n, k] - y[n, k].max()) / T
        p = np.exp(a) / np.exp(a).sum()
        logp, ids = a - np.log(np.exp(a).sum()), idx[n, k]
        loss[n] = T * T * np.sum(p * (logp - logq[ids]))
        if np.isfinite(loss[n]):
            ltol[n] = T * T * np.sum(p * E * (1 + np.abs(a)) * (1 + np.abs(logp) + np.abs(logq[ids])))
        if g[n] == 0:
            continue
        P, Pt = np.zeros(V), np.zeros(V)
        np.add.at(P, ids, p)
        np.add.at(Pt, ids, p * (1 + np.abs(a)))
        grad[n] = g[n] * T * (q - P)
        xt = np.where(np.isfinite(x), np.abs(x), 0.0)
        gtol[n] = abs(g[n]) * T * E * (q * (1 + xt) + Pt)
    return loss, ltol, np.stack([m, s], 1), grad, gtol


def make(N, V, K, dtype, seed=0, ld=None, base=0, std=3.0):
    """Logits in rows of ld elements, `base` elements into their memory, and a teacher whose entries
    are the best of a noisy reading of them (each id once)."""
    g = torch.Generator().manual_seed(seed)
    ld = ld or V
    buf = torch.full((base + N * ld,), 77.0, dtype=DT[dtype])
    z = buf[base:].view(N, ld)[:, :V]
    z.copy_(std * torch.randn(N, V, generator=g))
    noisy = z.float() + 2.0 * torch.randn(N, V, generator=g)
    best = noisy.topk(K, dim=1)
    gl = torch.rand(N, generator=g) - 0.3
    buf = buf.to(DEV)
    return (buf[base:].view(N, ld)[:, :V], best.indices.int().to(DEV), best.values.to(DEV), gl.to(DEV))


def check_all(z, idx, y, gl, T=1.0, n_valid=None):
    """The three calls against the formulas; returns the step's outputs."""
    loss, ltol, stats, grad, gtol = reference(z, idx, y, T, n_valid, gl)
    kw = dict(n_valid=n_valid, temperature=T)
    keep = z.clone()
    l1, s1 = dh.distill_topk(z, idx, y, **kw)
    g1 = dh.distill_topk_backward(z, idx, y, s1, gl, **kw)
    l2, g2 = dh.distill_topk_step(z, idx, y, gl, **kw)
    torch.cuda.synchronize()
    assert torch.equal(z, keep)
    u = torch.finfo(z.dtype).eps / 2
    for l in (l1, l2):
        l = l.double().cpu().numpy()
        assert np.array_equal(np.isinf(l), np.isinf(loss))
        f = np.isfinite(loss)
        bad = np.abs(l[f] - loss[f]) > ltol[f]
        assert not bad.any(), (np.abs(l[f] - loss[f])[bad], ltol[f][bad])
    st = s1.double().cpu().numpy()
    np.testing.assert_array_equal(st[:, 0], stats[:, 0])
    x = np.where(np.isfinite(z.double().cpu().numpy()), (stats[:, :1] - z.double().cpu().numpy()) / T, 0.0)
    x = np.where(np.isfinite(x), x, 0.0)
    with np.errstate(invalid="ignore"):
        dev = (np.exp(-x) * (1 + np.abs(x))).sum(axis=1)
    assert (np.abs(st[:, 1] - stats[:, 1]) <= 2.0 ** -20 * dev).all()
    for g in (g1, g2):
        assert g.dtype == z.dtype and g.shape == z.shape
        err = np.abs(g.double().cpu().numpy() - grad)
        tol = gtol + u * np.abs(grad) + 1e-37
        assert (err <= tol).all(), (np.argwhere(err > tol)[:4], err.max())
    return l2, g2


def near(got, want, z, idx, y, gl):
    """Two results of one gradient, by other orders of the sums: each is within its bound of the
    formula's, so they are within twice that of one another."""
    _, _, _, grad, gtol = reference(z, idx, y, 1.0, None, gl)
    u = torch.finfo(z.dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - want.double().cpu().numpy())
    return (err <= 2 * (gtol + u * np.abs(grad) + 1e-37)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,K,T", [(1, 1, 1, 1.0), (1, 7, 3, 1.0), (2, 8, 8, 2.0), (5, 1000, 16, 0.5),
                                     (3, 1024, 1, 1.0), (3, 1025, 33, 1.0), (4, 4096, 16, 1.0), (2, 8200, 200, 3.0),
                                     (2, 50257, 50, 1.0), (1, 151936, 64, 1.0)])
def test_sizes(N, V, K, T, dtype):
    check_all(*make(N, V, K, dtype, seed=V + K), T=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,ld,base", [(1001, 1001, 0), (1001, 1001, 1), (1001, 1008, 0), (1000, 1011, 3),
                                       (4096, 4096, 5), (2047, 2050, 2), (9, 11, 1), (5, 5, 3)])
def test_strides_and_alignment(V, ld, base, dtype):
    """Rows at every offset from 16 bytes; what lies between and around them stays."""
    N, K = 9, min(V, 12)
    z, idx, y, gl = make(N, V, K, dtype, seed=V + ld, ld=ld, base=base)
    check_all(z, idx, y, gl)
    # the gradient into rows that lie differently
    for gbase, gld in ((0, V), (1, V + 3), (4, V + 8)):
        out = torch.full((gbase + N * gld + 3,), 55.0, dtype=z.dtype, device=DEV)
        rows = out[gbase:gbase + N * gld].view(N, gld)[:, :V]
        want = dh.distill_topk_step(z, idx, y, gl)[1]
        _, got = dh.distill_topk_step(z, idx, y, gl, grad_out=rows)
        torch.cuda.synchronize()
        assert got.data_ptr() == rows.data_ptr()
        assert near(got, want, z, idx, y, gl)
        rest = out.clone()
        rest[gbase:gbase + N * gld].view(N, gld)[:, :V] = 55.0
        assert (rest == 55.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,ld", [(3, 4096, 4096), (3, 1001, 1001), (2, 151936, 151936), (40, 5000, 5008),
                                    (1, 300001, 300001)])
def test_in_place(N, V, ld, dtype):
    z, idx, y, gl = make(N, V, 24, dtype, seed=3, ld=ld)
    want_l, want_g = dh.distill_topk_step(z, idx, y, gl)
    loss, stats = dh.distill_topk(z, idx, y)
    keep = z.clone()
    a = z.clone() if ld == V else torch.as_strided(z.clone().new_zeros(N * ld), (N, V), (ld, 1)).copy_(z)
    b = a.clone()
    got_l, got_g = dh.distill_topk_step(a, idx, y, gl, grad_out=a)
    bg = dh.distill_topk_backward(b, idx, y, stats, gl, grad_out=b)
    torch.cuda.synchronize()
    assert got_g.data_ptr() == a.data_ptr()
    assert near(got_g, want_g, keep, idx, y, gl) and near(bg, want_g, keep, idx, y, gl)
    ref, ltol = reference(keep, idx, y, 1.0)[:2]
    for l in (want_l, got_l, loss):
        assert (np.abs(l.double().cpu().numpy() - ref) <= ltol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_entries_left_out_repeated_and_short(dtype):
    """Ids outside the vocabulary, the same id several times (the gradient takes their sum), short
    and empty teachers, values of -inf, weights of 0."""
    N, V, K = 8, 3000, 40
    z, idx, y, gl = make(N, V, K, dtype, seed=11)
    idx[0, 3], idx[0, 7], idx[1, 0], idx[1, 39] = -1, V, -2 ** 31, 2 ** 31 - 1
    idx[2] = 17                      # one id throughout
    idx[3, 1::2] = idx[3, ::2]       # pairs
    idx[4] = -5                      # none
    y[5, 10:] = -float("inf")
    y[6] = -float("inf")
    gl[7] = 0.0
    nv = torch.tensor([40, 40, 13, 40, 40, 20, 40, 40], dtype=torch.int32, device=DEV)
    loss, grad = check_all(z, idx, y, gl, T=1.25, n_valid=nv)
    assert loss[4] == 0 and loss[6] == 0 and (grad[4] == 0).all() and (grad[6] == 0).all()
    assert loss[7] != 0 and (grad[7] == 0).all()
    # counts beyond [0, K] are clamped
    far = torch.tensor([99, 40, 13, 2 ** 31 - 1, -3, 20, -2 ** 31, 40], dtype=torch.int32, device=DEV)
    l2, _ = dh.distill_topk_step(z, idx, y, gl, n_valid=far, temperature=1.25)
    assert torch.equal(l2, loss)


def test_rows_without_weight_or_entries_do_not_read_their_logits():
    z, idx, y, gl = make(4, 5000, 8, "f32", seed=5)
    _, stats = dh.distill_topk(z, idx, y)
    loss, _ = dh.distill_topk_step(z, idx, y, gl)
    bad = z.clone()
    bad[1], bad[2] = float("nan"), float("inf")
    gl[1] = 0.0
    nv = torch.tensor([8, 8, 0, 8], dtype=torch.int32, device=DEV)
    g = dh.distill_topk_backward(bad, idx, y, stats, gl, n_valid=nv)
    l2, g2 = dh.distill_topk_step(bad, idx, y, gl, n_valid=nv)
    torch.cuda.synchronize()
    for x in (g, g2):
        assert (x[1:3] == 0).all() and torch.isfinite(x).all()
    assert l2[2] == 0 and torch.isnan(l2[1]) and torch.equal(l2[[0, 3]], loss[[0, 3]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_logits(dtype):
    """-inf and the type's lowest value in masked places; a row in which nothing is left."""
    N, V, K = 6, 2500, 20
    z, idx, y, gl = make(N, V, K, dtype, seed=13)
    low = torch.finfo(DT[dtype]).min
    keep = torch.zeros(V, dtype=torch.bool, device=DEV)
    for n in range(5):
        keep[:] = False
        keep[idx[n].long()] = True
        z[n, ~keep & (torch.arange(V, device=DEV) % 3 != 0)] = -float("inf") if n % 2 else low
    z[1, :1024] = torch.where(keep[:1024], z[1, :1024], torch.full_like(z[1, :1024], -float("inf")))
    z[3, idx[3, 0].long()] = -float("inf")   # the teacher's best is masked: infinite loss
    z[5] = -float("inf")                     # nothing left
    loss, grad = check_all(z, idx, y, gl)
    assert torch.isinf(loss[3]) and torch.isinf(loss[5]) and torch.isfinite(grad).all()


def test_nan_and_inf_stay_in_their_rows():
    z, idx, y, gl = make(8, 3000, 16, "f32", seed=17)
    gl[:] = 1.0
    want_l, want_g = dh.distill_topk_step(z, idx, y, gl)
    z[1, 2999], z[2, 5], y[4, 3], y[5, 0] = float("nan"), float("inf"), float("nan"), float("inf")
    z[6] = float("nan")
    fwd, stats = dh.distill_topk(z, idx, y)
    l, g = dh.distill_topk_step(z, idx, y, gl)
    back = dh.distill_topk_backward(z, idx, y, stats, gl)
    torch.cuda.synchronize()
    for n in (1, 2, 4, 5, 6):
        assert torch.isnan(l[n]) and torch.isnan(fwd[n]) and torch.isnan(back[n]).all() and torch.isnan(g[n]).all()
    for n in (1, 2, 6):
        assert torch.isnan(stats[n, 1])
    for n in (0, 3, 7):
        assert torch.equal(l[n], want_l[n]) and torch.equal(g[n], want_g[n])
        assert torch.isfinite(fwd[n]) and torch.isfinite(back[n]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,K", [(2, 1024, 1024), (3, 40000, 1024), (200, 20001, 257), (2, 2 ** 21, 40)])
def test_the_largest_teachers_and_vocabularies(N, V, K, dtype):
    z, idx, y, gl = make(N, V, K, dtype, seed=K)
    check_all(z, idx, y, gl)
    idx[:, 1::3] = idx[:, ::3][:, :idx[:, 1::3].shape[1]]  # repeated ids in a long list
    check_all(z, idx, y, gl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(152, 12000), (160, 30000), (310, 33000), (77, 151936)])
def test_more_rows_than_clusters_run_at_once(N, V, dtype):
    """The forms that walk several rows per block: ragged teachers, weights of 0, packed odd rows."""
    z, idx, y, gl = make(N, V + 1, 6, dtype, seed=N)
    gl[::7] = 0.0
    nv = (torch.arange(N, device=DEV) % 7).int()
    check_all(z, idx, y, gl, n_valid=nv)


def test_offsets_beyond_32_bits():
    """Rows 2.4 GB apart."""
    N, V, ld = 3, 5000, 1_200_000_000
    small, idx, y, gl = make(N, V, 8, "bf16", seed=47)
    z = torch.empty(N * ld, dtype=torch.bfloat16, device=DEV).view(N, ld)[:, :V]
    z.copy_(small)
    want = dh.distill_topk_step(small, idx, y, gl)
    out = torch.empty(N * ld, dtype=torch.bfloat16, device=DEV).view(N, ld)[:, :V]
    got = dh.distill_topk_step(z, idx, y, gl, grad_out=out)
    back = dh.distill_topk_backward(z, idx, y, dh.distill_topk(z, idx, y)[1], gl)
    assert got[1].stride(0) == ld and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert near(back, want[1], small, idx, y, gl)
    wide = make(N, 40000, 8, "bf16", seed=48)  # the form for long rows
    z = torch.empty(N * ld, dtype=torch.bfloat16, device=DEV).view(N, ld)[:, :40000]
    z.copy_(wide[0])
    got = dh.distill_topk_step(z, *wide[1:], grad_out=z)
    want = dh.distill_topk_step(wide[0], *wide[1:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1e-18, 1e18, 1e-3, 1e3])
def test_extreme_temperatures(T):
    z, idx, y, gl = make(3, 9000, 12, "f32", seed=53)
    loss, grad = dh.distill_topk_step(z, idx, y, gl, temperature=T)
    ref = reference(z, idx, y, float(np.float32(T)), None, gl)
    assert torch.isfinite(loss).all() and torch.isfinite(grad).all()
    # terms below 2^-126 of the largest are flushed; the rest within the bounds
    assert (np.abs(loss.double().cpu().numpy() - ref[0]) <= ref[1] + 1e-37).all()
    g = grad.double().cpu().numpy()
    assert (np.abs(g - ref[3]) <= ref[4] + 2.0 ** -24 * np.abs(ref[3]) + 2.0 ** -120 * abs(T) + 1e-37).all()


@pytest.mark.parametrize("std", [0.0, 30.0, 1e4])
def test_flat_and_peaked_rows(std):
    check_all(*make(3, 6000, 32, "f32", seed=19, std=std))
    check_all(*make(3, 6000, 32, "bf16", seed=19, std=std))


def test_shared_rows_and_results_repeat():
    """One row read for several (stride 0), and bits that do not change from call to call."""
    z, idx, y, gl = make(1, 40000, 16, "bf16", seed=23)
    rows = z.expand(5, -1)
    i5, y5, g5 = idx.expand(5, -1).contiguous(), y.expand(5, -1).contiguous(), gl.expand(5).contiguous()
    l, g = check_all(rows, i5, y5, g5)
    for n in range(5):
        assert torch.equal(l[n], l[0]) and torch.equal(g[n], g[0])
    l2, g2 = dh.distill_topk_step(rows, i5, y5, g5)
    assert torch.equal(l, l2) and torch.equal(g, g2)


def test_many_rows():
    """More rows than blocks of the launch, each like its own call."""
    z, idx, y, gl = make(3000, 500, 5, "bf16", seed=29)
    l, g = dh.distill_topk_step(z, idx, y, gl)
    ref = reference(z, idx, y, 1.0, None, gl)
    assert (np.abs(l.double().cpu().numpy() - ref[0]) <= ref[1]).all()
    assert (np.abs(g.double().cpu().numpy() - ref[3]) <= ref[4] + 2.0 ** -8 * np.abs(ref[3]) + 1e-37).all()
    assert torch.equal(dh.distill_topk_step(z[2999:], idx[2999:], y[2999:], gl[2999:])[1][0], g[2999])


def test_autograd_against_differences():
    """The gradient of the differentiable form against central differences of the loss in 64 bits."""
    z, idx, y, gl = make(2, 40, 6, "f32", seed=31)
    idx[1, 2] = idx[1, 1]
    T = 1.5
    leaf = z.clone().requires_grad_(True)
    loss = distill.distill_loss(leaf, idx, y, temperature=T)
    (loss * gl).sum().backward()
    h = 1e-5
    z64 = z.double().cpu()
    for n in range(2):
        for v in range(40):
            d = []
            for sgn in (1, -1):
                zz = z64.clone()
                zz[n, v] += sgn * h
                d.append(reference(zz, idx, y, T)[0][n])
            num = float(gl[n]) * (d[0] - d[1]) / (2 * h)
            # differences: h^2 times a third derivative (below 1) and 2^-52 |loss| / h
            assert abs(float(leaf.grad[n, v]) - num) <= 1e-8 + E * 8


def test_autograd_shapes_and_broadcast():
    """Leading dimensions, a broadcast input (its gradient is the rows' sum), rows without grad."""
    z, idx, y, _ = make(1, 300, 4, "f32", seed=37)
    leaf = z[0].clone().requires_grad_(True)
    i6, y6 = idx.expand(6, -1).reshape(2, 3, 4).contiguous(), y.expand(6, -1).reshape(2, 3, 4).contiguous()
    loss = distill.distill_loss(leaf.expand(2, 3, 300), i6, y6)
    assert loss.shape == (2, 3)
    w = torch.arange(6, device=DEV, dtype=torch.float32).view(2, 3)
    (loss * w).sum().backward()
    _, _, _, grad, gtol = reference(z, idx, y, 1.0)
    # the six rows' weights add up to 15; their sums' roundings (2^-24 each) are far below the bound
    err = np.abs(leaf.grad.double().cpu().numpy() - 15 * grad[0])
    assert (err <= 16 * gtol[0] + 15 * 2.0 ** -22 * np.abs(grad[0])).all()
    with torch.no_grad():
        assert torch.equal(distill.distill_loss(leaf.expand(2, 3, 300), i6, y6), loss.detach())


def test_graph_capture_and_streams():
    """Two graphs captured one after the other and replayed together share no scratch; calls on a
    stream of their own give the same bits; the autograd form refuses a capture."""
    a, b = make(16, 20000, 16, "bf16", seed=41), make(16, 20000, 16, "bf16", seed=43)
    want = [dh.distill_topk_step(*x) for x in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dh.distill_topk_step(*x))
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
    s1.wait_stream(torch.cuda.current_stream())
    l, g = dh.distill_topk_step(*a, stream=s1)
    s1.synchronize()
    assert torch.equal(l, want[0][0]) and torch.equal(g, want[0][1])
    leaf = a[0].clone().requires_grad_(True)
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="distill_topk_step"):
        with torch.cuda.graph(g):
            distill.distill_loss(leaf, a[1], a[2])


def test_explicit_workspace_grows_and_serves_both_calls():
    ws = dh.Workspace()
    for N in (2, 64, 3):
        z, idx, y, gl = make(N, 9000, 8, "bf16", seed=N)
        want = dh.distill_topk_step(z, idx, y, gl)
        got = dh.distill_topk_step(z, idx, y, gl, workspace=ws)
        l, _ = dh.distill_topk(z, idx, y, workspace=ws)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        assert torch.equal(l, dh.distill_topk(z, idx, y)[0])


def test_refusals():
    z, idx, y, gl = make(4, 100, 5, "f32", seed=1)
    step = lambda **k: dh.distill_topk_step(*[k.get(n, v) for n, v in  # noqa: E731
                                              (("z", z), ("idx", idx), ("y", y), ("gl", gl))],
                                            **{n: v for n, v in k.items() if n not in ("z", "idx", "y", "gl")})
    with pytest.raises(TypeError):
        step(z=z.half())
    for bad in (dict(z=z[0]), dict(z=z.t()), dict(idx=idx.long()), dict(idx=idx[:3]), dict(y=y.double()),
                dict(y=y[:, :4]), dict(gl=gl[:3]), dict(gl=gl.cpu()), dict(n_valid=torch.ones(4, device=DEV)),
                dict(grad_out=z.bfloat16()), dict(grad_out=torch.empty(100, 4, device=DEV).t()),
                dict(grad_out=z[:1].expand(4, 100)), dict(idx=idx[:, ::2])):
        with pytest.raises(ValueError):
            step(**bad)
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        with pytest.raises(dh.DhError) as e:
            step(temperature=T)
        assert e.value.status == 1
    big = torch.zeros(8, 100, device=DEV)
    with pytest.raises(dh.DhError):  # partly the same memory
        step(z=big[:4], grad_out=big[1:5])
    with pytest.raises(dh.DhError):
        dh.distill_topk(z, torch.zeros(4, 1025, dtype=torch.int32, device=DEV), torch.zeros(4, 1025, device=DEV))
    empty = dh.distill_topk_step(z[:0], idx[:0], y[:0], gl[:0])
    assert empty[0].shape == (0,) and empty[1].shape == (0, 100)


def test_teacher_from_the_draft_head():
    """The candidate head's own training: exact candidates and logits of the full-rank head teach
    the low-rank scores, and the gradient flows on to U and V as the formulas say."""
    cfg = inputs.head_config("tiny", B=4)
    x = inputs.make_head(cfg, seed=2, device=DEV)
    idx, _, exact, _ = dh.draft_head(x["h"], x["U"], x["V"], x["W"], cfg.K)
    U, V = x["U"].clone().requires_grad_(True), x["V"].clone().requires_grad_(True)
    loss = distill.distill_loss((x["h"] @ U) @ V, idx, exact)
    loss.mean().backward()
    U64, V64 = x["U"].double().requires_grad_(True), x["V"].double().requires_grad_(True)
    logq = torch.log_softmax((x["h"].double() @ U64) @ V64, dim=1)
    logp = torch.log_softmax(exact.double(), dim=1)
    ref = (logp.exp() * (logp - logq.gather(1, idx.long()))).sum(1)
    ref.mean().backward()
    assert torch.allclose(loss.double(), ref, rtol=1e-4, atol=1e-4)
    for got, want in ((U.grad, U64.grad), (V.grad, V64.grad)):
        assert (got.double() - want).norm() <= 1e-3 * want.norm()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,ld", [(5000, 5008), (5000, 50003), (40000, 4000001), (1001, 1001)])
def test_memory_of_the_gradient(V, ld, dtype):
    """Rows far apart (one position of many) do not make the gradient as large as what they lie in, and
    its rows still lie like theirs."""
    N = 6
    small, idx, y, gl = make(N, V, 8, dtype, seed=53)
    z = torch.empty(N * ld, dtype=small.dtype, device=DEV).view(N, ld)[:, :V]
    z.copy_(small)
    stats = dh.distill_topk(small, idx, y)[1]
    want = dh.distill_topk_step(small, idx, y, gl)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = dh.distill_topk_step(z, idx, y, gl)[1]
    back = dh.distill_topk_backward(z, idx, y, stats, gl)
    torch.cuda.synchronize()
    size = N * V * z.element_size()
    # two gradients of at most 9/8 of their rows and 16 bytes each, and small outputs and workspaces
    assert torch.cuda.max_memory_allocated() - before <= 2 * (size * 9 // 8 + N * 16) + (1 << 16)
    assert (got.stride(0) - ld) * z.element_size() % 16 == 0 and (back.stride(0) - ld) * z.element_size() % 16 == 0
    assert near(got, want[1], small, idx, y, gl) and near(back, want[1], small, idx, y, gl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,K", [(1300, 500, 33), (300, 33001, 96), (40, 70000, 1024)])
def test_repeated_ids_of_many_rows(N, V, K, dtype):
    """Every row's ids repeat in another way: pairs held by one lane, by neighbouring and by far lanes."""
    z, idx, y, gl = make(N, V, K if K < V else V, dtype, seed=61)
    g = torch.Generator().manual_seed(67)
    pick = torch.stack([torch.randint(0, 1 + (n * 7) % K, (K,), generator=g) for n in range(N)]).to(DEV)
    idx = idx.gather(1, pick).contiguous()
    check_all(z, idx, y, gl)


@pytest.mark.parametrize("mode", [1, 2, 3])
@pytest.mark.parametrize("N,V", [(400, 65540), (333, 40001)])  # rows held by two blocks and by one
def test_a_wait_that_gives_up_leaves_no_result(N, V, mode):
    """Something held back from a row on (the copies, a warp's statistics, its buffers): the status bit is
    raised, every row that shares its blocks is NaN in loss and gradient, the others are as ever, and the
    next call works."""
    z, idx, y, gl = make(N, V, 8, "f32", seed=59)
    gl[:] = 0.5
    want_l, want_g = dh.distill_topk_step(z, idx, y, gl)
    loss, grad, status = dh.selftest_distill_timeout(0, 0, 100000, z, idx, y, gl)
    assert status == 0 and torch.equal(loss, want_l) and torch.equal(grad, want_g)
    # a block that has no more rows to load waits for no buffer, so those are held back from the start
    for row in ((0,) if mode == 3 else (0, N - 5)):
        loss, grad, status = dh.selftest_distill_timeout(mode, row, 3000, z, idx, y, gl)
        assert status == 1 << 5
        lost = torch.isnan(loss)
        assert lost[row:].all() and torch.isnan(grad[lost]).all()
        assert torch.equal(loss[~lost], want_l[~lost]) and torch.equal(grad[~lost], want_g[~lost])
        if row:
            assert lost.sum() <= 5 * (N // 60)  # five groups of blocks, of 76 or 152
    again = dh.distill_topk_step(z, idx, y, gl)
    assert torch.equal(again[0], want_l) and torch.equal(again[1], want_g)
    with pytest.raises(TypeError):
        dh.selftest_distill_timeout(1, 0, 3000, z.bfloat16(), idx, y, gl)


@pytest.mark.parametrize("T", [1.0, 1.27])
@pytest.mark.parametrize("K", [512, 1024])
def test_small_losses(K, T):
    """Losses of a student near its teacher, the difference of two logarithms many times their size: the
    deviation over 512 rows.  With d = (max - z)/T, a = (max - y)/T and u = 2^-24 a row's error is, always
    the same way, u (E_q[d] + E_p[a]) by the factors 1/T (log2(e)/T alone at T = 1) and the 2^x unit's
    mean of 5.1e-8; and at random the roundings of the terms (u d and 1.5e-7 for q; 2 u a and four steps'
    half, 2^-22 for p), of two sums' trees (variance below two of u / sqrt 3 each) and of the losses'
    own terms p (a - d).  A quarter more for the deviation of the deviation."""
    N, u = 512, 2.0 ** -24
    g = torch.Generator().manual_seed(73)
    z = 0.3 * torch.randn(N, K, generator=g)
    y = z + 0.3 * torch.randn(N, K, generator=g)
    idx = torch.arange(K, dtype=torch.int32).expand(N, K).contiguous()
    loss, _ = dh.distill_topk(z.to(DEV), idx.to(DEV), y.to(DEV), temperature=T)
    t = np.float64(np.float32(T))
    d = (z.double().amax(1, keepdim=True) - z.double()).numpy() / t
    a = (y.double().amax(1, keepdim=True) - y.double()).numpy() / t
    q, p = np.exp(-d) / np.exp(-d).sum(1)[:, None], np.exp(-a) / np.exp(-a).sum(1)[:, None]
    logq, logp = -d - np.log(np.exp(-d).sum(1))[:, None], -a - np.log(np.exp(-a).sum(1))[:, None]
    want = (p * (logp - logq)).sum(1)
    f = u if T != 1.0 else abs(float(np.float32(np.log2(np.e))) / np.log2(np.e) - 1)
    always = f * ((q * d).sum(1) + (p * a).sum(1) * (T != 1.0)) + 5.1e-8
    var = ((q * q * ((u * d) ** 2 / 3 + 1.5e-7 ** 2)).sum(1) + (p * p * ((2 * u * a) ** 2 / 3 + 2.0 ** -44)).sum(1)
           + 4 * u * u / 3 + (p * p * (u * (a + d)) ** 2).sum(1) + (u * want) ** 2)
    err = loss.double().cpu().numpy() / (t * t) - want
    assert np.sqrt((err ** 2).mean()) <= 1.25 * np.sqrt((always ** 2 + var).mean())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,ld,base", [(5, 40001, 40001, 1), (5, 40001, 40004, 3), (1, 40000, 40000, 2),
                                         (3, 40001, 40001, 0), (4, 1001, 4000001, 5)])
def test_gradient_lies_like_logits_off_16_bytes(N, V, ld, base, dtype):
    """Logits that start anywhere (the rows behind the first of an odd vocabulary, a part of wider rows)
    get a gradient that starts at the same place of 16 bytes, and the results of contiguous ones."""
    z, idx, y, gl = make(N, V, 8, dtype, seed=79, ld=ld, base=base)
    got = dh.distill_topk_step(z, idx, y, gl)[1]
    back = dh.distill_topk_backward(z, idx, y, dh.distill_topk(z, idx, y)[1], gl)
    torch.cuda.synchronize()
    for x in (got, back):
        assert (x.data_ptr() - z.data_ptr()) % 16 == 0
        assert N == 1 or (x.stride(0) - ld) * x.element_size() % 16 == 0
        assert x.untyped_storage().nbytes() <= N * (V * 9 // 8 + 8) * x.element_size() + 16
        assert near(x, dh.distill_topk_step(z.contiguous(), idx, y, gl)[1], z, idx, y, gl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [900, 70001])
@pytest.mark.parametrize("T", [0.1, 0.5, 0.8])
def test_entries_at_the_lowest_value_below_one(T, V, dtype):
    """Logits masked by the type's lowest value at the teacher's entries, divided by a temperature below
    one: the quotient has no fp32, the loss (T^2 times it) has one, and a share near nothing leaves little."""
    N, K = 6, 24
    z, idx, y, gl = make(N, V, K, dtype, seed=83)
    low = torch.finfo(DT[dtype]).min
    col = lambda n, k: (n, idx[n, k].long())  # noqa: E731
    z[col(0, 0)] = low                         # the likeliest entry
    y[1, 5] = y[1].max() - 90.0 * T            # a share of e^-90
    z[col(1, 5)] = low
    z[2, idx[2].long()] = low                  # all entries
    z[3] = low                                 # the whole row: q is flat
    y[4, 5:] = -float("inf")                   # entries without a share, and an unlikely one
    z[4, idx[4, 5:].long()] = low
    y[4, 4] = y[4].max() - 40.0 * T
    z[col(4, 4)] = low
    ref = reference(z, idx, y, float(np.float32(T)))[0]
    assert np.isfinite(ref).all() and (ref < 3.4e38).all() and ref[0] > 1e36 and ref[1] < 100
    loss, grad = check_all(z, idx, y, gl, T=float(np.float32(T)))
    assert torch.isfinite(loss).all() and torch.isfinite(grad).all()
    z[col(0, 0)] = -float("inf")
    assert torch.isinf(dh.distill_topk(z, idx, y, temperature=T)[0][0])


def test_entries_at_the_lowest_value_at_their_limits():
    """Shares that round up, at losses next to the largest fp32, and shares below the normal numbers."""
    low = torch.finfo(torch.float32).min
    for seed, N, V, K, T in ((89, 200, 197, 140, 0.1), (97, 60, 1290, 7, 0.1), (101, 60, 9000, 40, 0.25)):
        z, idx, y, gl = make(N, V, K, "f32", seed=seed)
        n = torch.arange(N, device=DEV)
        best = y.argmax(dim=1)
        z[n[::2], idx[n[::2], best[::2]].long()] = low           # the whole share of some rows, nearly
        for m in range(1, N, 2):                                  # e^-88 to e^-103 in the others
            k = int((best[m] + 1) % K)
            y[m, k] = y[m, best[m]] - (88.0 + 15.0 * m / N) * T
            z[m, idx[m, k].long()] = low
        t = float(np.float32(T))
        assert (reference(z, idx, y, t)[0] < 3.4e38).all()
        loss, _ = check_all(z, idx, y, gl, T=t)
        assert torch.isfinite(loss).all()
