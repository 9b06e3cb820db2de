"""Layer norm (dh_layer_norm, dh_layer_norm_backward) against the formulas in 64 bits.

fp32 sums: a row's sum passes through at most `steps(d)` additions (a thread's own elements one after another, then
trees over lanes and warps), so it is off by steps 2^-24 of the sum of the terms' sizes.  Forward: the second pass
corrects the mean, so that it and the variance carry such errors of the deviations, not of the values.  Backward: the
reference takes the same fp32 statistics, so their rounding is no error."""
import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding as dh

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


def steps(d):
    return max(16, -(-d // 1024)) + 10


def matrix(n, d, dtype, seed=0, ld=None, base=0, shift=0.0, std=1.0):
    """n rows of d random values, in memory whose other elements are NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ld = d if ld is None else ld
    buf = torch.full((base + max(n, 1) * ld,), float("nan"), dtype=DT[dtype], device=DEV)
    view = buf[base:base + n * ld].view(n, ld)[:, :d]
    view.copy_((shift + std * torch.randn(n, d, generator=g, device=DEV)).to(DT[dtype]))
    return view


def params(d, dtype, seed=0, base=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 77)
    make = lambda c, s: torch.cat([torch.zeros(base, device=DEV), c + s * torch.randn(d, generator=g, device=DEV)]  # noqa: E731
                                  ).to(DT[dtype])[base:]
    return make(1.0, 0.3), make(0.0, 0.2)


def check_forward(x, w, b, eps=1e-5, **kw):
    X = x.double()
    mean = X.mean(1, keepdim=True)
    dev = X - mean
    var = (dev * dev).mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    hat = dev * rstd
    W = 1.0 if w is None else w.double()
    B = 0.0 if b is None else b.double()
    want = hat * W + B
    n = steps(x.shape[1]) + 4
    # the mean, in units of the deviations' mean size (and its own rounding to fp32 when it is stated)
    e_mean = 2 * n * U * dev.abs().mean(1, keepdim=True) + (n * U) ** 2 * X.abs().mean(1, keepdim=True)
    e_rstd = rstd * (n + 6) * U  # half of the variance's (2 n + 4) 2^-24, the root's and the division's
    y, stats = dh.layer_norm(x, w, b, eps=eps, with_stats=True, **kw)
    torch.cuda.synchronize()
    Wa = W.abs() if torch.is_tensor(W) else W
    Ba = B.abs() if torch.is_tensor(B) else B
    # x - mean - delta, times rstd and weight: four roundings of the product, one of the sum with the bias
    bound = Wa * (rstd * e_mean + dev.abs() * e_rstd + 4 * U * hat.abs()) + U * (want.abs() + Ba)
    # x - mean0 is rounded too, where mean0 differs from the mean by its own error of the values
    bound = bound + Wa * rstd * U * n * U * X.abs().mean(1, keepdim=True)
    bound = bound * 1.01 + torch.finfo(x.dtype).eps / 2 * (want.abs() + bound)
    off = (y.double() - want).abs() - bound
    assert (off <= 0).all(), (off.max(), want.abs().max())
    assert ((stats[:, :1].double() - mean).abs() <= e_mean * 1.01 + U * mean.abs() * 2).all()
    assert ((stats[:, 1:].double() - rstd).abs() <= e_rstd * 1.01).all()
    return y, stats


def check_backward(g, x, stats, w, ptype, **kw):
    N, d = x.shape
    X, G, m, r = x.double(), g.double(), stats[:, :1].double(), stats[:, 1:].double()
    hat = (X - m) * r
    h = G if w is None else G * w.double()
    c1, c2 = h.mean(1, keepdim=True), (h * hat).mean(1, keepdim=True)
    want = r * (h - c1 - hat * c2)
    n = steps(d) + 4
    bound = r.abs() * (n * U * (h.abs().mean(1, keepdim=True) + hat.abs() * (h * hat).abs().mean(1, keepdim=True))
                       + 6 * U * (h.abs() + c1.abs() + (hat * c2).abs()))
    bound = bound * 1.01 + torch.finfo(x.dtype).eps / 2 * (want.abs() + bound)
    dx, dw, db = dh.layer_norm_backward(g, x, stats, w, param_dtype=None if w is not None else DT[ptype], **kw)
    torch.cuda.synchronize()
    if dx is not None:
        off = (dx.double() - want).abs() - bound
        assert (off <= 0).all(), off.max()
    # a column's sum: a block's rows one after another, then the blocks' sums and a few more
    L = min(N, -(-N // 152) + 80) + 4
    for got, terms in ((dw, G * hat), (db, G)):
        if got is None:
            continue
        want, size = terms.sum(0), terms.abs().sum(0)
        bound = L * U * size
        bound = bound + torch.finfo(got.dtype).eps / 2 * (want.abs() + bound)
        assert got.dtype == DT[ptype] and ((got.double() - want).abs() <= bound * 1.01).all()
    return dx, dw, db


SIZES = [(1, 1), (3, 2), (5, 8), (2, 31), (9, 64), (33, 257), (4, 1000), (7, 1001), (6, 1024), (3, 1025), (11, 2048),
         (3, 4097), (8, 5120), (4, 8192), (3, 8193), (2, 20000), (2, 65536), (700, 128), (2500, 100), (1300, 640)]


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("N,d", SIZES)
def test_sizes(N, d, dtype, ptype):
    x, g = matrix(N, d, dtype, seed=d, shift=0.5), matrix(N, d, dtype, seed=d + 1)
    w, b = params(d, ptype)
    _, stats = check_forward(x, w, b)
    check_backward(g, x, stats, w, ptype)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_forward(x, ww, bb)
    check_backward(g, x, stats, None, ptype)


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("d,ld,base", [(64, 72, 0), (64, 64, 1), (65, 65, 0), (640, 643, 3), (5120, 5128, 0),
                                       (5120, 5121, 2), (1001, 1001, 1), (9000, 9001, 1)])
def test_strides_and_alignment(d, ld, base, dtype, ptype):
    N = 19
    x, g = matrix(N, d, dtype, 1, ld, base, shift=-1.0), matrix(N, d, dtype, 2, ld, base)
    w, b = params(d, ptype, base=base)
    out, into = matrix(N, d, dtype, 3, ld, base), matrix(N, d, dtype, 4, ld, base)
    y, stats = check_forward(x, w, b, out=out)
    assert y is out
    check_backward(g, x, stats, w, ptype, grad_x=into)
    for t in (out, into):  # what lies between the rows stays
        if ld > d:
            assert t.as_strided((N - 1, ld - d), (ld, 1), t.storage_offset() + d).isnan().all()
    # one row for all, and in place
    same = x[:1].expand(N, d)
    y, st = check_forward(same, w, b)
    assert (y == y[0]).all() and (st == st[0]).all()
    want = dh.layer_norm(x, w, b)[0].clone()
    for into in ("x", "grad"):
        xx, gg = matrix(N, d, dtype, 1, ld, base, shift=-1.0), matrix(N, d, dtype, 2, ld, base)
        dx = dh.layer_norm_backward(gg, xx, stats, w)[0].clone()
        got = dh.layer_norm_backward(gg, xx, stats, w, grad_x=xx if into == "x" else gg)
        assert torch.equal(got[0], dx)
    xx = matrix(N, d, dtype, 1, ld, base, shift=-1.0)
    assert torch.equal(dh.layer_norm(xx, w, b, out=xx)[0], want)


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("N,d", [(5000, 64), (1500, 1001), (2000, 5120), (20011, 40), (700, 9000)])
def test_many_rows(N, d, dtype, ptype):
    x, g = matrix(N, d, dtype, 5), matrix(N, d, dtype, 6)
    w, b = params(d, ptype)
    _, stats = check_forward(x, w, b)
    a = check_backward(g, x, stats, w, ptype)
    again = dh.layer_norm_backward(g, x, stats, w)
    assert all(torch.equal(p, q) for p, q in zip(a, again))


@pytest.mark.parametrize("shift,std", [(1e4, 1.0), (-3e5, 0.5), (1e-6, 1e-7), (0.0, 1e15), (1e18, 1e12)])
@pytest.mark.parametrize("d", [100, 1000, 5120, 10000])
def test_means_far_from_zero(d, shift, std):
    check_forward(matrix(9, d, "f32", 7, shift=shift, std=std), None, None, eps=1e-5 if std < 1e9 else 0.0)


def test_constant_rows():
    """No variance: rstd is 1 / sqrt(eps), y the bias; without eps the row is NaN, as 0 / 0 is."""
    for d in (7, 640, 5120, 9000):
        x = torch.full((3, d), 2.75, device=DEV)
        w, b = params(d, "f32")
        y, stats = dh.layer_norm(x, w, b, eps=1e-5, with_stats=True)
        assert torch.equal(y, b.expand(3, d)) and (stats[:, 0] == 2.75).all()
        assert (stats[:, 1] - 1e-5 ** -0.5).abs().max() <= 1e-4
        assert dh.layer_norm(x, eps=0.0)[0].isnan().all()


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("d", [40, 1000, 5120, 9000])
def test_nan_and_inf_stay_in_their_rows(d, dtype, ptype):
    x, g = matrix(30, d, dtype, 8), matrix(30, d, dtype, 9)
    w, b = params(d, ptype)
    clean, st0 = dh.layer_norm(x, w, b, with_stats=True)
    dx0 = dh.layer_norm_backward(g, x, st0, w)[0].clone()
    clean = clean.clone()
    x[3, d // 2], x[11, 0] = float("nan"), float("inf")
    y, stats = dh.layer_norm(x, w, b, with_stats=True)
    good = torch.ones(30, dtype=torch.bool, device=DEV)
    good[3] = good[11] = False
    assert y[~good].isnan().all() and torch.equal(y[good], clean[good])
    dx, dw, db = dh.layer_norm_backward(g, x, stats, w)
    assert dx[~good].isnan().all() and torch.equal(dx[good], dx0[good])
    assert dw.isnan().all() and db.isfinite().all()


def test_offsets_beyond_32_bits():
    d, ld = 100, (1 << 31) + 8
    buf = torch.zeros(2 * ld + d, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, d), (ld, 1))
    x.copy_(matrix(3, d, "bf16", 3))
    w, b = params(d, "bf16")
    _, stats = check_forward(x, w, b)
    check_backward(matrix(3, d, "bf16", 4), x, stats, w, "bf16")
    dh.layer_norm(x, w, b, out=x)
    assert torch.equal(x, dh.layer_norm(matrix(3, d, "bf16", 3), w, b)[0])


@pytest.mark.parametrize("d", [24, 1000, 9000])
def test_only_what_is_wanted(d):
    N = 50
    x, g = matrix(N, d, "f32", 1), matrix(N, d, "f32", 2)
    w, b = params(d, "f32")
    y, none = dh.layer_norm(x, w, b)
    assert none is None and torch.equal(y, dh.layer_norm(x, w, b, with_stats=True)[0])
    stats = dh.layer_norm(x, w, b, with_stats=True)[1]
    full = dh.layer_norm_backward(g, x, stats, w)
    for i in range(8):
        want = [bool(i & 1), bool(i & 2), bool(i & 4)]
        got = dh.layer_norm_backward(g, x, stats, w, with_x=want[0], with_weight=want[1], with_bias=want[2])
        for q, p, k in zip(got, full, want):
            assert (q is None) == (not k) and (q is None or torch.equal(q, p))
    # against differences of the forward pass in 64 bits
    X, G, W = x[:3].double(), g[:3].double(), w.double()

    def f(v, ww):
        m = v.mean(1, keepdim=True)
        return (((v - m) / ((v - m) ** 2).mean(1, keepdim=True).add(1e-5).sqrt() * ww + b.double()) * G).sum()
    dx, dw, _ = dh.layer_norm_backward(g[:3].contiguous(), x[:3].contiguous(), stats[:3].contiguous(), w)
    for at in ((0, 0), (1, d // 2), (2, d - 1)):
        h = 1e-5
        e = torch.zeros_like(X)
        e[at] = h
        assert abs((f(X + e, W) - f(X - e, W)) / (2 * h) - dx[at]) <= 1e-4 * (1 + abs(dx[at]))
        e = torch.zeros_like(W)
        e[at[1]] = h
        assert abs((f(X, W + e) - f(X, W - e)) / (2 * h) - dw[at[1]]) <= 1e-4 * (1 + abs(dw[at[1]]))


def test_empty_calls():
    x = matrix(0, 64, "f32")
    assert dh.layer_norm(x)[0].shape == (0, 64)
    w, _ = params(64, "f32")
    dx, dw, db = dh.layer_norm_backward(x, x, torch.empty(0, 2, device=DEV), w, grad_weight=torch.ones(64, device=DEV))
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_graphs_streams_and_a_workspace():
    N, d = 900, 1280
    x, g = matrix(N, d, "bf16", 1), matrix(N, d, "bf16", 2)
    w, b = params(d, "f32")
    y, stats = dh.layer_norm(x, w, b, with_stats=True)
    want = dh.layer_norm_backward(g, x, stats, w)
    ws = dh.Workspace()
    for n in (3, N, 40):
        a = dh.layer_norm_backward(g[:n], x[:n], stats[:n], w, workspace=ws)
        c = dh.layer_norm_backward(g[:n], x[:n], stats[:n], w)
        assert all(torch.equal(p, q) for p, q in zip(a, c))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ys, _ = dh.layer_norm(x, w, b, stream=s)
    a = dh.layer_norm_backward(g, x, stats, w, stream=s)
    s.synchronize()
    assert torch.equal(ys, y) and all(torch.equal(p, q) for p, q in zip(a, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, st = dh.layer_norm(x, w, b, with_stats=True)
        out = dh.layer_norm_backward(g, x, st, w)
    x.copy_(matrix(N, d, "bf16", 11))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    y2, st2 = dh.layer_norm(x, w, b, with_stats=True)
    assert torch.equal(y, y2) and torch.equal(st, st2)
    assert all(torch.equal(p, q) for p, q in zip(out, dh.layer_norm_backward(g, x, st2, w)))


def test_refusals():
    x, (w, b) = matrix(4, 16, "f32"), params(16, "f32")
    stats = torch.zeros(4, 2, device=DEV)
    with pytest.raises(ValueError, match="adjacent"):
        dh.layer_norm(x.t())
    with pytest.raises(ValueError, match="weight must be"):
        dh.layer_norm(x, w[:8])
    with pytest.raises(ValueError, match="weight must be fp32"):
        dh.layer_norm(x, w.bfloat16())
    with pytest.raises(ValueError, match="share"):
        dh.layer_norm(x.bfloat16(), w, b.bfloat16())
    with pytest.raises(ValueError, match="out must be"):
        dh.layer_norm(x, out=x.bfloat16())
    with pytest.raises(ValueError, match="overlap"):
        dh.layer_norm(x, out=torch.empty(1, 16, device=DEV).expand(4, 16))
    with pytest.raises(dh.DhError, match="INVALID_ARG"):
        dh.layer_norm(x[:3], out=x[1:])
    with pytest.raises(dh.DhError, match="INVALID_ARG"):
        dh.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError, match="stats must be"):
        dh.layer_norm_backward(x, x, stats[:3])
    with pytest.raises(ValueError, match="grad_out must be"):
        dh.layer_norm_backward(x.bfloat16(), x, stats)
    with pytest.raises(ValueError, match="param_dtype"):
        dh.layer_norm_backward(x, x, stats, param_dtype=torch.bfloat16)
    with pytest.raises(dh.DhError, match="INVALID_ARG"):
        dh.layer_norm_backward(x[1:], x[:3].clone(), stats[:3], grad_x=x[:3])
    with pytest.raises(TypeError, match="dtype"):
        dh.layer_norm(x.half())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [5, 700])
@pytest.mark.parametrize("d", [1000, 1001, 5120, 8191, 8192, 9000])
@pytest.mark.parametrize("value", [30.0, 1e3, 3e4, 1e15])
def test_outliers(value, d, N, dtype):
    """One element, a thread's first vector or a warp's columns far above the others: the sums are as exact wherever in
    the row they stand, since they are taken about means, not about single elements."""
    places = [[0], range(4), range(8), [d - 1], [512], [1024], range(256, 260), range(512), range(d - 5, d), [3, d // 2]]
    for i, at in enumerate(places):
        at = [c for c in at if c < d]
        x = matrix(N, d, dtype, seed=i)
        x[:, at] = x[:, at].sign() * value if i % 2 else value
        w, b = params(d, dtype)
        check_forward(x, w, b)
    x = matrix(N, d, dtype, seed=20, ld=d + 3, base=1)  # off 16 bytes
    x[:, :8] = value
    check_forward(x, None, None)


def test_column_sums_over_many_rows():
    """One row many times over (a row stride of 0), so that every column adds up equal terms and roundings do not cancel:
    a share's rows are added 32 at a time in fp32 (31 roundings and the product's), those sums without further loss, and
    a few more roundings lead to the result."""
    for N, d, dtype in ((60000, 65536, "bf16"), (150000, 9001, "f32"), (150000, 8200, "bf16")):
        x, g = matrix(1, d, dtype, 1), matrix(1, d, dtype, 2)
        _, stats = dh.layer_norm(x, with_stats=True)
        dx, dw, db = dh.layer_norm_backward(g.expand(N, d), x.expand(N, d), stats.repeat(N, 1), with_x=False,
                                            param_dtype=torch.float32)
        hat = (x.double() - stats[:, :1].double()) * stats[:, 1:].double()
        for got, term in ((dw, g.double() * hat), (db, g.double())):
            off = (got.double() - N * term[0]).abs() / (N * term[0].abs()).clamp(min=1e-30)
            assert off.max() <= (32 + 8) * U, (N, d, dtype, off.max() / U)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [3, 700])
@pytest.mark.parametrize("d,k", [(7714, 8), (5656, 8), (7200, 2), (7711, 3), (1032, 4), (4104, 8), (545, 16)])
def test_outliers_in_a_short_last_warp(d, k, N, dtype):
    """The last columns are all that some warp has, and most of them are outliers."""
    for i, value in enumerate((3e3, 1e6, -1e9)):
        for ld, base in ((d, 0), (d + 1, 0), (d, 2)):
            x = matrix(N, d, dtype, i, ld, base)
            x[:, d - k:] = value
            check_forward(x, None, None)
