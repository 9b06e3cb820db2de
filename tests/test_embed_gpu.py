"""Embedding (dh_embed, dh_embed_backward).  The lookup is exact: one product in fp32, rounded once.  The gradient's
sums of L terms in fp32 are off by (L + 1) 2^-24 of the sum of the terms' sizes (the additions and the scaling), and
the result is rounded once more."""
import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding as dh

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def matrix(n, d, dtype, seed=0, ld=None, base=0):
    """n rows of d random values, in memory whose other elements are NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ld = d if ld is None else ld
    buf = torch.full((base + max(n, 1) * ld,), float("nan"), dtype=DT[dtype], device=DEV)
    view = buf[base:base + n * ld].view(n, ld)[:, :d]
    view.copy_(torch.randn(n, d, generator=g, device=DEV).to(DT[dtype]))
    return view


def tokens(N, V, kind="zipf", seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "zipf":
        t = (torch.rand(N, generator=g).double() * torch.log(torch.tensor(float(V)))).exp().int() - 1
    elif kind == "uniform":
        t = torch.randint(0, V, (N,), generator=g).int()
    elif kind == "one":
        t = torch.full((N,), V // 2, dtype=torch.int32)
    elif kind == "falling":
        t = (V - 1 - torch.arange(N) % V).int()
    elif kind == "padding":
        t = torch.full((N,), -1, dtype=torch.int32)
    else:  # padding and ids out of range among the others
        t = torch.randint(0, V, (N,), generator=g).int()
        t[::3] = -1
        t[1::7] = V
        t[4::11] = 2 ** 31 - 1
        t[5::13] = -2 ** 31
    return t.clamp(max=V - 1).to(DEV) if kind == "zipf" else t.to(DEV)


def forward(table, tok, scale):
    held = (tok >= 0) & (tok < table.shape[0])
    rows = table[torch.where(held, tok, 0).long()].float() * torch.tensor(scale, dtype=torch.float32)
    return torch.where(held[:, None], rows, torch.zeros_like(rows)).to(table.dtype)


def check_backward(grad, tok, V, scale=1.0, base=None, **kw):
    """`base`: what the gradient is added to."""
    N, d = grad.shape
    held = (tok >= 0) & (tok < V)
    t = tok[held].long()
    g = grad[held].double()
    want = torch.zeros(V, d, dtype=torch.float64, device=DEV).index_add_(0, t, g)
    size = torch.zeros(V, d, dtype=torch.float64, device=DEV).index_add_(0, t, g.abs())
    terms = torch.bincount(t, minlength=V)[:, None].double()
    scale = float(torch.tensor(scale, dtype=torch.float32))
    want, size = want * scale, size * abs(scale)
    bound = (terms + 1) * 2.0 ** -24 * size
    if base is not None:
        want = want + base.double()
        bound = bound + (terms > 0) * 2.0 ** -24 * want.abs() * 1.01
    got = dh.embed_backward(grad, tok, V, scale=scale, **kw)
    torch.cuda.synchronize()
    bound = bound * 1.001 + torch.finfo(grad.dtype).eps / 2 * (want.abs() + bound)
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), off.max()
    none = terms[:, 0] == 0
    assert torch.equal(got[none], (torch.zeros_like(got) if base is None else base)[none])
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,d", [(1, 1, 1), (3, 5, 7), (8, 1000, 8), (17, 333, 100), (100, 50, 1001), (5, 40, 5120),
                                   (2, 3, 65536), (5000, 700, 64), (1, 151936, 512)])
def test_lookup(N, V, d, dtype):
    table = matrix(V, d, dtype, seed=d)
    for kind, scale in (("zipf", 1.0), ("mixed", 0.37), ("uniform", 71.5)):
        tok = tokens(N, V, kind, seed=N)
        assert torch.equal(dh.embed(table, tok, scale=scale), forward(table, tok, scale))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,ld,base", [(64, 64, 0), (64, 64, 1), (64, 72, 0), (65, 65, 0), (64, 67, 3), (40, 0, 0)])
def test_strides_and_alignment(d, ld, base, dtype):
    V, N = 90, 300
    table = matrix(V, d, dtype, 1, ld, base) if ld else matrix(1, d, dtype, 1).expand(V, d)
    tok = tokens(N, V, "mixed", 3)
    want = forward(table, tok, 1.5)
    out = matrix(N, d, dtype, 2, ld or d, base)
    beside = out.as_strided((N, max(ld - d, 0)), (out.stride(0), 1), out.storage_offset() + d) if ld > d else None
    assert dh.embed(table, tok, scale=1.5, out=out) is out and torch.equal(out, want)
    grad = matrix(N, d, dtype, 4, ld, base) if ld else matrix(1, d, dtype, 4).expand(N, d)
    into = matrix(V, d, dtype, 5, ld or d, base)
    check_backward(grad, tok, V, 1.5, grad_table=into)
    if beside is not None:  # what lies between the rows stays
        assert beside[:-1].isnan().all()
        between = into.as_strided((V - 1, ld - d), (into.stride(0), 1), into.storage_offset() + d)
        assert between.isnan().all()
    was = into.clone()
    check_backward(grad, tok, V, 1.5, base=was, grad_table=into, accumulate=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["zipf", "uniform", "one", "falling", "padding", "mixed"])
@pytest.mark.parametrize("N,V,d", [(1, 1, 1), (7, 3, 33), (65, 1000, 128), (1000, 17, 40), (4096, 511, 24),
                                   (4097, 512, 72), (9000, 513, 16), (30011, 5000, 8), (12345, 151936, 8)])
def test_gradient(N, V, d, kind, dtype):
    grad, tok = matrix(N, d, dtype, seed=N), tokens(N, V, kind, seed=d)
    got = check_backward(grad, tok, V, 0.75)
    again = dh.embed_backward(grad, tok, V, scale=0.75)
    assert torch.equal(got, again)
    base = matrix(V, d, dtype, seed=3)
    check_backward(grad, tok, V, 0.75, base=base.clone(), grad_table=base, accumulate=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,d", [(300, 2000, 5120), (64, 10, 65536), (200, 151936, 1001), (40, 1 << 21, 16)])
def test_wide_rows_and_large_tables(N, V, d, dtype):
    check_backward(matrix(N, d, dtype, 1), tokens(N, V), V)


def test_many_tokens():
    N, V, d = 1 << 20, 30000, 8
    grad, tok = matrix(N, d, "f32", 1), tokens(N, V)
    check_backward(grad, tok, V)
    assert torch.equal(dh.embed(grad, torch.arange(N - 1, -1, -1, device=DEV, dtype=torch.int32)), grad.flip(0))


def test_the_sum_goes_by_position():
    """Up to 8 tokens of one id and nothing else: the fp32 sum in the order of the positions, bit for bit."""
    g = matrix(8, 256, "f32", 5) * 10 ** torch.arange(8, device=DEV)[:, None].float()
    tok = torch.full((8,), 3, dtype=torch.int32, device=DEV)
    want = torch.zeros(256, device=DEV)
    for n in range(8):
        want = want + g[n]
    assert torch.equal(dh.embed_backward(g, tok, 5)[3], want)


def test_nan_and_inf_stay_in_their_rows():
    V, d = 50, 64
    for dtype in ("f32", "bf16"):
        g, tok = matrix(200, d, dtype, 1), tokens(200, V, "uniform")
        g[3, 5], g[9, 6] = float("nan"), float("inf")
        tok[3], tok[9], tok[11] = 7, 8, -1
        g[11] = float("nan")  # padding: not read into any sum
        got = dh.embed_backward(g, tok, V)
        bad = ~got.isfinite()
        assert bad[7, 5] and bad[8, 6] and bad.sum() == 2


def test_offsets_beyond_32_bits():
    V, d, ld = 3, 40, (1 << 31) + 8
    buf = torch.zeros(2 * ld + d, dtype=torch.bfloat16, device=DEV)
    table = buf.as_strided((V, d), (ld, 1))
    table.copy_(matrix(V, d, "bf16", 3))
    tok = tokens(9, V, "mixed")
    assert torch.equal(dh.embed(table, tok), forward(table, tok, 1.0))
    out = dh.embed_backward(matrix(9, d, "bf16", 4), tok, V, grad_table=table)
    assert torch.equal(out, dh.embed_backward(matrix(9, d, "bf16", 4), tok, V))


def test_empty_calls():
    table, none = matrix(20, 8, "f32"), torch.empty(0, dtype=torch.int32, device=DEV)
    assert dh.embed(table, none).shape == (0, 8)
    assert not dh.embed_backward(table[:0], none, 20, grad_table=matrix(20, 8, "f32")).any()
    into = matrix(20, 8, "f32", ld=12)
    dh.embed_backward(table[:0], none, 20, grad_table=into)
    assert not into.any() and into.as_strided((19, 4), (12, 1), 8).isnan().all()
    was = table.clone()
    dh.embed_backward(table[:0].clone(), none, 20, grad_table=table, accumulate=True)
    assert torch.equal(table, was)


def test_graphs_streams_and_a_workspace():
    V, d, N = 4000, 96, 6000
    grad, tok, table = matrix(N, d, "bf16", 1), tokens(N, V), matrix(V, d, "bf16", 2)
    ws = dh.Workspace()
    want = dh.embed_backward(grad, tok, V)
    for n in (10, N, 300, N):
        a = dh.embed_backward(grad[:n], tok[:n], V, workspace=ws)
        assert torch.equal(a, dh.embed_backward(grad[:n], tok[:n], V))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = dh.embed_backward(grad, tok, V, stream=s), dh.embed(table, tok, stream=s)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, forward(table, tok, 1.0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = dh.embed_backward(grad, tok, V), dh.embed(table, tok)
    tok.copy_(tokens(N, V, "mixed", 5))
    a.fill_(float("nan"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, dh.embed_backward(grad, tok, V)) and torch.equal(b, forward(table, tok, 1.0))


def test_refusals():
    table, tok = matrix(10, 8, "f32"), tokens(4, 10)
    with pytest.raises(ValueError, match="tokens must be"):
        dh.embed(table, tok.long())
    with pytest.raises(ValueError, match="tokens must be"):
        dh.embed(table, tok.view(2, 2))
    with pytest.raises(ValueError, match="adjacent"):
        dh.embed(table.t(), tok)
    with pytest.raises(ValueError, match="out must be"):
        dh.embed(table, tok, out=torch.empty(4, 9, device=DEV))
    with pytest.raises(ValueError, match="overlap"):
        dh.embed(table, tok, out=torch.empty(1, 8, device=DEV).expand(4, 8))
    with pytest.raises(dh.DhError, match="INVALID_ARG"):
        dh.embed(table, tok, out=table[2:6])
    with pytest.raises(ValueError, match="accumulate"):
        dh.embed_backward(table[:4], tok, 10, accumulate=True)
    with pytest.raises(ValueError, match="grad_table must be"):
        dh.embed_backward(table[:4], tok, 10, grad_table=table.bfloat16())
    with pytest.raises(dh.DhError, match="INVALID_ARG"):
        dh.embed_backward(table[:4], tok, 10, grad_table=table)
    with pytest.raises(TypeError, match="dtype"):
        dh.embed(table.half(), tok)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 1001, 5120])
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -float("inf")])
def test_padding_is_zeros_at_any_scale(scale, d, dtype):
    V = 50
    for N in (9, 20000):
        table, tok = matrix(V, d, dtype, seed=1), tokens(N, V, "mixed", seed=2)
        held = (tok >= 0) & (tok < V)
        got = dh.embed(table, tok, scale=scale)
        assert not got[~held].any() and not got[held].isfinite().any()
        assert torch.equal(got[held].isnan(), forward(table, tok, scale)[held].isnan())
    grad = dh.embed_backward(matrix(9, d, dtype, 3), tok[:9], V, scale=scale)
    none = torch.ones(V, dtype=torch.bool, device=DEV)
    none[tok[:9][held[:9]].long()] = False
    assert not grad[none].any() and not grad[~none].isfinite().any()
