"""Sampling (dh_sample) against the definition in 64 bits: the token that a uniform falls on, and its probability.

The kernel's running sums are off by 2^-30 of themselves at most, so a token has to be the reference's wherever no
border that decides it (of top-p, of the draw) is nearer than 2^-28 of the mass.  Random rows come that near a border
once in 10^5; each test allows one such row.  Probabilities: both masses' errors and one rounding, 2^-24 + 2^-29,
taken as 2^-23."""
import numpy as np
import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding as dh

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NEAR = 2.0 ** -28


def reference(row, u, T, k, p, m):
    """(token, probability, nearness of the nearest border, in the kept mass)."""
    T, p, m, u = (float(np.float32(v)) for v in (T, p, m, u))
    z = row.double().cpu().numpy()
    if np.isnan(z).any() or np.isposinf(z).any() or not (z > -np.inf).any() or not (0 <= T < np.inf) \
            or np.isnan([u, p, m]).any():
        return -1, 0.0, 1.0
    order = np.argsort(-z, kind="stable")
    if T == 0 or k == 1 or p <= 0:
        return int(order[0]), 1.0, 1.0
    V = len(z)
    k = k if 0 < k < V else V
    with np.errstate(over="ignore"):
        w = np.exp((z[order] - z[order[0]]) / T)
    w[k:] = 0
    run = np.cumsum(w)
    M, near = run[-1], 1.0
    n = np.searchsorted(run, p * M) + 1 if p < 1 else k
    if p < 1:
        near = np.abs(run / M - p).min()
    if m > 0:
        n = min(n, max(1, int((w >= min(m, 1.0)).sum())))
    n = min(n, k)
    K = run[n - 1]
    at = min(int(np.searchsorted(run[:n], u * K, side="right")), n - 1)
    near = min(near, np.abs(run[:n - 1] / K - u).min()) if n > 1 else near
    while at > 0 and w[at] == 0:  # nothing without weight is drawn
        at -= 1
    return int(order[at]), w[at] / K, near


def check(z, u, T=1.0, k=0, p=1.0, m=0.0, **kw):
    token, prob = dh.sample(z, u, temperature=T, top_k=k, top_p=p, min_p=m, **kw)
    torch.cuda.synchronize()
    at = lambda v, n: v[n].item() if torch.is_tensor(v) else v  # noqa: E731
    near = 0
    for n in range(z.shape[0]):
        want, q, border = reference(z[n], u[n].item(), at(T, n), at(k, n), at(p, n), at(m, n))
        if border < NEAR:
            near += 1
            continue
        assert token[n].item() == want, (n, token[n].item(), want, border)
        assert abs(prob[n].item() - q) <= 2.0 ** -23 * q, (n, prob[n].item(), q)
    assert near <= 1
    return token, prob


def rows(N, V, dtype, seed=0, std=2.5, hot=8, ld=None, base=0):
    g = torch.Generator().manual_seed(seed)
    z = std * torch.randn(N, V, generator=g)
    if hot:
        at = torch.randint(0, V, (N, hot), generator=g)
        z.scatter_add_(1, at, 6 + 6 * torch.rand(N, hot, generator=g))
    ld = V if ld is None else ld
    buf = torch.full((base + N * ld + 64,), float("nan"), dtype=DT[dtype], device=DEV)
    view = buf[base:base + N * ld].view(N, ld)[:, :V]
    view.copy_(z.to(DT[dtype]))
    return view, torch.rand(N, generator=g).to(DEV)


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 20, 0.8, 0.0), (1.0, 0, 0.95, 0.0), (1.5, 50, 1.0, 0.0), (0.8, 0, 1.0, 0.05),
            (1.0, 300, 0.9, 0.01), (2.0, 0, 0.5, 0.001), (0.0, 0, 1.0, 0.0), (1.0, 1, 0.9, 0.0), (3.0, 0, 1.0, 0.0),
            (1.0, 5000, 0.99, 0.0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (2, 7), (5, 33), (4, 1000), (7, 4096), (3, 5003), (2, 50257),
                                 (2, 151936), (300, 2000)])
def test_sizes(N, V, dtype):
    z, u = rows(N, V, dtype, seed=V)
    for s in SETTINGS:
        check(z, u, *s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,ld,base", [(1001, 1001, 0), (1001, 1008, 0), (1003, 1003, 1), (5000, 5003, 3), (9, 9, 5),
                                       (70001, 70001, 7)])
def test_strides_and_alignment(V, ld, base, dtype):
    z, u = rows(4, V, dtype, seed=3, ld=ld, base=base)
    for s in SETTINGS[:7]:
        got = check(z, u, *s)
        again = dh.sample(z.contiguous(), u, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_settings_of_each_row(dtype):
    N = 3 * len(SETTINGS)
    z, u = rows(N, 20011, dtype, seed=8)
    col = lambda i, t: torch.tensor([SETTINGS[n % len(SETTINGS)][i] for n in range(N)], dtype=t, device=DEV)  # noqa: E731
    T, k, p, m = col(0, torch.float32), col(1, torch.int32), col(2, torch.float32), col(3, torch.float32)
    both = check(z, u, T, k, p, m)
    for n in range(0, N, 5):  # as the same row alone, with numbers
        s = SETTINGS[n % len(SETTINGS)]
        token, prob = dh.sample(z[n:n + 1], u[n:n + 1], temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        assert token.item() == both[0][n].item() and prob.item() == both[1][n].item()
    # settings beyond their ranges count as the nearest end, those that are no numbers leave no token
    T = torch.full((8,), 1.0, device=DEV)
    k = torch.zeros(8, dtype=torch.int32, device=DEV)
    p, m = torch.ones(8, device=DEV), torch.zeros(8, device=DEV)
    k[0], k[1], p[2], p[3], m[4], m[5] = -7, 10 ** 9, -1.0, 2.5, -3.0, 9.0
    check(z[:8], u[:8], T, k, p, m)
    k[:], p[:], m[:] = 0, 1, 0
    T[0], T[1], T[2], p[3], m[4] = float("nan"), -1.0, float("inf"), float("nan"), float("nan")
    u = u[:8].clone()
    u[5], u[6], u[7] = float("nan"), -0.5, 1.5
    token, prob = dh.sample(z[:8], u, temperature=T, top_k=k, top_p=p, min_p=m)
    assert (token[:6] == -1).all() and (prob[:6] == 0).all()
    assert token[6] == z[6].float().argmax() and token[7] >= 0 and prob[7] > 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_rows(dtype):
    """Rows with -inf, of nothing else, with the type's lowest value, with one token, with NaN and +inf."""
    V = 5001
    z, u = rows(12, V, dtype, seed=4)
    inf = float("inf")
    z[0] = -inf
    z[1, 1:] = -inf
    z[2, :V - 1] = -inf
    z[3, ::2] = -inf
    z[4] = torch.finfo(z.dtype).min
    z[5, 10:] = torch.finfo(z.dtype).min
    z[6, V - 1] = float("nan")
    z[7, 0] = inf
    z[8, 17:] = -inf
    z[9, 100] = torch.finfo(z.dtype).max
    z[10] = 0.0
    z[10, ::3] = -0.0
    for s in [(1.0, 0, 1.0, 0.0), (1.0, 10, 0.9, 0.0), (0.5, 0, 0.7, 0.0), (1.0, 0, 1.0, 0.1), (0.0, 0, 1.0, 0.0),
              (1.0, 4000, 1.0, 0.0), (1.0, 1, 1.0, 0.0)]:
        token, prob = check(z, u, *s)
        for n in (0, 6, 7):
            assert token[n] == -1 and prob[n] == 0
        assert token[1] == 0 and token[2] == V - 1 and prob[1] == 1 and prob[2] == 1
        assert token[3] % 2 == 1 and 0 <= token[5] < 10 and 0 <= token[8] < 17 and token[9] == 100


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 31, 1000, 40009])
def test_equal_logits_go_by_id(V, dtype):
    """Constant rows: the token is floor(u n) of the n kept, whatever the temperature."""
    u = torch.tensor([0.0, 0.125, 0.25, 0.4999999, 0.5, 0.75, 0.99999994], device=DEV)
    for value in (0.0, -3.5, 1e4, -1e30):
        z = torch.full((len(u), V), value, dtype=DT[dtype], device=DEV)
        for T, k, p in ((1.0, 0, 1.0), (0.01, 0, 1.0), (30.0, 8, 1.0), (1.0, 0, 0.5), (1.0, 24, 0.25), (1.0, 0, 0.75)):
            n = min(k, V) if k else V
            n = int(np.ceil(p * n)) if p < 1 else n
            token, prob = dh.sample(z, u, temperature=T, top_k=k, top_p=p)
            want = [int(np.floor(float(x) * n)) for x in u]
            assert token.tolist() == want, (value, T, k, p)
            assert (prob - 1 / n).abs().max() <= 2.0 ** -23 / n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["two", "steps", "rising", "falling", "cluster"])
def test_rows_of_few_values(kind, dtype):
    V, N = 30001, 6
    i = torch.arange(V).float()
    z = {"two": (i % 7 == 3).float(), "steps": torch.floor(i / 1000), "rising": i / V, "falling": 5 - i / V,
         "cluster": torch.where(i % 5000 == 1, 9.0, -i % 13)}[kind].to(DT[dtype]).to(DEV).expand(N, V)
    g = torch.Generator().manual_seed(1)
    for s in SETTINGS:
        check(z, torch.rand(N, generator=g).to(DEV), *s)


@pytest.mark.parametrize("scale,T", [(1.0, 1e-3), (1.0, 1e-6), (1.0, 1e3), (1e4, 1.0), (1e4, 1e4), (1e30, 1e30),
                                     (1e-30, 1e-30), (1e-3, 1e-3), (300.0, 0.01), (1.0, 1e-38), (1.0, 3e38)])
def test_extreme_scales(scale, T):
    z, u = rows(24, 3001, "f32", seed=6, hot=0)
    z = (z * scale).contiguous()
    for k, p, m in ((0, 1.0, 0.0), (40, 0.9, 0.0), (0, 0.5, 0.0), (0, 1.0, 0.2)):
        check(z, u, T, k, p, m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("s", [(1.0, 0, 1.0, 0.0), (1.0, 40, 1.0, 0.0), (0.9, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.02)])
def test_draws_follow_the_distribution(s, dtype):
    """Evenly spread uniforms over one shared row: each token comes as often as its probability says, within one,
    since the uniforms that fall on it are an interval; its stated probability is that."""
    N, V = 40000, 1999
    z, _ = rows(1, V, dtype, seed=12, std=1.5)
    u = (torch.arange(N, device=DEV).double() + 0.5) / N
    token, prob = dh.sample(z.expand(N, V), u.float(), temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
    count = torch.bincount(token.long(), minlength=V).cpu().numpy()
    row = z[0].double().cpu().numpy()
    order = np.argsort(-row, kind="stable")
    w = np.exp((row[order] - row[order[0]]) / float(np.float32(s[0])))
    n = s[1] or V
    w[n:] = 0
    if s[2] < 1:
        w[np.searchsorted(np.cumsum(w), float(np.float32(s[2])) * w.sum()) + 1:] = 0
    if s[3] > 0:
        w[w < float(np.float32(s[3]))] = 0
    q = np.zeros(V)
    q[order] = w / w.sum()
    # one for the interval's ends, and the uniforms' own rounding, half of 2^-24 at each of two ends
    assert np.abs(count - q * N).max() <= 1 + N * 2.0 ** -24
    got = prob.double().cpu().numpy()
    assert np.abs(got - q[token.cpu().numpy()]).max() <= 2.0 ** -23
    # the uniforms rise, so the tokens come in the order of their logits
    assert (np.diff(row[token.cpu().numpy()]) <= 0).all()


LONG = {  # of V ids i
    "flat": lambda V, g: 2 * torch.randn(V, generator=g),
    "narrow": lambda V, g: 1e-3 * torch.randn(V, generator=g),
    "steps": lambda V, g: torch.floor(torch.arange(V) / 1000.0) / 16,
    "few values": lambda V, g: (torch.arange(V) % 3).float(),
    "equal": lambda V, g: torch.full((V,), -2.5),
    "ramp": lambda V, g: torch.arange(V) * (10.0 / V),
    "above": lambda V, g: torch.where(torch.arange(V) % 37 == 5, 4.0, 0.0) + 0.25 * torch.randn(V, generator=g),
    "large": lambda V, g: 1e6 + torch.randn(V, generator=g),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", LONG)
def test_long_rows_without_a_short_list(kind, dtype):
    """Rows of which thousands of tokens are kept, nearly equal or equal.  A weight is rounded to 2^-45 of the largest;
    of the likeliest tokens' z the others' are 14 T below it at most, so that this is 2^-24.8 of each: with the sums'
    2^-29 and the result's 2^-24 less than 2^-23."""
    V, N = 150011, 3
    g = torch.Generator().manual_seed(len(kind))
    row = LONG[kind](V, g).to(DT[dtype])
    for ld in (V, 150016):  # the second in whole vectors
        buf = torch.full((N, ld), float("nan"), dtype=DT[dtype], device=DEV)
        z = buf[:, :V]
        z.copy_(row)
        u = torch.rand(N, generator=g).to(DEV)
        for s in [(3.0, 0, 1.0, 0.0), (3.0, 0, 0.99, 0.0), (2.0, 0, 0.5, 0.001), (1.0, 0, 1.0, 0.05), (1.0, 0, 1.0, 0.97),
                  (1.0, 3000, 1.0, 0.0), (1.0, 1800, 0.9, 0.01), (1.0, 900, 1.0, 0.0), (5.0, 20000, 0.9, 0.0),
                  (0.0, 0, 1.0, 0.0)]:
            check(z, u, *s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,top", [(0.7, 40.0), (1.0, 40.0), (0.7, 5.0), (0.3, 13.0)])
def test_fewer_tokens_with_a_weight_than_top_k(T, top, dtype):
    """Logits that fall by 40 T: of 3500 the last three hundred or so weigh less than 2^-52 of the first and count as
    none, so top-k reaches past the tokens that count."""
    V, N = 3500, 24
    z = torch.linspace(top, top - 40 * T, V)[torch.randperm(V, generator=torch.Generator().manual_seed(1))]
    z = z.to(DT[dtype]).to(DEV).expand(N, V)
    u = torch.rand(N, generator=torch.Generator().manual_seed(2)).to(DEV)
    for s in [(T, 3400, 1.0, 0.0), (T, 3400, 0.99, 0.0), (T, 3400, 0.9, 1e-4), (T, 3400, 1.0, 1.0), (T, 1500, 0.99, 0.0)]:
        check(z, u, *s)


def test_rows_that_are_searched_beside_others():
    """Each row of a batch as it is alone, whatever its neighbours need; again with one workspace and given outputs."""
    V, N = 60000, 40
    z, u = rows(N, V, "bf16", seed=21)
    g = torch.Generator().manual_seed(2)
    z[::3] = (0.5 * torch.randn(V, generator=g)).bfloat16().to(DEV)
    z[4], z[7, 5] = -float("inf"), float("nan")
    T = torch.tensor([[0.0, 0.7, 1.0, 2.5][n % 4] for n in range(N)], device=DEV)
    k = torch.tensor([[0, 30, 4000][n % 3] for n in range(N)], dtype=torch.int32, device=DEV)
    p = torch.tensor([[1.0, 0.9][n // 3 % 2] for n in range(N)], device=DEV)
    m = torch.tensor([[0.0, 0.0, 0.02][n // 5 % 3] for n in range(N)], device=DEV)
    token, prob = check(z, u, T, k, p, m)
    ws = dh.Workspace()
    out = torch.empty(N, dtype=torch.int32, device=DEV), torch.empty(N, device=DEV)
    for n in (N, 7, N):
        dh.sample(z[:n], u[:n], temperature=T[:n], top_k=k[:n], top_p=p[:n], min_p=m[:n], token_out=out[0][:n],
                  prob_out=out[1][:n], workspace=ws)
        assert torch.equal(out[0][:n], token[:n]) and torch.equal(out[1][:n], prob[:n])
        out[0][:n], out[1][:n] = -5, -5
    for n in range(N):
        one = dh.sample(z[n:n + 1], u[n:n + 1], temperature=T[n].item(), top_k=k[n].item(), top_p=p[n].item(),
                        min_p=m[n].item())
        assert one[0][0] == token[n] and one[1][0] == prob[n]


def test_many_rows():
    """More rows than blocks can run at once, of both kinds of length."""
    for N, V in ((70000, 9), (20000, 9000)):
        g = torch.Generator(device=DEV).manual_seed(N)
        z = torch.randn(N, V, generator=g, device=DEV).bfloat16()
        u = torch.rand(N, generator=g, device=DEV)
        token, prob = dh.sample(z, u, temperature=0.0)
        first = (z == z.max(1, keepdim=True).values).int().argmax(1)
        assert torch.equal(token.long(), first) and (prob == 1).all()
        token, prob = dh.sample(z, u, temperature=1.5)
        for n in (0, 1, N // 2, N - 1):
            one = check(z[n:n + 1], u[n:n + 1], 1.5)
            assert one[0][0] == token[n] and one[1][0] == prob[n]


def test_offsets_beyond_32_bits():
    V, ld = 1000, (1 << 31) + 8
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device=DEV)
    z = buf.as_strided((3, V), (ld, 1))
    src, u = rows(3, V, "bf16", seed=2)
    z.copy_(src)
    for s in SETTINGS[:4]:
        check(z, u, *s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_largest_vocabulary(dtype):
    z, u = rows(2, 1 << 21, dtype, seed=5)
    for s in SETTINGS[:7]:
        check(z, u, *s)


def test_results_repeat_and_streams_and_graphs():
    z, u = rows(64, 30000, "bf16", seed=9)
    kw = dict(temperature=0.9, top_k=100, top_p=0.9)
    token, prob = dh.sample(z, u, **kw)
    out = torch.full((64,), -9, dtype=torch.int32, device=DEV), torch.zeros(64, device=DEV)
    v = out[0]._version
    for _ in range(5):
        got = dh.sample(z, u, token_out=out[0], prob_out=out[1], **kw)
        assert got[0] is out[0] and torch.equal(out[0], token) and torch.equal(out[1], prob)
    assert out[0]._version > v
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = dh.sample(z, u, stream=s, **kw)
    s.synchronize()
    assert torch.equal(a[0], token)
    graphs, outs = [], []
    for settings in (kw, dict(temperature=1.0)):
        for _ in range(2):
            dh.sample(z, u, **settings)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dh.sample(z, u, **settings))
        graphs.append(g)
    z2, u2 = rows(64, 30000, "bf16", seed=10)
    z.copy_(z2), u.copy_(u2)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for got, settings in zip(outs, (kw, dict(temperature=1.0))):
        want = dh.sample(z, u, **settings)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_without_probabilities_and_refusals():
    z, u = rows(3, 500, "f32")
    with pytest.raises(ValueError, match="u must be"):
        dh.sample(z, u[:2])
    with pytest.raises(ValueError, match="adjacent"):
        dh.sample(z.t(), u[:1].expand(500))
    with pytest.raises(ValueError, match="top_k must be"):
        dh.sample(z, u, top_k=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="temperature must be"):
        dh.sample(z, u, temperature=torch.ones(2, device=DEV))
    with pytest.raises(TypeError, match="dtype"):
        dh.sample(z.half(), u)
    for bad in (dict(temperature=-1.0), dict(top_p=1.5), dict(min_p=-0.1), dict(top_k=-2), dict(temperature=float("nan"))):
        with pytest.raises(dh.DhError, match="INVALID_ARG"):
            dh.sample(z, u, **bad)
    assert dh.sample(z[:0], u[:0])[0].shape == (0,)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.2e-38, 2e-38, 1e-37, 2.6e-37, 3e-37, 1.3e-36, 1.6e-36, 1e-34])
def test_tiny_temperatures_of_searched_rows(T, dtype):
    """Long flat rows whose logits and temperature lie near the smallest normal number: 64 steps of a weight's octave per
    unit of logit pass fp32's range there.  (The tokens of one weight's step are thousands, and of one bin.)"""
    V, N = 150016, 4
    g = torch.Generator().manual_seed(31)
    row = (2 * torch.randn(V, generator=g).double() * float(np.float32(T))).float().to(DT[dtype])
    z = row.to(DEV).expand(N, V)
    u = torch.rand(N, generator=g).to(DEV)
    for s in [(T, 0, 1.0, 0.0), (T, 0, 0.95, 0.0), (T, 3000, 1.0, 0.0), (T, 20000, 0.9, 0.001), (T, 0, 1.0, 0.05)]:
        token, _ = check(z, u, *s)
        assert ((token >= 0) & (token < V)).all()
    # and of one step's worth of values only, which are searched by their keys
    z = torch.where(torch.arange(V) % 2 == 0, 1.0, 2.0).mul(float(np.float32(T)) / 512).to(DT[dtype]).to(DEV).expand(N, V)
    for s in [(T, 0, 1.0, 0.0), (T, 0, 0.75, 0.0), (T, 100000, 1.0, 0.0)]:
        token, _ = check(z, u, *s)
        assert ((token >= 0) & (token < V)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [151936, 1 << 21])
@pytest.mark.parametrize("below", [15.0, 18.0, 21.0, 24.0, 28.0, "half a unit"])
def test_unlikely_tokens(below, V, dtype):
    """One likely token over a long tail, and uniforms that fall on the tail.  With f fraction bits a weight is off by
    2^-27.5 of itself (the table's and the cubic's 2^-29 each, and a few of 2^-31) and half a unit, 2^-(f + 1) of the
    largest; a sum of n by n times that.  So the token's own interval, widened by the sums' errors, has to hold
    u K, and the probability is off by its weight's and the mass's errors and 2^-24."""
    f = min(62 - (V - 1).bit_length(), 52)
    rel, unit = 2.0 ** -27.5, 2.0 ** -(f + 1)
    g = torch.Generator().manual_seed(V % 97 + 3)
    for tail in ("equal", "spread"):
        if below == "half a unit":  # equal logits whose weights are just under what counts
            if tail == "spread":
                continue
            z = torch.full((V,), -float((f + 1) * np.log(2.0) + 0.004))
        else:
            z = torch.full((V,), -below)
            if tail == "spread":
                z += 0.3 * torch.randn(V, generator=g)
        z[V // 3] = 0.0
        z = z.to(DT[dtype])
        row = z.double().numpy()
        order = np.argsort(-row, kind="stable")
        place = np.empty(V, dtype=np.int64)
        place[order] = np.arange(V)
        w = np.exp(row[order] - row[order[0]])
        run = np.cumsum(w)
        for k in (0, V // 2):
            n = k or V
            K = run[n - 1]
            share = 1 - w[0] / K
            u = torch.tensor(np.concatenate([1 - share * (np.arange(24) + 0.5) / 24, [0.3, 1 - 2.0 ** -24]]),
                             dtype=torch.float32, device=DEV).clamp(max=1 - 2.0 ** -24)
            token, prob = dh.sample(z.to(DEV).expand(len(u), V), u, top_k=k)
            torch.cuda.synchronize()
            for at, q, x in zip(token.tolist(), prob.tolist(), u.double().tolist()):
                i = place[at]
                assert 0 <= i < n
                slack = 2 * rel * K + 2 * n * unit + 2 * unit
                assert run[i] - w[i] - slack <= x * K <= run[i] + slack, (tail, k, i, x)
                off = w[i] / K * (2 * rel + n * unit / K + 1.01 * 2.0 ** -24) + unit / K
                assert abs(q - w[i] / K) <= 1.01 * off, (tail, k, i, q, w[i] / K)


def test_without_probabilities():
    """prob_out NULL: the tokens of the call with probabilities, in a row that one block takes, in long rows with a top-k
    for all, and where some rows are searched."""
    lib = dh.load_library()
    for V, N, k in ((500, 9, 0), (151936, 5, 30), (60000, 12, 0)):
        z, u = rows(N, V, "bf16", seed=V)
        if k == 0:
            z[::2] = (0.5 * torch.randn(V, generator=torch.Generator().manual_seed(3))).bfloat16().to(DEV)
        want, _ = dh.sample(z, u, temperature=1.5, top_k=k)
        token = torch.full((N,), -7, dtype=torch.int32, device=DEV)
        nbytes = lib.dh_sample_workspace(N, V, dh.BF16)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=DEV)
        status = lib.dh_sample(z.data_ptr(), z.stride(0), u.data_ptr(), None, None, None, None, 1.5, k, 1.0, 0.0, N, V,
                               dh.BF16, token.data_ptr(), None, ws.data_ptr(), nbytes,
                               torch.cuda.current_stream().cuda_stream)
        assert status == 0 and torch.equal(token, want)


def test_results_in_the_place_of_settings():
    """A row's token or probability over its own uniform or setting, searched rows and rows of one block among them."""
    for V, N in ((400, 30), (60000, 30)):
        z, u = rows(N, V, "bf16", seed=V)
        z[::2] = (0.5 * torch.randn(V, generator=torch.Generator().manual_seed(3))).bfloat16().to(DEV)
        at = torch.arange(N, device=DEV)
        given = {"temperature": 0.7 + 0.1 * (at % 5).float(), "top_k": (at % 4 * 50).int(),
                 "top_p": 1 - 0.05 * (at % 3).float(), "min_p": 0.001 * (at % 2).float()}
        want = dh.sample(z, u, **given)
        for name in ("u", "temperature", "top_p", "min_p", "top_k"):
            kw = {k: t.clone() for k, t in given.items()}
            uu = u.clone()
            place = uu if name == "u" else kw[name]
            out = {"token_out" if name == "top_k" else "prob_out": place}
            token, prob = dh.sample(z, uu, **kw, **out)
            assert torch.equal(token, want[0]) and torch.equal(prob, want[1])
            assert place is (token if name == "top_k" else prob)
