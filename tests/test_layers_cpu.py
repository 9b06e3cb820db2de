"""Host-side checks of the sampling, embedding and layer norm calls: bad arguments are refused before a device is
touched, empty ones are no-ops, and workspaces are sized."""
import ctypes

import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding, build, layers

FAKE = 0x10000  # never dereferenced by rejected calls
P, F = ctypes.c_void_p, ctypes.c_float
DH_OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def sample(lib, N=2, V=1000, dt=binding.F32, ld=1000, z=FAKE, u=FAKE, T=1.0, k=0, p=1.0, m=0.0, tp=0, kp=0, pp=0, mp=0,
           tok=FAKE, prob=FAKE, ws=FAKE * 16, nbytes=1 << 40):
    return lib.dh_sample(P(z), ld, P(u), P(tp), P(kp), P(pp), P(mp), F(T), k, F(p), F(m), N, V, dt, P(tok), P(prob),
                         P(ws), nbytes, None)


def test_sample_rejects_bad_arguments(lib):
    call = lambda **a: sample(lib, **a)  # noqa: E731
    assert call(N=-1) == INVALID and call(V=0) == INVALID and call(ld=-1) == INVALID
    for T in (-1.0, -1e-30, NAN, INF, -INF):
        assert call(T=T) == INVALID
    for x in (-0.1, 1.1, NAN, INF):
        assert call(p=x) == INVALID and call(m=x) == INVALID
    assert call(k=-1) == INVALID
    assert call(dt=2) == UNSUPPORTED and call(V=(1 << 21) + 1) == UNSUPPORTED
    assert call(N=(1 << 31) - 1, V=1) == UNSUPPORTED
    assert call(z=FAKE + 2) == UNSUPPORTED and call(dt=binding.BF16, z=FAKE + 1) == UNSUPPORTED
    for name in ("z", "u", "tok"):
        assert call(**{name: 0}) == INVALID
    assert call(N=0, z=0, u=0, tok=0, prob=0, ws=0) == DH_OK
    # a value of all rows is not looked at where the rows have their own
    assert call(T=NAN, tp=FAKE, N=0) == call(k=-5, kp=FAKE, N=0) == call(p=7.0, pp=FAKE, N=0) == DH_OK
    for bad in ((0, 100, 0), (-1, 100, 0), (1, 0, 0), (1, 100, 2), (1, (1 << 21) + 1, 0)):
        assert lib.dh_sample_workspace(*bad) == 0
    if lib.dh_sample_workspace(2, 1000, binding.F32):
        assert call(ws=0) == WORKSPACE and call(ws=FAKE * 16 + 16) == WORKSPACE and call(nbytes=15) == WORKSPACE


def test_embed_rejects_bad_arguments(lib):
    def call(N=2, V=1000, d=64, dt=binding.F32, ts=64, os=64, t=FAKE, tok=FAKE, o=FAKE << 8):
        return lib.dh_embed(P(t), ts, P(tok), N, V, d, dt, F(1.0), P(o), os, None)
    assert call(N=-1) == INVALID and call(V=0) == INVALID and call(d=0) == INVALID
    assert call(ts=-1) == INVALID and call(os=63) == INVALID
    assert call(dt=3) == UNSUPPORTED and call(V=(1 << 21) + 1) == UNSUPPORTED
    assert call(d=65537, os=65537) == UNSUPPORTED and call(N=(1 << 24) + 1) == UNSUPPORTED
    assert call(t=0) == INVALID and call(tok=0) == INVALID and call(o=0) == INVALID
    assert call(t=FAKE + 2) == UNSUPPORTED and call(o=(FAKE << 8) + 2) == UNSUPPORTED
    assert call(o=FAKE + 64) == INVALID                 # part of the table
    assert call(N=0, t=0, tok=0, o=0) == DH_OK


def test_embed_backward_rejects_bad_arguments(lib):
    def call(N=2, V=1000, d=64, dt=binding.F32, gs=64, ts=64, g=FAKE, tok=FAKE, o=FAKE << 8, acc=0, ws=FAKE * 16,
             nbytes=1 << 40):
        return lib.dh_embed_backward(P(g), gs, P(tok), N, V, d, dt, F(1.0), acc, P(o), ts, P(ws), nbytes, None)
    assert call(N=-1) == INVALID and call(V=0) == INVALID and call(d=0) == INVALID
    assert call(gs=-1) == INVALID and call(ts=63) == INVALID and call(acc=2) == INVALID and call(acc=-1) == INVALID
    assert call(dt=3) == UNSUPPORTED and call(V=(1 << 21) + 1) == UNSUPPORTED
    assert call(d=65537, ts=65537) == UNSUPPORTED and call(N=(1 << 24) + 1) == UNSUPPORTED
    assert call(g=0) == INVALID and call(tok=0) == INVALID and call(o=0) == INVALID
    assert call(g=FAKE + 2) == UNSUPPORTED and call(o=(FAKE << 8) + 2) == UNSUPPORTED
    assert call(o=FAKE) == INVALID and call(o=FAKE - 1000) == INVALID
    assert call(ws=0) == WORKSPACE and call(ws=FAKE * 16 + 16) == WORKSPACE and call(nbytes=255) == WORKSPACE
    assert call(N=0, acc=1, g=0, tok=0, o=0, ws=0) == DH_OK
    need = lib.dh_embed_backward_workspace(4096, 151936, 5120, binding.BF16)
    assert need % 256 == 0 and need >= 4096 * 16 + 151936 // 8
    for bad in ((0, 10, 8, 0), (-1, 10, 8, 0), (1, 0, 8, 0), (1, 10, 0, 0), (1, 10, 8, 2), ((1 << 24) + 1, 10, 8, 0)):
        assert lib.dh_embed_backward_workspace(*bad) == 0


def test_layer_norm_rejects_bad_arguments(lib):
    def call(N=2, d=64, dt=binding.BF16, pt=binding.BF16, xs=64, ys=64, x=FAKE, w=FAKE, b=FAKE, eps=1e-5, y=FAKE << 8,
             st=FAKE):
        return lib.dh_layer_norm(P(x), xs, P(w), P(b), N, d, dt, pt, F(eps), P(y), ys, P(st), None)
    assert call(N=-1) == INVALID and call(d=0) == INVALID and call(xs=-1) == INVALID and call(ys=63) == INVALID
    for eps in (-1e-5, NAN, INF):
        assert call(eps=eps) == INVALID
    assert call(dt=2, pt=2) == UNSUPPORTED and call(pt=2) == UNSUPPORTED
    assert call(dt=binding.F32, pt=binding.BF16) == UNSUPPORTED
    assert call(d=65537, ys=65537) == UNSUPPORTED and call(N=(1 << 31) - 1, ys=1 << 20) == UNSUPPORTED
    assert call(x=0) == INVALID and call(y=0) == INVALID
    assert call(x=FAKE + 1) == UNSUPPORTED and call(y=(FAKE << 8) + 1) == UNSUPPORTED
    assert call(w=FAKE + 1) == UNSUPPORTED and call(b=FAKE + 1) == UNSUPPORTED and call(st=FAKE + 4) == UNSUPPORTED
    assert call(pt=binding.F32, w=FAKE + 2) == UNSUPPORTED
    assert call(y=FAKE + 128) == INVALID and call(y=FAKE, ys=72) == INVALID  # partly x; the same memory in other rows
    assert call(N=0, x=0, y=0) == DH_OK


def test_layer_norm_backward_rejects_bad_arguments(lib):
    def call(N=2, d=64, dt=binding.F32, pt=binding.F32, gs=64, xs=64, ds=64, g=FAKE, x=FAKE << 4, st=FAKE, w=FAKE,
             dx=FAKE << 8, dw=FAKE << 9, db=FAKE << 10, ws=FAKE * 16, nbytes=1 << 40):
        return lib.dh_layer_norm_backward(P(g), gs, P(x), xs, P(st), P(w), N, d, dt, pt, P(dx), ds, P(dw), P(db),
                                          P(ws), nbytes, None)
    assert call(N=-1) == INVALID and call(d=0) == INVALID and call(gs=-1) == INVALID and call(xs=-1) == INVALID
    assert call(ds=63) == INVALID
    assert call(dt=2, pt=2) == UNSUPPORTED and call(pt=binding.BF16) == UNSUPPORTED
    assert call(d=65537, ds=65537) == UNSUPPORTED and call(N=(1 << 31) - 1) == UNSUPPORTED
    assert call(g=0) == INVALID and call(x=0) == INVALID and call(st=0) == INVALID
    for name in ("g", "x", "w", "dx", "dw", "db"):
        assert call(**{name: (FAKE << 12) + 2}) == UNSUPPORTED
    assert call(st=FAKE + 4) == UNSUPPORTED
    assert call(dx=FAKE + 64) == INVALID and call(dx=(FAKE << 4) - 64) == INVALID
    assert call(ws=0) == WORKSPACE and call(ws=FAKE * 16 + 16) == WORKSPACE and call(nbytes=255) == WORKSPACE
    assert call(dx=0, dw=0, db=0, ws=0, g=0) == DH_OK
    need = lib.dh_layer_norm_backward_workspace(4096, 5120, binding.BF16)
    assert need % 256 == 0 and need >= 256 + 2 * 5120 * 4
    for bad in ((0, 8, 0), (-1, 8, 0), (1, 0, 0), (1, 65537, 0), (1, 8, 2)):
        assert lib.dh_layer_norm_backward_workspace(*bad) == 0


def test_binding_refuses_cpu_tensors_and_other_shapes():
    z, tok = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: binding.sample(z, torch.zeros(2)), lambda: binding.embed(z, tok),
                 lambda: binding.embed_backward(z, tok, 5), lambda: binding.layer_norm(z),
                 lambda: binding.layer_norm_backward(z, z, torch.zeros(2, 2)), lambda: layers.embedding(z, tok),
                 lambda: layers.layer_norm(z)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="vocab"):
        binding.sample(z[0], torch.zeros(2))
    for call in (lambda: binding.embed(z[0], tok), lambda: binding.embed_backward(z[0], tok, 5),
                 lambda: binding.layer_norm(z[0])):
        with pytest.raises(ValueError, match="rows, d"):
            call()


class Rows:  # what the checks look at of a tensor that no memory here would hold
    dtype, device = torch.float32, torch.device("cuda", 0)

    def __init__(self, *shape):
        self.shape = torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def stride(self, d):
        return 1


def test_binding_refuses_sizes_beyond_32_bits():
    n = (1 << 31) + 5
    for call in (lambda: binding.sample(Rows(n, 4), None), lambda: binding.sample(Rows(4, n), None),
                 lambda: binding.layer_norm(Rows(n, 4)), lambda: binding.layer_norm(Rows(4, n)),
                 lambda: binding.embed(Rows(n, 4), Rows(1)), lambda: binding.embed_backward(Rows(n, 4), None, 5)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    tok = Rows(1)
    tok.dtype, tok.is_contiguous = torch.int32, lambda: True
    for vocab in (0, -1, n):
        with pytest.raises(ValueError, match="vocab"):
            binding.embed_backward(Rows(1, 4), tok, vocab)
    u = Rows(1)
    u.is_contiguous = lambda: True
    with pytest.raises(ValueError, match="top_k"):
        binding.sample(Rows(1, 4), u, top_k=n)


@pytest.mark.parametrize("name", ["sample", "embed", "embed_backward", "layer_norm", "layer_norm_backward",
                                  "embedding"])
def test_public_names(name):
    import speculative_decoding_draft_dh_gb300 as pkg
    assert callable(getattr(pkg, name))


def test_results_that_share_memory_are_refused(lib):
    """Small results (tokens, probabilities, statistics, parameters' gradients) over an input or one another.  The
    accepted neighbours end at a later check, so that nothing is launched."""
    A = [(i + 1) << 24 for i in range(12)]  # arrays far apart

    def draw(N=4, ld=100002, z=A[0], u=A[1], T=A[2], k=A[3], p=A[4], m=A[5], tok=A[6], prob=A[7]):
        return sample(lib, N=N, V=100000, ld=ld, z=z, u=u, tp=T, kp=k, pp=p, mp=m, tok=tok,
                      prob=prob, ws=0)
    assert draw() == WORKSPACE
    assert draw(tok=A[7]) == draw(tok=A[7] + 12) == INVALID and draw(tok=A[7] + 16) == WORKSPACE
    assert draw(tok=A[0] + 64) == draw(prob=A[0] + 64) == draw(prob=A[0] - 4) == INVALID
    assert draw(prob=A[0] + 4 * 100000) == INVALID  # 2 elements between the rows, 4 probabilities
    assert draw(prob=A[0] + 4 * 100000, ld=100016) == WORKSPACE  # they fit
    for x in A[1:6]:
        assert draw(tok=x) == draw(prob=x) == WORKSPACE
        assert draw(tok=x + 4) == draw(prob=x - 12) == draw(prob=x + 12) == INVALID

    def look(tok=A[0], out=A[1], os=64):
        return lib.dh_embed(P(A[2]), 64, P(tok), 4, 1000, 64, binding.F32, F(1.0), P(out), os, None)
    assert look(tok=A[1]) == look(tok=A[1] + 1000) == look(tok=A[1] - 8) == look(out=A[0] - 64) == INVALID

    def grad(tok=A[0], out=A[1], ts=64):
        return lib.dh_embed_backward(P(A[2]), 64, P(tok), 4, 1000, 64, binding.F32, F(1.0), 0, P(out), ts, P(0), 0,
                                     None)
    assert grad() == WORKSPACE and grad(tok=A[1] + 256) == INVALID
    assert grad(tok=A[1] + 256, ts=72) == WORKSPACE and grad(tok=A[1] + 260, ts=68) == INVALID

    def norm(y=A[1], w=A[2], b=A[3], st=A[4], eps=1e-5):
        return lib.dh_layer_norm(P(A[0]), 64, P(w), P(b), 4, 64, binding.F32, binding.F32, F(eps), P(y), 64, P(st),
                                 None)
    for bad in (dict(w=A[1] + 512), dict(b=A[1] + 512), dict(st=A[0] + 8), dict(st=A[1] + 1000), dict(st=A[2] + 248),
                dict(st=A[3] - 24), dict(y=A[4] - 1000)):
        assert norm(**bad) == INVALID

    def back(g=A[0], x=A[1], st=A[2], w=A[3], dx=A[4], dw=A[5], db=A[6], xs=64):
        return lib.dh_layer_norm_backward(P(g), 64, P(x), xs, P(st), P(w), 4, 64, binding.F32, binding.F32, P(dx), 64,
                                          P(dw), P(db), P(0), 0, None)
    assert back() == back(dx=A[0]) == back(dx=A[1]) == WORKSPACE
    for bad in (dict(dx=A[2]), dict(dx=A[3] - 800), dict(dw=A[0]), dict(dw=A[1] + 64), dict(db=A[2] + 24), dict(dw=A[3]),
                dict(db=A[4] + 768), dict(db=A[5] + 128), dict(dw=A[6])):
        assert back(**bad) == INVALID, bad
    assert back(dw=A[1] + 256, xs=128) == WORKSPACE and back(dw=A[1] + 260, xs=128) == INVALID
