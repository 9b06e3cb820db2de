"""Host-side checks of the distillation, beam selection and state calls: bad arguments are refused
before a device is touched, empty ones are no-ops, and workspaces are sized."""
import ctypes

import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding, build, distill

FAKE = 0x10000  # never dereferenced by rejected calls
P, F = ctypes.c_void_p, ctypes.c_float
DH_OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def distill_call(lib, which, N=2, V=1000, K=8, dt=binding.F32, T=1.0, ld=1000, gld=1000, z=FAKE, idx=FAKE, y=FAKE,
                 loss=FAKE, stats=FAKE, gl=FAKE, grad=FAKE << 8, ws=FAKE * 16, nbytes=1 << 30):
    if which == "loss":
        return lib.dh_distill_topk(P(z), ld, P(idx), P(y), None, N, V, K, dt, F(T), P(loss), P(stats), P(ws), nbytes,
                                   None)
    if which == "backward":
        return lib.dh_distill_topk_backward(P(z), ld, P(idx), P(y), None, P(stats), P(gl), N, V, K, dt, F(T), P(grad),
                                            gld, None)
    return lib.dh_distill_topk_step(P(z), ld, P(idx), P(y), None, P(gl), N, V, K, dt, F(T), P(loss), P(grad), gld,
                                    P(ws), nbytes, None)


@pytest.mark.parametrize("which", ["loss", "backward", "step"])
def test_distill_rejects_bad_arguments(lib, which):
    call = lambda **k: distill_call(lib, which, **k)  # noqa: E731
    assert call(N=-1) == INVALID
    assert call(V=0) == INVALID
    assert call(K=0) == INVALID and call(K=1025) == INVALID
    assert call(ld=-1) == INVALID
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-45, 1e-20, 1e20):
        assert call(T=T) == INVALID
    assert call(dt=2) == UNSUPPORTED
    assert call(V=(1 << 21) + 1, ld=1 << 22, gld=1 << 22) == UNSUPPORTED
    assert call(z=0) == INVALID and call(idx=0) == INVALID and call(y=0) == INVALID
    assert call(z=FAKE + 2) == UNSUPPORTED
    assert call(N=0, z=0, idx=0, y=0, loss=0, gl=0, grad=0, ws=0) == DH_OK
    if which != "backward":
        assert call(loss=0) == INVALID
        long = dict(V=100000, ld=100000, gld=100000, grad=FAKE << 12)  # short rows need no workspace
        assert call(**long, ws=0) == WORKSPACE and call(**long, ws=FAKE * 16 + 16) == WORKSPACE
        assert call(**long, nbytes=15) == WORKSPACE
    if which != "step":
        assert call(stats=FAKE + 4) == UNSUPPORTED
    if which == "backward":
        assert call(stats=0) == INVALID
    if which != "loss":
        assert call(gl=0) == INVALID and call(grad=0) == INVALID
        assert call(gld=999) == INVALID                      # rows of the gradient would overlap
        assert call(grad=FAKE + 4000) == INVALID             # partly the logits' memory
        assert call(grad=FAKE, gld=1004) == INVALID          # the same memory in other rows
        assert call(grad=FAKE - 4) == INVALID
        assert call(grad=(FAKE << 8) + 2) == UNSUPPORTED


def test_distill_workspaces(lib):
    ws = lib.dh_distill_topk_workspace(512, 151936, binding.BF16)
    assert ws % 256 == 0 and ws >= 512 * 149 * 8  # a pair per 1024 logits
    assert lib.dh_distill_topk_step_workspace(512, 151936, 64, binding.BF16) >= ws + 512 * (8 + 64 * 4)
    assert lib.dh_distill_topk_workspace(4, 4096, binding.F32) == 0  # one launch, nothing between
    assert lib.dh_distill_topk_workspace(600, 4096, binding.F32) > 0
    assert lib.dh_distill_topk_step_workspace(600, 4096, 16, binding.F32) == 0
    for bad in ((0, 100, 0), (-1, 100, 0), (1, 0, 0), (1, 100, 2), (1, (1 << 21) + 1, 0)):
        assert lib.dh_distill_topk_workspace(*bad) == 0
        assert lib.dh_distill_topk_step_workspace(bad[0], bad[1], 8, bad[2]) == 0
    assert lib.dh_distill_topk_step_workspace(1, 100, 0, 0) == 0 == lib.dh_distill_topk_step_workspace(1, 100, 1025, 0)


def test_beam_select_rejects_bad_arguments(lib):
    def call(R=2, W=4, V=1000, M=8, dt=binding.F32, T=1.0, rs=4000, bs=1000, z=FAKE, score=FAKE, par=FAKE, tok=FAKE,
             out=FAKE, ws=FAKE * 16, nbytes=1 << 30):
        return lib.dh_beam_select(P(z), rs, bs, P(score), None, R, W, V, M, dt, F(T), 0, P(par), P(tok), P(out), P(ws),
                                  nbytes, None)
    assert call(R=-1) == INVALID and call(W=0) == INVALID and call(V=0) == INVALID and call(M=0) == INVALID
    assert call(rs=-1) == INVALID and call(bs=-1) == INVALID
    for T in (0.0, -1.0, float("nan"), float("inf")):
        assert call(T=T) == INVALID
    assert call(dt=9) == UNSUPPORTED and call(W=129) == UNSUPPORTED and call(M=257) == UNSUPPORTED
    assert call(V=(1 << 21) + 1) == UNSUPPORTED and call(z=FAKE + 1) == UNSUPPORTED
    assert call(R=1 << 30, W=4) == UNSUPPORTED
    for name in ("z", "score", "par", "tok", "out"):
        assert call(**{name: 0}) == INVALID
    assert call(ws=0) == WORKSPACE and call(ws=FAKE * 16 + 8) == WORKSPACE and call(nbytes=15) == WORKSPACE
    assert call(R=0, z=0, ws=0) == DH_OK
    assert lib.dh_beam_select_workspace(2, 4, 1024, binding.BF16) >= 8 * 8
    assert lib.dh_beam_select_workspace(2, 129, 1024, binding.BF16) == 0


def test_reorder_rejects_bad_arguments(lib):
    S = ctypes.c_int64 * 5

    def call(src=FAKE, dst=FAKE << 8, ss=(6400, 3200, 640, 160, 16), ds=None, idx=FAKE, A=2, R=2, n=5, m=5, M=4, H=4,
             T=10, unit=16):
        ds = ss if ds is None else ds
        return lib.dh_reorder_states(P(src), S(*ss) if ss else None, P(dst), S(*ds) if ds else None, P(idx), None, None,
                                     None, A, R, n, m, M, H, T, unit, None)
    for name in ("A", "R", "n", "m", "M", "H", "T", "unit"):
        assert call(**{name: -1}) == INVALID
        assert call(**{name: 0}, src=0, dst=0, idx=0) == DH_OK
    assert call(M=1025) == UNSUPPORTED
    assert call(src=0) == INVALID and call(dst=0) == INVALID and call(idx=0) == INVALID
    assert call(ss=(6400, 3200, 640, 160, -16)) == INVALID
    assert call(ds=(6400, 3200, 0, 160, 16)) == INVALID          # targets on one another
    assert call(dst=FAKE + 16) == INVALID                        # partly the source's memory
    assert call(dst=FAKE, m=4) == INVALID                        # the same memory with other slots
    assert call(dst=FAKE, ds=(6400, 3200, 640, 160, 32)) == INVALID
    assert call(unit=1 << 33, ss=(1 << 40, 1 << 39, 1 << 38, 1 << 36, 1 << 33), dst=1 << 50) == UNSUPPORTED
    big = (1 << 55, 1 << 54, 1 << 53, 1 << 35, 16)
    assert call(ss=big, dst=1 << 60, H=1 << 18, T=1 << 30) == UNSUPPORTED
    assert call(ss=big, dst=1 << 60, H=1, T=1 << 27, A=1 << 20, R=1 << 10) in (INVALID, UNSUPPORTED)


def test_binding_refuses_cpu_tensors():
    z, idx, y = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        binding.distill_topk(z, idx, y)
    with pytest.raises(ValueError, match="CUDA"):
        binding.beam_select(z[None], torch.zeros(1, 2), 2)
    with pytest.raises(ValueError, match="CUDA"):
        binding.reorder_states(torch.zeros(1, 2, 3, 4), torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="logits' rows"):
        distill.distill_loss(z, idx[:1], y)


def test_copy_dimensions():
    """Which dimensions join the contiguous unit, and which are merged."""
    d = binding._copy_dims
    assert d([(2, 800, 800), (5, 160, 160), (10, 16, 16), (8, 2, 2)], 2) == (1600, [])
    assert d([(2, 1600, 1600), (5, 160, 160), (10, 16, 16), (8, 2, 2)], 2) == (800, [(2, 1600, 1600)])
    assert d([(4, 100, 400), (1, 7, 9), (3, 32, 40), (8, 4, 4)], 4) == (32, [(4, 100, 400), (3, 32, 40)])
    assert d([(4, 300, 600), (3, 100, 200), (2, 3, 3)], 4) == (4, [(12, 100, 200), (2, 3, 3)])
    assert d([(1, 5, 5)], 2) == (2, [])
    assert d([(3, 0, 64), (8, 8, 8)], 8) == (64, [(3, 0, 64)])


@pytest.mark.parametrize("name", ["distill_topk", "distill_topk_backward", "distill_topk_step", "beam_select",
                                  "reorder_states", "distill_loss"])
def test_public_names(name):
    import speculative_decoding_draft_dh_gb300 as pkg
    assert callable(getattr(pkg, name))


def test_largest_sizes_and_smallest_temperatures(lib):
    """Row numbers that would leave 32 bits, and temperatures whose exponents' factor would overflow."""
    for which in ("loss", "backward", "step"):
        assert distill_call(lib, which, N=(1 << 31) - 1, V=1, ld=1, gld=1, K=1, grad=1 << 45) == UNSUPPORTED
    beam = lambda R, W, T: lib.dh_beam_select(  # noqa: E731
        P(FAKE), 1, 1, P(FAKE), None, R, W, 1, 1, binding.F32, F(T), 0, P(FAKE), P(FAKE), P(FAKE), P(FAKE * 16), 15,
        None)
    assert beam((1 << 31) - 1, 1, 1.0) == UNSUPPORTED and beam(1 << 24, 128, 1.0) == UNSUPPORTED
    assert beam(1, 1, 3e-39) == INVALID and beam(1, 1, 1e-38) == WORKSPACE


def test_binding_refuses_sizes_beyond_32_bits():
    n = (1 << 31) + 5
    plan = binding._reorder_plan.__wrapped__
    with pytest.raises(ValueError, match="2\\^31"):  # positions
        plan((2, 1, 2, n, 4), (2 * n * 8, 2 * n * 8, n * 8, 8, 1), (2, 1, 2, n, 4), (2 * n * 8, 2 * n * 8, n * 8, 8, 1),
             2, 1, 2, 2, 3)
    with pytest.raises(ValueError, match="2\\^31"):  # dimensions that lie together
        plan((1, 1, 2, 1 << 16, 1 << 16, 4), (1 << 36, 1 << 36, 1 << 35, 1 << 19, 8, 1), (1, 1, 2, 1 << 16, 1 << 16, 4),
             (1 << 36, 1 << 36, 1 << 35, 1 << 19, 8, 1), 2, 1, 2, 2, None)

    class Rows:  # what the check looks at of a tensor of logits that no memory here would hold
        dtype, device = torch.float32, torch.device("cuda", 0)

        def __init__(self, *shape):
            self.shape = torch.Size(shape)

        def dim(self):
            return len(self.shape)

        def get_device(self):
            return 0

        def stride(self, d):
            return 1

    with pytest.raises(ValueError, match="32 bits"):
        binding._distill_inputs(Rows(n, 1), Rows(n, 1), None, None)
    score = Rows(n, 1)
    score.is_contiguous = lambda: True
    with pytest.raises(ValueError, match="32 bits"):
        binding.beam_select(Rows(n, 1, 4), score, 1)
    score = Rows(1, 1)
    score.is_contiguous = lambda: True
    for m, pad in ((1 << 33, 0), (1, 1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            binding.beam_select(Rows(1, 1, 4), score, m, pad_token=pad)


def test_distill_selftest_rejects_bad_arguments(lib):
    def call(mode=1, row=0, us=1000, z=FAKE, nbytes=1 << 30):
        return lib.dh_selftest_distill_timeout(mode, row, us, P(z), 100000, P(FAKE), P(FAKE), P(FAKE), 2, 100000, 8,
                                               F(1.0), P(FAKE), P(FAKE << 12), 100000, P(FAKE * 16), nbytes, None)
    assert call(mode=-1) == INVALID and call(mode=4) == INVALID and call(row=-1) == INVALID
    assert call(us=0) == INVALID and call(us=1000001) == INVALID and call(z=0) == INVALID
    assert call(nbytes=15) == WORKSPACE
