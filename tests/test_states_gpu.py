"""Reordering of states (dh_reorder_states) against plain indexing, bit for bit: what moves, and
everything that must stay."""
import numpy as np
import pytest
import torch

from speculative_decoding_draft_dh_gb300 import binding as dh
from speculative_decoding_draft_dh_gb300 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def expect(states, idx, out=None, lengths=None, length_dim=None, src_base=None, dst_base=None, request_dim=1,
           slot_dim=2, out_slot_dim=None):
    """The definition, slot by slot, on copies."""
    osd = slot_dim if out_slot_dim is None else out_slot_dim
    src = states.clone()
    dst = (states if out is None else out).clone()
    R, M = idx.shape
    for r in range(R):
        sb = 0 if src_base is None else int(src_base[r])
        db = 0 if dst_base is None else int(dst_base[r])
        for j in range(M):
            p = int(idx[r, j])
            if p < 0 or not 0 <= sb + p < src.shape[slot_dim] or not 0 <= db + j < dst.shape[osd]:
                continue
            s, d = src.select(request_dim, r), dst.select(request_dim, r)
            s = s.select(slot_dim - (slot_dim > request_dim), sb + p)
            d = d.select(osd - (osd > request_dim), db + j)
            if lengths is not None:
                ld = length_dim - (length_dim > request_dim) - (length_dim > slot_dim)
                n = min(max(int(lengths[r]), 0), s.shape[ld])
                d.narrow(ld, 0, n).copy_(s.narrow(ld, 0, n))
            else:
                d.copy_(s)
    return dst


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def check(states, idx, **kw):
    want = expect(states, idx, **kw)
    got = dh.reorder_states(states, idx, **kw)
    torch.cuda.synchronize()
    assert got.data_ptr() == (states if kw.get("out") is None else kw["out"]).data_ptr()
    assert same(got, want)


def rand(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    if dtype in (torch.int8, torch.uint8, torch.int64):
        return torch.randint(0, 100, shape, generator=g).to(dtype).to(DEV)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


def parents(R, M, W, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1, W, (R, M), generator=g).int().to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float64, torch.int8])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("A,R,W,H,T,D", [(1, 1, 1, 1, 1, 1), (2, 3, 4, 2, 5, 8), (1, 2, 8, 3, 7, 80), (2, 1, 16, 1, 33, 3),
                                         (1, 2, 17, 2, 3, 64), (1, 3, 40, 1, 2, 24), (3, 5, 5, 2, 130, 16)])
def test_beams(A, R, W, H, T, D, in_place, dtype):
    x = rand((A, R, W, H, T, D), dtype, seed=W)
    idx = parents(R, W, W, seed=T)
    lengths = torch.tensor([(7 * r) % (T + 2) for r in range(R)], dtype=torch.int32, device=DEV)
    for kw in ({}, dict(lengths=lengths, length_dim=4)):
        if in_place:
            check(x.clone(), idx, **kw)
        else:
            check(x, idx, out=rand(x.shape, dtype, seed=99), **kw)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("M", [1, 8, 16, 17, 100, 1000, 1024])
def test_many_slots(M, in_place):
    """More moves than registers hold, in place: reversal, rotation, everything from one slot."""
    x = rand((1, 2, M, 5, 40), torch.float32, seed=M)
    i = torch.arange(M, device=DEV)
    for idx in (i.flip(0), (i + 1) % M, i * 0 + M // 2, i, torch.randperm(M, generator=torch.Generator().manual_seed(M)).to(DEV)):
        idx = torch.stack([idx, i]).int().contiguous()
        check(x.clone(), idx, **({} if in_place else {"out": torch.zeros_like(x)}))


def test_layouts():
    """Slots and positions in other places, strided and expanded sources, odd addresses."""
    x = rand((3, 4, 6, 5, 10), torch.bfloat16)
    idx = parents(4, 6, 6, seed=3)
    check(x.clone(), idx)
    # positions before the heads, contiguous per position
    n = torch.tensor([0, 2, 5, 9], dtype=torch.int32, device=DEV)
    check(x.clone(), idx, lengths=n, length_dim=3)
    # requests first, slots second
    check(x.clone(), parents(3, 4, 4, seed=4), request_dim=0, slot_dim=1)
    # slots last: every element a unit of its own
    check(x.clone(), parents(4, 10, 10, seed=5), slot_dim=4)
    # a wider buffer's part, at an odd place
    big = rand((3, 4, 6, 5, 13), torch.bfloat16, seed=7)
    check(big[..., 1:11], idx)
    flat = rand((3 * 4 * 6 * 50 + 3,), torch.bfloat16, seed=8)
    check(flat[3:].view(3, 4, 6, 50), idx)
    # one source for all layers
    check(x[:1].expand(3, -1, -1, -1, -1), idx, out=torch.zeros_like(x))
    # transposed target
    out = torch.zeros(3, 6, 4, 5, 10, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    check(x, idx, out=out)


def test_bases_and_entries_that_do_not_exist():
    x = rand((2, 4, 9, 16), torch.float32)
    idx = torch.tensor([[0, 3, -1, 8], [8, 9, 2 ** 31 - 1, 0], [-2 ** 31, 1, 2, 3], [5, 5, 5, 5]], dtype=torch.int32,
                       device=DEV)
    sb = torch.tensor([0, 0, -1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    db = torch.tensor([7, -2, 0, 1], dtype=torch.int32, device=DEV)
    for kw in (dict(src_base=sb), dict(dst_base=db), dict(src_base=sb, dst_base=db)):
        check(x.clone(), idx, **kw)
        check(x, idx, out=rand((2, 4, 6, 16), torch.float32, seed=5), **kw)


def test_accepted_path_is_appended():
    """Tree acceptance's path moves the tree's states behind the committed ones, out of a scratch of
    their own and within one cache."""
    cfg = inputs.tree_config("tiny_tree", B=5, N=8)
    t = inputs.make_tree(cfg, seed=4, device=DEV)
    acc = dh.tree_accept(t["logits"], t["parent"], t["token"])
    tree = rand((2, 5, 8, 3, 16), torch.bfloat16, seed=1)       # layers, requests, nodes, heads, size
    cache = rand((2, 5, 3, 40, 16), torch.bfloat16, seed=2)     # layers, requests, heads, positions, size
    held = torch.tensor([0, 7, 31, 32, 39], dtype=torch.int32, device=DEV)
    check(tree, acc["path"], out=cache, dst_base=held, out_slot_dim=3)
    n = (acc["len"] + 1).cpu()
    for r in range(5):
        for i in range(min(int(n[r]), 40 - int(held[r]))):
            assert torch.equal(cache[:, r, :, int(held[r]) + i], tree[:, r, int(acc["path"][r, i])])
    check(cache.clone(), acc["path"], src_base=held, dst_base=held, slot_dim=3)


def test_long_cache_beyond_32_bits():
    """Offsets of more than 2^32 bytes, in both forms."""
    x = torch.zeros(2, 2, 3, 4, 100000, 512, dtype=torch.bfloat16, device=DEV)  # 4.9 GB
    x[..., 0] = torch.arange(48, device=DEV).view(2, 2, 3, 4, 1).to(torch.bfloat16)
    assert x.numel() * 2 > 2 ** 32
    idx = torch.tensor([[2, 0, 0], [1, 2, 0]], dtype=torch.int32, device=DEV)
    n = torch.tensor([100000, 99999], dtype=torch.int32, device=DEV)
    want = x[..., 0].clone()
    for r in range(2):
        want[:, r, :, :, :int(n[r])] = x[..., 0][:, r][:, idx[r].long()][..., :int(n[r])]
    out = torch.zeros_like(x)
    out[..., 0] = x[..., 0]
    dh.reorder_states(x, idx, out=out, lengths=n, length_dim=4)
    assert torch.equal(out[..., 0], want)
    dh.reorder_states(x, idx, lengths=n, length_dim=4)
    assert torch.equal(x[..., 0], want) and not x[..., 1:].any()


def test_empty_sizes_and_graphs():
    x = rand((2, 3, 4, 8), torch.float32)
    keep = x.clone()
    dh.reorder_states(x, torch.zeros(3, 0, dtype=torch.int32, device=DEV))
    dh.reorder_states(x[:0], parents(3, 4, 4))
    dh.reorder_states(x, parents(3, 4, 4), lengths=torch.zeros(3, dtype=torch.int32, device=DEV), length_dim=3)
    assert torch.equal(x, keep)
    idx = parents(3, 4, 4, seed=2)
    want = expect(expect(x, idx), idx)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dh.reorder_states(x, idx)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dh.reorder_states(x, idx, stream=s)
    s.synchronize()
    assert torch.equal(x, expect(want, idx))


def test_refusals():
    x = rand((2, 3, 4, 8), torch.float32)
    idx = parents(3, 4, 4)
    n = torch.ones(3, dtype=torch.int32, device=DEV)
    for bad in (lambda: dh.reorder_states(x.cpu(), idx), lambda: dh.reorder_states(x, idx.long()),
                lambda: dh.reorder_states(x, idx[:2]), lambda: dh.reorder_states(x, idx.cpu()),
                lambda: dh.reorder_states(x, idx, lengths=n), lambda: dh.reorder_states(x, idx, length_dim=3),
                lambda: dh.reorder_states(x, idx, lengths=n, length_dim=2),
                lambda: dh.reorder_states(x, idx, request_dim=2), lambda: dh.reorder_states(x, idx, slot_dim=4),
                lambda: dh.reorder_states(x, idx, out=x.double()), lambda: dh.reorder_states(x, idx, out=x[:1]),
                lambda: dh.reorder_states(x, idx, out=torch.empty(2, 3, 4, 9, device=DEV)),
                lambda: dh.reorder_states(x, idx, out=x[:, :, :1].expand(2, 3, 4, 8)),
                lambda: dh.reorder_states(x[:, :, :1].expand(2, 3, 4, 8), idx),
                lambda: dh.reorder_states(rand((2, 3, 4, 2, 6, 6), torch.float32)[..., ::2, ::3, ::2], idx)):
        with pytest.raises(ValueError):
            bad()
    leaf = x.clone().requires_grad_(True)
    with pytest.raises(ValueError, match="autograd"):
        dh.reorder_states(leaf, idx)
    with torch.no_grad():
        assert dh.reorder_states(leaf, idx) is leaf
    with pytest.raises(dh.DhError):  # partly the same memory
        dh.reorder_states(x[:, :, 1:], parents(3, 3, 3), out=x[:, :, :3])
    with pytest.raises(dh.DhError):
        dh.reorder_states(x, torch.zeros(3, 1025, dtype=torch.int32, device=DEV))


def test_conjugate_views():
    """A conjugate view holds other bits than it shows: it moves among such views alone."""
    x = torch.randn(1, 1, 3, 4, dtype=torch.complex64, device=DEV)
    idx = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    with pytest.raises(ValueError, match="conjugate"):
        dh.reorder_states(x.conj(), idx, out=out)
    got = dh.reorder_states(x.conj(), idx, out=out.conj())
    torch.cuda.synchronize()
    assert torch.equal(got.resolve_conj(), x.conj().resolve_conj()[:, :, [2, 0, 1]])
