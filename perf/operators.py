"""The training, search and state operators of the draft head, as they are measured.

Three groups of operators over rows of vocabulary logits and the states that follow a selection:

* ``distill``  the loss of a student's logits against a teacher's top logits, its gradient, and both
  in one call.  Row n has logits z over the vocabulary and teacher entries (id, y); with p the
  softmax of y / T over the entries and q the softmax of z / T over the vocabulary,
  loss = T^2 sum_k p_k (log p_k - log q[id_k]) and dz[v] = g T (q[v] - sum of p_k with id_k = v).
  A row without entries has loss 0 and gradient 0; a row whose weight g is 0 has gradient 0.
* ``beam``  one step of beam search: over the beams w and the vocabulary v of a request, the M best
  of score[w] + z[w, v] / T - log sum exp(z[w, :] / T), ordered by score, then beam, then token.  A
  finished beam has one candidate, the padding token at its own score.
* ``reorder``  states moved as a selection says: slot j of the target takes slot idx[j] of the
  source, for the positions below a request's length; everything else stays as it was.

Where ``own`` is false ``run`` computes them with elementary torch operations.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# A pass reads or writes at most this many logits (the largest listed cases have 2048 x 151936) and
# moves at most this many bytes of states.
MAX_LOGITS = 2048 * 151936
MAX_STATE = 1 << 31


def listed():
    return [
        # One speculative round's rows checked against the full-rank head's candidates: the loss
        # alone, at the sizes of the tiny head.
        {"name": "distill_loss_tiny", "op": "distill", "dir": "loss", "N": 4, "vocab": 4096, "K": 16, "dtype": "f32",
         "T": 1.0, "ragged": False, "ld": 4096},
        # An evaluation pass of the candidate head over a batch of positions.
        {"name": "distill_loss_eval", "op": "distill", "dir": "loss", "N": 512, "vocab": 151936, "K": 256,
         "dtype": "bf16", "T": 1.0, "ragged": False, "ld": 151936},
        # The gradient alone, as the autograd form runs it after a forward pass.
        {"name": "distill_backward", "op": "distill", "dir": "backward", "N": 1024, "vocab": 151936, "K": 128,
         "dtype": "bf16", "T": 2.0, "ragged": True, "ld": 151936},
        # A training step's loss and gradient in one call: the largest batch.
        {"name": "distill_step", "op": "distill", "dir": "step", "N": 2048, "vocab": 151936, "K": 64, "dtype": "bf16",
         "T": 1.0, "ragged": False, "ld": 151936},
        # A vocabulary that is no multiple of anything, packed rows, fp32, ragged teachers.
        {"name": "distill_step_odd", "op": "distill", "dir": "step", "N": 333, "vocab": 50257, "K": 50, "dtype": "f32",
         "T": 1.5, "ragged": True, "ld": 50257},
        # One request's beams: the latency of a step.
        {"name": "beam_single", "op": "beam", "R": 1, "W": 4, "vocab": 151936, "M": 4, "dtype": "bf16", "T": 1.0,
         "finished": False, "ld": 151936},
        # A serving batch, some of whose beams have ended.
        {"name": "beam_batch", "op": "beam", "R": 32, "W": 8, "vocab": 151936, "M": 16, "dtype": "bf16", "T": 1.0,
         "finished": True, "ld": 151936},
        # Odd vocabulary inside padded fp32 rows, wide beams.
        {"name": "beam_odd", "op": "beam", "R": 24, "W": 16, "vocab": 50257, "M": 32, "dtype": "f32", "T": 0.75,
         "finished": True, "ld": 50304},
        # The largest selection: many requests with wide beams.
        {"name": "beam_wide", "op": "beam", "R": 128, "W": 16, "vocab": 151936, "M": 16, "dtype": "bf16", "T": 1.0,
         "finished": False, "ld": 151936},
        # A draft layer's cache of one request follows its four beams.
        {"name": "reorder_single", "op": "reorder", "form": "beams", "A": 2, "R": 1, "W": 4, "H": 8, "T": 700,
         "D": 128, "M": 4, "dtype": "bf16", "out_T": 0},
        # Long caches of a batch of beams, lengths from a quarter to the whole of them.
        {"name": "reorder_long", "op": "reorder", "form": "beams", "A": 4, "R": 8, "W": 8, "H": 8, "T": 4096,
         "D": 128, "M": 8, "dtype": "bf16", "out_T": 0},
        # The accepted path of a 64-node draft tree appended to the committed cache.
        {"name": "reorder_append", "op": "reorder", "form": "append", "A": 8, "R": 64, "W": 64, "H": 8, "T": 1,
         "D": 128, "M": 11, "dtype": "bf16", "out_T": 512},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["distill", "distill", "beam", "beam", "reorder"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "reorder":
        A, H, D = rng.randint(1, 8), rng.randint(1, 8), rng.choice([24, 64, 80, 128])
        size = 4 if dtype == "f32" else 2
        if rng.random() < 0.5:
            R, W = _log_int(rng, 1, 32), rng.randint(1, 16)
            most = max(1, MAX_STATE // (A * R * W * H * D * size))
            T = _log_int(rng, 1, min(4096, most))
            return {"op": op, "form": "beams", "A": A, "R": R, "W": W, "H": H, "T": T, "D": D, "M": W, "dtype": dtype,
                    "out_T": 0}
        R, W = _log_int(rng, 1, 64), rng.randint(8, 96)
        return {"op": op, "form": "append", "A": A, "R": R, "W": W, "H": H, "T": 1, "D": D, "M": rng.randint(2, 12),
                "dtype": dtype, "out_T": rng.randint(32, 512)}
    vocab = _log_int(rng, 1000, 151936)
    ld = vocab if rng.random() < 0.5 else (vocab + 63) // 64 * 64
    # a 32-bit logit is counted as two
    rows = max(1, MAX_LOGITS // (ld * (2 if dtype == "f32" else 1)))
    T = rng.choice([1.0, rng.randint(32, 192) / 64])
    if op == "distill":
        return {"op": op, "dir": rng.choice(["loss", "backward", "step"]), "N": _log_int(rng, 1, min(2048, rows)),
                "vocab": vocab, "K": _log_int(rng, 1, 256), "dtype": dtype, "T": T, "ragged": rng.random() < 0.5,
                "ld": ld}
    W = rng.randint(1, 16)
    return {"op": op, "R": _log_int(rng, 1, max(1, min(128, rows // W))), "W": W, "vocab": vocab,
            "M": rng.randint(W, 2 * W), "dtype": dtype, "T": T, "finished": rng.random() < 0.5, "ld": ld}


# ---------------------------------------------------------------- inputs

def _logit_rows(g, n, case):
    """n rows of `vocab` logits, 3 N(0, 1), in rows of `ld` elements; the storage dtype's values."""
    buf = torch.empty(n, case["ld"], dtype=DTYPES[case["dtype"]], device="cuda")
    buf.normal_(0.0, 3.0, generator=g)
    return buf[:, :case["vocab"]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "distill":
        N, K, V = case["N"], case["K"], case["vocab"]
        z = _logit_rows(g, N, case)
        # the teacher agrees with the student in part: its K best ids come from a noisy reading of
        # the student's logits, with the noisy values, the best first
        y = torch.empty(N, K, dtype=torch.float32, device="cuda")
        ids = torch.empty(N, K, dtype=torch.int32, device="cuda")
        for at in range(0, N, 256):
            noisy = z[at:at + 256].float()
            noisy += 2.0 * torch.randn(noisy.shape, generator=g, device="cuda")
            best = noisy.topk(K, dim=1)
            y[at:at + 256], ids[at:at + 256] = best.values, best.indices.int()
        n_valid, weight = _rows(case)
        n_valid = torch.tensor(n_valid, dtype=torch.int32, device="cuda") if case["ragged"] else None
        weight = torch.tensor(weight, dtype=torch.float32, device="cuda")
        state.update(logits=z, idx=ids, teacher=y, n_valid=n_valid, weight=weight)
        if case["dir"] == "backward":
            # what the forward pass left: each row's maximum and the sum of exp((z - max) / T)
            stats = torch.empty(N, 2, dtype=torch.float32, device="cuda")
            for at in range(0, N, 128):
                zz = z[at:at + 128].double()
                m = zz.amax(dim=1, keepdim=True)
                stats[at:at + 128, 0] = m[:, 0].float()
                stats[at:at + 128, 1] = ((zz - m) / case["T"]).exp().sum(dim=1).float()
            state["stats"] = stats
    elif case["op"] == "beam":
        R, W, V = case["R"], case["W"], case["vocab"]
        rows = _logit_rows(g, R * W, case)
        # a few likely tokens in every row, as a model's rows have
        hot = torch.randint(0, V, (R * W, 8), generator=g, device="cuda")
        lift = 8.0 + 3.0 * torch.rand(R * W, 8, generator=g, device="cuda")
        rows.scatter_(1, hot, (rows.gather(1, hot).float() + lift).to(rows.dtype))
        score = -10.0 * torch.rand(R, W, generator=g, device="cuda")
        score = score.sort(dim=1, descending=True).values.contiguous()
        finished = None
        if case["finished"]:
            finished = torch.tensor(_finished(case), dtype=torch.int32, device="cuda").view(R, W)
        state.update(logits=rows.view(R, W, case["vocab"]) if case["ld"] == V else
                     rows.as_strided((R, W, V), (W * case["ld"], case["ld"], 1)), score=score, finished=finished)
    else:
        A, R, W, H, T, D, M = (case[k] for k in ("A", "R", "W", "H", "T", "D", "M"))
        dt = DTYPES[case["dtype"]]
        if case["form"] == "beams":
            src = torch.empty(A, R, W, H, T, D, dtype=dt, device="cuda").normal_(generator=g)
            dst = torch.zeros_like(src)
            # two beams of three survive; each keeps a slot at least and the rest branch from them
            S = _survivors(W)
            keys = torch.rand(R, W, generator=g, device="cuda")
            alive = keys.argsort(dim=1)[:, :S]
            more = torch.randint(0, S, (R, W - S), generator=g, device="cuda")
            idx = torch.cat([alive, alive.gather(1, more)], dim=1)
            idx = idx.gather(1, torch.rand(R, W, generator=g, device="cuda").argsort(dim=1)).int().contiguous()
            state.update(src=src, dst=dst, idx=idx, lengths=torch.tensor(_lengths(case), dtype=torch.int32, device="cuda"))
        else:
            src = torch.empty(A, R, W, H, D, dtype=dt, device="cuda").normal_(generator=g)
            dst = torch.zeros(A, R, H, case["out_T"], D, dtype=dt, device="cuda")
            # an accepted path: ascending node numbers from the root, then -1
            n = torch.tensor(_lengths(case), device="cuda")
            path = torch.rand(R, W, generator=g, device="cuda").argsort(dim=1)[:, :M].sort(dim=1).values
            path = torch.where(torch.arange(M, device="cuda") < n[:, None], path, torch.full_like(path, -1))
            base = torch.randint(0, case["out_T"] - M + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
            state.update(src=src, dst=dst, idx=path.int().contiguous(), base=base)
    return state


def _rows(case):
    """The teacher's entries and the weight of each row.  Ragged: short teachers, some without any
    entry, and one position in ten that does not count."""
    N, K = case["N"], case["K"]
    if not case["ragged"]:
        return [K] * N, [1.0 / N] * N
    return [(7919 * n + 5) % (K + 1) for n in range(N)], [0.0 if n % 10 == 3 else 1.0 / N for n in range(N)]


def _finished(case):
    return [1 if case["finished"] and n % 5 == 2 else 0 for n in range(case["R"] * case["W"])]


def _survivors(W):
    return (2 * W + 2) // 3


def _lengths(case):
    """Beams: the positions that each request's cache holds, from a quarter of it to all.  Append:
    the accepted nodes of each request's path, from one to all."""
    R, T, M = case["R"], case["T"], case["M"]
    if case["form"] == "beams":
        return [T if R == 1 else max(1, T // 4 + (T - T // 4) * r // (R - 1)) for r in range(R)]
    return [1 + (5 * r + 2) % min(M, case["W"]) for r in range(R)]


# ---------------------------------------------------------------- the plain forms

def _teacher(ids, y, n_valid, vocab, T):
    """(kept entries, p) of the teacher's rows; p is 0 where an entry is not kept."""
    keep = (ids >= 0) & (ids < vocab)
    if n_valid is not None:
        keep = keep & (torch.arange(ids.shape[1], device=ids.device) < n_valid[:, None])
    top = torch.where(keep, y, torch.full_like(y, -math.inf)).amax(dim=1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    e = torch.where(keep, ((y - top) / T).exp(), torch.zeros_like(y))
    total = e.sum(dim=1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    log_p = (y - top) / T - torch.where(total > 0, total, torch.ones_like(total)).log()
    return keep, p, log_p


def _plain_distill(s):
    case = s["case"]
    T, V = case["T"], case["vocab"]
    z = s["logits"].float()
    keep, p, log_p = _teacher(s["idx"], s["teacher"], s["n_valid"], V, T)
    at = torch.where(keep, s["idx"], torch.zeros_like(s["idx"])).long()
    if case["dir"] == "backward":
        top, total = s["stats"][:, :1], s["stats"][:, 1:]
    else:
        top = z.amax(dim=1, keepdim=True)
        total = ((z - top) / T).exp().sum(dim=1, keepdim=True)
    if case["dir"] != "backward":
        log_q = (z.gather(1, at) - top) / T - total.log()
        loss = T * T * torch.where(p > 0, p * (log_p - log_q), torch.zeros_like(p)).sum(dim=1)
        if case["dir"] == "loss":
            return {"loss": loss, "stats": torch.cat([top, total], dim=1)}
    grad = ((z - top) / T).exp() / total
    grad.scatter_add_(1, at, -p)
    grad *= (s["weight"] * T * keep.any(dim=1))[:, None]
    grad = grad.to(s["logits"].dtype)
    return {"grad": grad} if case["dir"] == "backward" else {"loss": loss, "grad": grad}


def _plain_beam(s):
    case = s["case"]
    R, W, V, M = (case[k] for k in ("R", "W", "vocab", "M"))
    # in 64 bits: the order of two candidates of different beams hangs on the rows' sums
    z = s["logits"].double() / case["T"]
    top = z.amax(dim=2, keepdim=True)
    total = top + (z - top).exp().sum(dim=2, keepdim=True).log()
    z += s["score"].double()[:, :, None] - total
    if s["finished"] is not None:
        done = s["finished"][:, :, None] != 0
        z = torch.where(done, torch.full_like(z, -math.inf), z)
        z[:, :, :1] = torch.where(done, s["score"].double()[:, :, None], z[:, :, :1])
    flat = z.view(R, W * V)
    last = flat.topk(M, dim=1).values[:, -1:]
    # of the entries equal to the last, the first ones
    above, level = flat > last, flat == last
    room = M - above.sum(dim=1, keepdim=True)
    at = (above | (level & (level.cumsum(dim=1) <= room))).nonzero()[:, 1].view(R, M)
    best = flat.gather(1, at).sort(dim=1, descending=True, stable=True)
    at = at.gather(1, best.indices)
    live = best.values > -math.inf
    parent = torch.where(live, at // V, torch.full_like(at, -1)).int()
    token = torch.where(live, at % V, torch.full_like(at, -1)).int()
    if s["finished"] is not None:
        ended = live & (s["finished"].gather(1, parent.clamp(min=0).long()) != 0)
        token = torch.where(ended, torch.full_like(token, PAD), token)
    return {"parent": parent, "token": token, "score": best.values.float()}


def _plain_reorder(s):
    case = s["case"]
    A, R, H, T, D, M = (case[k] for k in ("A", "R", "H", "T", "D", "M"))
    if case["form"] == "beams":
        rows = torch.arange(R, device="cuda")[:, None]
        held = torch.arange(T, device="cuda") < s["lengths"][:, None]
        moved = s["src"][:, rows, s["idx"].long()]
        s["dst"].copy_(torch.where(held[None, :, None, None, :, None], moved, s["dst"]))
    else:
        r, j = (s["idx"] >= 0).nonzero(as_tuple=True)
        s["dst"][:, r, :, s["base"][r].long() + j] = s["src"][:, r, s["idx"][r, j].long()].transpose(0, 1)
    return {"states": s["dst"]}


PAD = 0  # the token of a finished beam's candidate


def run(state):
    case = state["case"]
    if own:
        from speculative_decoding_draft_dh_gb300 import binding as dh
        if case["op"] == "distill":
            a = (state["logits"], state["idx"], state["teacher"])
            kw = {"n_valid": state["n_valid"], "temperature": case["T"]}
            if case["dir"] == "loss":
                loss, stats = dh.distill_topk(*a, **kw)
                return {"loss": loss, "stats": stats}
            if case["dir"] == "backward":
                return {"grad": dh.distill_topk_backward(*a, state["stats"], state["weight"], **kw)}
            loss, grad = dh.distill_topk_step(*a, state["weight"], **kw)
            return {"loss": loss, "grad": grad}
        if case["op"] == "beam":
            parent, token, score = dh.beam_select(state["logits"], state["score"], case["M"],
                                                  finished=state["finished"], pad_token=PAD, temperature=case["T"])
            return {"parent": parent, "token": token, "score": score}
        if case["form"] == "beams":
            return {"states": dh.reorder_states(state["src"], state["idx"], out=state["dst"],
                                                lengths=state["lengths"], length_dim=4)}
        return {"states": dh.reorder_states(state["src"], state["idx"], out=state["dst"], dst_base=state["base"],
                                            out_slot_dim=3)}
    return {"distill": _plain_distill, "beam": _plain_beam, "reorder": _plain_reorder}[case["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "distill":
        # the gradients' rows without entries are not read, nor those of weight 0 for the gradient alone
        n_valid, weight = _rows(case)
        rows = sum(1 for v, w in zip(n_valid, weight)
                   if case["dir"] == "loss" or v and (w or case["dir"] == "step"))
        small, n = 8 * sum(n_valid) + 8 * case["N"], rows * case["vocab"]
        if case["dir"] == "loss":
            return {"bytes": n * size + small, "flops": 4 * n}
        return {"bytes": (n + case["N"] * case["vocab"]) * size + small,
                "flops": (5 if case["dir"] == "backward" else 8) * n}
    if case["op"] == "beam":
        n = (case["R"] * case["W"] - sum(_finished(case))) * case["vocab"]
        return {"bytes": n * size + 4 * case["R"] * case["W"] + 12 * case["R"] * case["M"], "flops": 4 * n}
    one = case["A"] * case["H"] * case["D"] * size
    if case["form"] == "beams":
        return {"bytes": sum(_lengths(case)) * one * (_survivors(case["W"]) + case["M"]), "flops": 0}
    return {"bytes": sum(_lengths(case)) * one * 2, "flops": 0}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    if case["op"] == "reorder":
        return None  # values are moved, not computed
    s = prepare(case, seed)
    if case["op"] == "beam":
        logp = torch.log_softmax(s["logits"].double().div_(case["T"]), dim=-1)
        out = s["score"].double().unsqueeze(-1) + logp
        del logp
        if s["finished"] is not None:
            done = s["finished"].bool()
            out[done] = -math.inf
            out[..., 0][done] = s["score"].double()[done]
        best = out.flatten(1).topk(case["M"], dim=1).values
        return {"parent": None, "token": None, "score": best}
    T, V = case["T"], case["vocab"]
    out = {"loss": [], "stats": [], "grad": []}
    for at in range(0, case["N"], 256):
        rows = slice(at, at + 256)
        logq = torch.log_softmax(s["logits"][rows].double() / T, dim=1)
        ids, y = s["idx"][rows].long(), s["teacher"][rows].double() / T
        if s["n_valid"] is not None:
            y = y.masked_fill(torch.arange(y.shape[1], device=y.device)[None] >= s["n_valid"][rows][:, None], -math.inf)
        none = (y == -math.inf).all(dim=1)
        logp = torch.log_softmax(y.masked_fill(none[:, None], 0.0), dim=1)
        p = logp.exp().masked_fill(none[:, None], 0.0)
        kl = torch.where(p > 0, p * (logp - logq.gather(1, ids)), 0.0).sum(dim=1)
        out["loss"].append(T * T * kl)
        if case["dir"] == "loss":
            # 1 / q at the row's largest logit is the sum of the exponentials relative to it
            out["stats"].append(torch.stack([s["logits"][rows].double().amax(dim=1), (-logq.amax(dim=1)).exp()], dim=1))
        if case["dir"] != "loss":
            grad = logq.exp()
            grad = grad - torch.zeros_like(grad).scatter_add_(1, ids, p)
            grad = grad * (s["weight"][rows].double() * T)[:, None]
            out["grad"].append(grad.masked_fill(none[:, None], 0.0))
    want = {"loss": ["loss", "stats"], "backward": ["grad"], "step": ["loss", "grad"]}[case["dir"]]
    return {k: torch.cat(out[k]) for k in want}
