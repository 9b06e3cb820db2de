"""The operators between a row of logits and the head's next hidden rows, as they are measured.

* ``sample``  one token per row of vocabulary logits from a given uniform, with temperature, top-k, top-p and
  min-p.  In the order of a row's tokens by logit (equal ones by id), with w = exp((z - max z) / T): top-k keeps the
  first k, top-p of those the first ones up to and with the one at which the running sum of w reaches top_p of their
  mass, min-p those with w >= min_p.  The token is the first kept one whose running sum exceeds u times the kept mass,
  and its probability is its share of that mass.  Temperature 0 takes the first one, with probability 1.
* ``embed``   rows of a table looked up by token and scaled; the table's gradient, the scaled sum of the rows'
  gradients per token.  A token outside the vocabulary (padding) has a row of zeros and no gradient.
* ``norm``    layer norm over the last dimension, with weight and bias; its gradients.

Where ``own`` is false ``run`` computes them with elementary torch operations.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}

# The largest passes: logits of a sampling batch, elements of a table and of a batch of hidden rows (a 32-bit
# element is counted as two).
MAX_LOGITS = 512 * 151936
MAX_TABLE = 151936 * 5120
MAX_ROWS = 32768 * 5120
EPS = 1e-5


def listed():
    return [
        # One request's next token with a chat model's usual settings: latency.
        {"name": "sample_single", "op": "sample", "N": 1, "vocab": 151936, "dtype": "bf16", "ld": 151936, "mix": False,
         "T": 0.7, "k": 20, "p": 0.8, "m": 0.0},
        # A serving batch whose requests each bring their own settings.
        {"name": "sample_batch", "op": "sample", "N": 256, "vocab": 151936, "dtype": "bf16", "ld": 151936, "mix": True,
         "T": 1.0, "k": 0, "p": 1.0, "m": 0.0},
        # Odd vocabulary in padded fp32 rows, wide top-k and min-p.
        {"name": "sample_odd", "op": "sample", "N": 77, "vocab": 50257, "dtype": "f32", "ld": 50304, "mix": False,
         "T": 1.3, "k": 400, "p": 0.97, "m": 0.002},
        # The largest batch, top-p over the whole vocabulary: no top-k bounds what is kept.
        {"name": "sample_nucleus", "op": "sample", "N": 512, "vocab": 151936, "dtype": "bf16", "ld": 151936,
         "mix": False, "T": 1.0, "k": 0, "p": 0.95, "m": 0.0},
        # The tokens of one draft level: latency.
        {"name": "embed_level", "op": "embed", "dir": "forward", "N": 8, "vocab": 151936, "d": 5120, "dtype": "bf16",
         "scale": 1.0, "padded": False},
        # A training batch of 8 sequences of 4096 tokens.
        {"name": "embed_batch", "op": "embed", "dir": "forward", "N": 32768, "vocab": 151936, "d": 5120,
         "dtype": "bf16", "scale": 71.5, "padded": True},
        # The gradient of the whole table from that many tokens.
        {"name": "embed_backward", "op": "embed", "dir": "backward", "N": 32768, "vocab": 151936, "d": 5120,
         "dtype": "bf16", "scale": 71.5, "padded": True},
        # A small fp32 table with an odd width and more tokens than rows.
        {"name": "embed_backward_odd", "op": "embed", "dir": "backward", "N": 20011, "vocab": 4096, "d": 1001,
         "dtype": "f32", "scale": 0.5, "padded": False},
        # The hidden rows of one draft level before the head: latency, no statistics kept.
        {"name": "norm_level", "op": "norm", "dir": "forward", "N": 8, "d": 5120, "dtype": "bf16", "params": "bf16",
         "stats": False},
        # A training batch's hidden rows.
        {"name": "norm_batch", "op": "norm", "dir": "forward", "N": 32768, "d": 5120, "dtype": "bf16",
         "params": "bf16", "stats": True},
        # Their gradients, those of 32-bit weights among them.
        {"name": "norm_backward", "op": "norm", "dir": "backward", "N": 32768, "d": 5120, "dtype": "bf16",
         "params": "f32", "stats": True},
        # Odd fp32 rows.
        {"name": "norm_backward_odd", "op": "norm", "dir": "backward", "N": 4097, "d": 1001, "dtype": "f32",
         "params": "f32", "stats": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "embed", "norm"])
    dtype = rng.choice(["f32", "bf16"])
    weight = 2 if dtype == "f32" else 1
    if op == "sample":
        vocab = _log_int(rng, 1000, 151936)
        ld = vocab if rng.random() < 0.5 else (vocab + 63) // 64 * 64
        return {"op": op, "N": _log_int(rng, 1, min(512, MAX_LOGITS // (ld * weight))), "vocab": vocab, "dtype": dtype,
                "ld": ld, "mix": rng.random() < 0.4, "T": rng.choice([1.0, rng.randint(16, 128) / 64]),
                "k": rng.choice([0, _log_int(rng, 1, 1000)]), "p": rng.choice([1.0, rng.randint(16, 63) / 64]),
                "m": rng.choice([0.0, rng.randint(1, 64) / 512])}
    if op == "embed":
        d = _log_int(rng, 16, 8192)
        vocab = _log_int(rng, 1000, min(151936, MAX_TABLE // (d * weight)))
        return {"op": op, "dir": rng.choice(["forward", "backward"]), "vocab": vocab, "d": d, "dtype": dtype,
                "N": _log_int(rng, 1, min(32768, MAX_ROWS // (d * weight))), "scale": rng.choice([1.0, 0.5, 71.5]),
                "padded": rng.random() < 0.5}
    d = _log_int(rng, 16, 8192)
    return {"op": op, "dir": rng.choice(["forward", "backward"]), "d": d, "dtype": dtype,
            "N": _log_int(rng, 1, min(65536, MAX_ROWS // (d * weight))), "params": rng.choice([dtype, "f32"]),
            "stats": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

# What the requests of a mixed batch ask for, one after another: (temperature, top-k, top-p, min-p).
REQUESTS = [(0.7, 20, 0.8, 0.0), (1.0, 0, 0.95, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 50, 1.0, 0.0), (0.6, 20, 0.95, 0.0),
            (1.25, 0, 1.0, 0.0625), (0.75, 40, 0.9, 0.05), (1.0, 0, 1.0, 0.0), (0.5, 1000, 0.5, 0.0)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    N, dt = case["N"], DTYPES[case["dtype"]]
    if case["op"] == "sample":
        V = case["vocab"]
        rows = torch.empty(N, case["ld"], dtype=dt, device="cuda").normal_(0.0, 2.5, generator=g)
        # likely tokens over a long tail, as a model's rows have
        hot = torch.randint(0, V, (N, 32), generator=g, device="cuda")
        lift = 6.0 + 10.0 * torch.rand(N, 32, generator=g, device="cuda")
        rows.scatter_(1, hot, (rows.gather(1, hot).float() + lift).to(dt))
        state.update(logits=rows[:, :V], u=torch.rand(N, generator=g, device="cuda"))
        ask = [REQUESTS[n % len(REQUESTS)] for n in range(N)] if case["mix"] else None
        for i, (key, kind) in enumerate((("T", torch.float32), ("k", torch.int32), ("p", torch.float32),
                                         ("m", torch.float32))):
            state[key] = torch.tensor([a[i] for a in ask], dtype=kind, device="cuda") if ask else case[key]
    elif case["op"] == "embed":
        V, d = case["vocab"], case["d"]
        # token v with a probability near 1 / (v + 1), as in text
        tokens = (torch.rand(N, generator=g, device="cuda", dtype=torch.float64) * math.log(V)).exp().int() - 1
        tokens.clamp_(0, V - 1)
        if case["padded"]:
            tokens[torch.arange(N, device="cuda") % 16 == 15] = -1
        state["tokens"] = tokens
        if case["dir"] == "forward":
            state["table"] = torch.empty(V, d, dtype=dt, device="cuda").normal_(0.0, 1 / math.sqrt(d), generator=g)
        else:
            state["grad"] = torch.empty(N, d, dtype=dt, device="cuda").normal_(generator=g)
    else:
        d, pt = case["d"], DTYPES[case["params"]]
        x = torch.empty(N, d, dtype=dt, device="cuda").normal_(generator=g)
        x += 0.5 * torch.randn(d, generator=g, device="cuda")
        state.update(x=x, weight=(1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(pt),
                     bias=(0.1 * torch.randn(d, generator=g, device="cuda")).to(pt))
        if case["dir"] == "backward":
            # what the forward pass left: each row's mean and 1 / sqrt(variance + eps)
            state["grad"] = torch.empty(N, d, dtype=dt, device="cuda").normal_(generator=g)
            stats = torch.empty(N, 2, dtype=torch.float32, device="cuda")
            for at in range(0, N, 4096):
                v, m = torch.var_mean(x[at:at + 4096].double(), dim=1, correction=0)
                stats[at:at + 4096, 0], stats[at:at + 4096, 1] = m.float(), (v + EPS).rsqrt().float()
            state["stats"] = stats
    return state


# ---------------------------------------------------------------- the plain forms

def _column(x, N, kind):
    return x[:, None].to(kind) if torch.is_tensor(x) else torch.full((N, 1), x, dtype=kind, device="cuda")


def _plain_sample(s):
    # in 64 bits: which token a uniform falls on hangs on the running sums
    N = s["case"]["N"]
    T, p, m = (_column(s[k], N, torch.float32).double() for k in "Tpm")
    k = _column(s["k"], N, torch.int64)
    greedy = T == 0
    T = torch.where(greedy, torch.ones_like(T), T)
    z, ids = s["logits"].double().sort(dim=1, descending=True, stable=True)
    V = z.shape[1]
    k = torch.where(greedy, torch.ones_like(k), torch.where((k <= 0) | (k > V), torch.full_like(k, V), k))
    w = ((z - z[:, :1]) / T).exp()
    first = torch.arange(V, device="cuda") < k
    run_sum = torch.where(first, w, torch.zeros_like(w)).cumsum(dim=1)
    kept = first & (w >= m) & ((run_sum - w < p * run_sum[:, -1:]) | (p >= 1))
    kept[:, 0] = True
    run_sum = torch.where(kept, w, torch.zeros_like(w)).cumsum(dim=1)
    mass = run_sum[:, -1:]
    at = (kept & (run_sum <= s["u"].double()[:, None] * mass)).sum(dim=1, keepdim=True)
    at = torch.minimum(at, kept.sum(dim=1, keepdim=True) - 1)
    return {"token": ids.gather(1, at)[:, 0].int(), "prob": (w.gather(1, at) / mass)[:, 0].float()}


def _plain_embed(s):
    case, t = s["case"], s["tokens"].long()
    V, dt = case["vocab"], DTYPES[case["dtype"]]
    held = (t >= 0) & (t < V)
    if case["dir"] == "forward":
        rows = s["table"][t.clamp(0, V - 1)].float() * case["scale"]
        return {"rows": torch.where(held[:, None], rows, torch.zeros_like(rows)).to(dt)}
    grad = torch.zeros(V + 1, case["d"], dtype=torch.float32, device="cuda")
    grad.index_add_(0, torch.where(held, t, torch.full_like(t, V)), s["grad"].float())
    return {"grad": (grad[:V] * case["scale"]).to(dt)}


def _plain_norm(s):
    case = s["case"]
    x, w = s["x"].float(), s["weight"].float()
    if case["dir"] == "forward":
        mean = x.mean(dim=1, keepdim=True)
        x = x - mean
        rstd = 1.0 / ((x * x).mean(dim=1, keepdim=True) + EPS).sqrt()
        out = {"y": (x * rstd * w + s["bias"].float()).to(s["x"].dtype)}
        if case["stats"]:
            out["stats"] = torch.cat([mean, rstd], dim=1)
        return out
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    g = s["grad"].float()
    hat = (x - mean) * rstd
    gw = g * w
    dx = rstd * (gw - gw.mean(dim=1, keepdim=True) - hat * (gw * hat).mean(dim=1, keepdim=True))
    # long sums over the batch
    return {"dx": dx.to(s["x"].dtype), "dw": (g * hat).sum(dim=0, dtype=torch.float64).to(s["weight"].dtype),
            "db": g.sum(dim=0, dtype=torch.float64).to(s["bias"].dtype)}


def run(state):
    case = state["case"]
    if own:
        from speculative_decoding_draft_dh_gb300 import binding as dh
        if case["op"] == "sample":
            token, prob = dh.sample(state["logits"], state["u"], temperature=state["T"], top_k=state["k"],
                                    top_p=state["p"], min_p=state["m"])
            return {"token": token, "prob": prob}
        if case["op"] == "embed":
            if case["dir"] == "forward":
                return {"rows": dh.embed(state["table"], state["tokens"], scale=case["scale"])}
            return {"grad": dh.embed_backward(state["grad"], state["tokens"], case["vocab"], scale=case["scale"])}
        if case["dir"] == "forward":
            y, stats = dh.layer_norm(state["x"], state["weight"], state["bias"], eps=EPS, with_stats=case["stats"])
            return {"y": y, "stats": stats} if case["stats"] else {"y": y}
        dx, dw, db = dh.layer_norm_backward(state["grad"], state["x"], state["stats"], state["weight"])
        return {"dx": dx, "dw": dw, "db": db}
    return {"sample": _plain_sample, "embed": _plain_embed, "norm": _plain_norm}[case["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _distinct(case):
    """About how many different tokens N draws with probability 1 / ((v + 1) ln V) bring."""
    V, n = case["vocab"], case["N"] * (15 / 16 if case["padded"] else 1.0)
    total, v = 0.0, 0
    while v < V:
        step = max(1, v // 16)
        total += min(step, V - v) * -math.expm1(-n / ((v + 0.5 + step / 2) * math.log(V)))
        v += step
    return int(min(total, n))


def work(case):
    size, N = SIZE[case["dtype"]], case["N"]
    if case["op"] == "sample":
        n = N * case["vocab"]
        return {"bytes": n * size + 12 * N, "flops": (1 if case["k"] else 4) * n}
    d = case["d"]
    if case["op"] == "embed":
        held = N - (N // 16 if case["padded"] else 0)
        if case["dir"] == "forward":
            return {"bytes": (_distinct(case) + N) * d * size + 4 * N, "flops": held * d}
        return {"bytes": (held + case["vocab"]) * d * size + 4 * N, "flops": held * d}
    par = SIZE[case["params"]] * d
    if case["dir"] == "forward":
        return {"bytes": 2 * N * d * size + 2 * par + (8 * N if case["stats"] else 0), "flops": 7 * N * d}
    return {"bytes": 3 * N * d * size + 3 * par + 8 * N, "flops": 13 * N * d}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _exact_sample(s):
    case, out = s["case"], []
    for n in range(case["N"]):
        T, k, p, m = (float(s[c][n]) if torch.is_tensor(s[c]) else s[c] for c in "Tkpm")
        if torch.is_tensor(s["p"]) is False:
            T, p, m = (float(torch.tensor(v, dtype=torch.float32)) for v in (T, p, m))
        if T == 0:
            out.append(1.0)
            continue
        row = s["logits"][n].double() / T
        V = row.numel()
        k = int(k) if 0 < k < V else V
        top = row.topk(k).values
        q = (top - top.logsumexp(0)).exp()
        n_keep = k if p >= 1 else min(k, int(torch.searchsorted(q.cumsum(0), p)) + 1)
        if m > 0:
            n_keep = min(n_keep, int((q >= m * q[0]).sum()))
        q = q[:max(n_keep, 1)]
        q = q / q.sum()
        at = int(torch.searchsorted(q.cumsum(0), float(s["u"][n]), right=True))
        out.append(float(q[min(at, q.numel() - 1)]))
    return {"token": None, "prob": torch.tensor(out, dtype=torch.float64, device="cuda")}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "embed":
        t, V = s["tokens"].long(), case["vocab"]
        at = ((t >= 0) & (t < V)).nonzero()[:, 0]
        if case["dir"] == "forward":
            rows = torch.zeros(case["N"], case["d"], dtype=torch.float64, device="cuda")
            rows[at] = s["table"].index_select(0, t[at]).double().mul_(case["scale"])
            return {"rows": rows}
        grad = torch.zeros(V, case["d"], dtype=torch.float64, device="cuda")
        for i in range(0, at.numel(), 4096):
            part = at[i:i + 4096]
            grad.index_add_(0, t[part], s["grad"][part].double())
        return {"grad": grad.mul_(case["scale"])}
    out = {"y": [], "stats": [], "dx": []}
    w, b = s["weight"].double(), s["bias"].double()
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    for i in range(0, case["N"], 4096):
        x = s["x"][i:i + 4096].double()
        if case["dir"] == "forward":
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            sd = (var + EPS).sqrt()
            out["y"].append(torch.addcmul(b, (x - mean) / sd, w))
            out["stats"].append(torch.cat([mean, 1 / sd], dim=1))
            continue
        # the forward pass's statistics are inputs of the gradient
        st = s["stats"][i:i + 4096].double()
        g = s["grad"][i:i + 4096].double()
        hat = (x - st[:, :1]) * st[:, 1:]
        dw += torch.einsum("nd,nd->d", g, hat)
        db += g.sum(dim=0)
        g = g * w
        a, c = g.mean(dim=1, keepdim=True), torch.einsum("nd,nd->n", g, hat)[:, None] / case["d"]
        out["dx"].append((g - a - hat * c) * st[:, 1:])
    if case["dir"] == "backward":
        return {"dx": torch.cat(out["dx"]), "dw": dw, "db": db}
    want = ["y", "stats"] if case["stats"] else ["y"]
    return {k: torch.cat(out[k]) for k in want}
