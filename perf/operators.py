"""Measured calls of the vocabulary-side operators that score and distil tokens.

Four kinds of case, one pass each:

  logprobs       log-probability of one given token per row, entropy and the top alternatives
                 of [T, v] logits (vp_logprobs_fwd)
  logprobs_grad  the gradient of those log-probabilities and entropies (vp_logprobs_bwd)
  distill        loss against a teacher's top entries and, if asked for, its gradient in the
                 same call (vp_distill)
  linear         log-probabilities and entropy straight from hidden states and the output
                 table, without the logits matrix (tp_linear_logprobs_fwd), and with "grad"
                 the gradient at the logits too (tp_linear_logprobs_dlogits)

Each case runs in a plain form (elementary torch operations in fp32) or, when ``own`` is set,
through the library's entry points, on the same inputs.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_INF = float("inf")
_MAX_ELEMENTS = 8192 * 50304          # logits of the largest listed case
_MAX_PRODUCTS = 4096 * 4096 * 50304   # T·h·v of the largest listed output layer


def _logprobs(name, T, v, dtype, K, scale=1.0, masked=0.0, N=1):
    return {"name": name, "op": "logprobs", "T": T, "v": v, "dtype": dtype, "K": K,
            "scale": scale, "masked": masked, "N": N}


def _logprobs_grad(name, T, v, dtype, grad_dtype, scale=1.0, N=1):
    return {"name": name, "op": "logprobs_grad", "T": T, "v": v, "dtype": dtype,
            "grad_dtype": grad_dtype, "scale": scale, "N": N}


def _distill(name, T, v, dtype, grad_dtype, K, renormalize=True, grad=True, scale=1.0,
             ragged=False, N=1):
    return {"name": name, "op": "distill", "T": T, "v": v, "dtype": dtype,
            "grad_dtype": grad_dtype, "K": K, "renormalize": renormalize, "grad": grad,
            "scale": scale, "ragged": ragged, "N": N}


def _linear(name, T, h, v, grad, scale=1.0, N=1):
    return {"name": name, "op": "linear", "T": T, "h": h, "v": v, "grad": grad, "scale": scale,
            "N": N}


def listed():
    return [
        # one decoding step of one sequence, with the alternatives that an API returns
        _logprobs("logprobs, one token", 1, 50304, "f32", 20, N=8),
        # a decoding batch under a grammar that bans nine tokens in ten; odd vocabulary
        _logprobs("logprobs, decoding batch", 64, 50257, "bf16", 8, scale=1.25, masked=0.9),
        # scoring a batch of prompts: log-probabilities and entropy only
        _logprobs("logprobs, scoring", 4096, 50304, "f32", 0, N=8),
        # a teacher's pass that records its top entries for later distillation
        _logprobs("logprobs, top entries", 8192, 50304, "bf16", 64, N=8),
        # policy-gradient step: gradient of log-probabilities and an entropy bonus
        _logprobs_grad("logprobs gradient", 8192, 50304, "f32", "bf16", N=8),
        # the same on a small vocabulary of odd width, bf16 throughout, sampled at 0.7
        _logprobs_grad("logprobs gradient, odd", 1031, 32003, "bf16", "bf16", scale=1 / 0.7),
        # validation loss of a distillation run
        _distill("distill, loss only", 512, 50304, "f32", "bf16", 64, grad=False, N=8),
        # a distillation step: loss and gradient of a whole batch
        _distill("distill, step", 8192, 50304, "f32", "bf16", 64, N=8),
        # ragged teacher entries with their tail mass dropped, padded rows, odd vocabulary
        _distill("distill, ragged", 777, 50257, "bf16", "bf16", 33, renormalize=False,
                 scale=0.5, ragged=True),
        # a large multilingual vocabulary, gradients kept in fp32
        _distill("distill, large vocabulary", 512, 200001, "f32", "f32", 128),
        # log-probabilities of a short batch from the output layer of a width-1600 model
        _linear("linear logprobs", 500, 1600, 50304, False, scale=1.25, N=4),
        # the forward and gradient of a policy step that never stores its logits
        _linear("linear logprobs, step", 4096, 4096, 50304, True, N=8),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "distill", "distill", "linear"])
    scale = rng.choice([1.0, 1.0, 0.5, 1.25, 1 / 0.7])
    dtype = rng.choice(["f32", "bf16"])
    grad_dtype = rng.choice(["f32", "bf16"])
    if op == "linear":
        h = 8 * _spread(rng, 8, 512)
        v = 8 * _spread(rng, 128, 12576)
        T = _spread(rng, 1, max(1, min(8192, _MAX_PRODUCTS // (h * v))))
        c = _linear("", T, h, v, rng.random() < 0.5, scale, rng.choice([1, 2, 4, 8]))
    else:
        v = _spread(rng, 500, 262144)
        T = _spread(rng, 1, max(1, min(8192, _MAX_ELEMENTS // (2 * v))))
        N = rng.choice([n for n in (1, 2, 3, 4, 8) if v % n == 0])
        if op == "logprobs":
            K = rng.choice([0, 1, rng.randint(2, 32), rng.randint(33, 128)])
            c = _logprobs("", T, v, dtype, K, scale, rng.choice([0.0, 0.0, 0.5, 0.99]), N)
        elif op == "logprobs_grad":
            c = _logprobs_grad("", T, v, dtype, grad_dtype, scale, N)
        else:
            K = rng.choice([1, rng.randint(2, 64), rng.randint(65, 256)])
            c = _distill("", T, v, dtype, grad_dtype, K, rng.random() < 0.6, rng.random() < 0.7,
                         scale, rng.random() < 0.5, N)
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs
def _logits(g, T, v, dtype):
    """Rows as a trained model gives them: a broad body and sixteen tokens that stand out."""
    x = torch.randn(T, v, generator=g, device="cuda").mul_(2.0)
    at = torch.randint(0, v, (T, 16), generator=g, device="cuda")
    x.scatter_(1, at, torch.rand(T, 16, generator=g, device="cuda") * 9.0 + 5.0)
    return x.to(dtype), at


def _given(g, at, v):
    """Mostly tokens that the model finds likely, some that it does not."""
    T = at.shape[0]
    any_token = torch.randint(0, v, (T,), generator=g, device="cuda")
    return torch.where(torch.rand(T, generator=g, device="cuda") < 0.75, at[:, 0], any_token)


def _upstream(g, T):
    """Gradients at the log-probabilities and entropies of a batch, one row in eight padded."""
    keep = torch.rand(T, generator=g, device="cuda") >= 0.125
    if T < 8:
        keep = torch.ones_like(keep)
    dlogprob = torch.randn(T, generator=g, device="cuda") / T * keep
    dentropy = torch.full((T,), -0.01 / T, device="cuda") * keep
    return dlogprob, dentropy


def _chunks(T, v):
    step = max(1, (1 << 27) // v)
    return [slice(i, min(T, i + step)) for i in range(0, T, step)]


def _statistics64(x, scale):
    """log-sum-exp and entropy of scale·x in 64 bits."""
    lse, ent = [], []
    for s in _chunks(*x.shape):
        lp = torch.log_softmax(x[s].double() * scale, dim=1)
        lse.append(torch.logsumexp(x[s].double() * scale, dim=1))
        ent.append(-torch.xlogy(lp.exp(), lp.exp()).sum(1))
    return torch.cat(lse), torch.cat(ent)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    T, v = c["T"], c["v"]
    if c["op"] == "linear":
        H = torch.randn(T, c["h"], generator=g, device="cuda").bfloat16()
        E = (torch.randn(v, c["h"], generator=g, device="cuda") * (1.6 / math.sqrt(c["h"]))).bfloat16()
        y = torch.randint(0, v, (T,), generator=g, device="cuda")
        c.update(H=H, E=E, targets=y)
        c["dlogprob"], c["dentropy"] = _upstream(g, T)
        return c
    x, at = _logits(g, T, v, _TYPES[c["dtype"]])
    if c["op"] == "logprobs":
        y = _given(g, at, v)
        if c["masked"]:
            ban = torch.rand(T, v, generator=g, device="cuda") < c["masked"]
            ban.scatter_(1, y[:, None], False)      # the given token was allowed
            x.masked_fill_(ban, -_INF)
        c.update(logits=x, targets=y)
    elif c["op"] == "logprobs_grad":
        lse, ent = _statistics64(x, c["scale"])
        c.update(logits=x, targets=_given(g, at, v), lse=lse.float(), entropy=ent.float())
        c["dlogprob"], c["dentropy"] = _upstream(g, T)
    else:
        K = c["K"]
        # distinct ids: the student's likely tokens are partly the teacher's too
        first = torch.randint(0, v, (T, 1), generator=g, device="cuda")
        stride = max(1, v // K - 1)
        ids = (first + stride * torch.arange(K, device="cuda")) % v
        ids[:, 0] = at[:, 0]
        t = torch.randn(T, K, generator=g, device="cuda").mul_(2.0).sort(1, descending=True).values
        if not c["renormalize"]:                    # log-probabilities, some mass outside
            kept = 0.8 + 0.2 * torch.rand(T, 1, generator=g, device="cuda")
            t = torch.log_softmax(t, 1) + kept.log()
        weight = torch.ones(T, device="cuda")
        if c["ragged"]:
            n = torch.randint(0, K + 1, (T, 1), generator=g, device="cuda")
            ids = torch.where(torch.arange(K, device="cuda") < n, ids, torch.full_like(ids, -1))
            weight = (torch.rand(T, generator=g, device="cuda") >= 0.125).float()
        c.update(logits=x, ids=ids.int(), teacher=t.contiguous(), weight=weight)
    return c


# --------------------------------------------------------------- plain forms
def _plain_statistics(x, scale):
    z = x.float() * scale
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    S = e.sum(1)
    U = torch.where(e > 0, e * (z - m), 0.0).sum(1)
    log_S = torch.log(S)
    return z, m[:, 0] + log_S, log_S - U / S


def _plain_top(x, z, lse, K):
    """Top K by value, equal values in index order: keys that order both."""
    word = (x.float() + 0.0).view(torch.int32)
    word = torch.where(word >= 0, word, word ^ 0x7fffffff).long()
    last = 0xffffffff
    key = (word << 32) | (last - torch.arange(x.shape[1], device=x.device))
    idx = last - (torch.topk(key, K, dim=1, sorted=True).values & last)
    return idx.int(), z.gather(1, idx) - lse[:, None]


def _plain_logprobs(x, y, scale, K):
    z, lse, ent = _plain_statistics(x, scale)
    out = {"logprob": z.gather(1, y[:, None])[:, 0] - lse, "entropy": ent, "lse": lse}
    if K:
        out["top_idx"], out["top_logprob"] = _plain_top(x, z, lse, K)
    return out


def _plain_logprobs_grad(z, y, lse, ent, dlogprob, dentropy, scale):
    lp = z - lse[:, None]
    p = torch.exp(lp)
    d = -p * (dlogprob[:, None] + dentropy[:, None] * torch.where(p > 0, lp + ent[:, None], 0.0))
    d[torch.arange(z.shape[0], device=z.device), y] += dlogprob
    return d * scale


def _plain_distill(s):
    z, lse, _ = _plain_statistics(s["logits"], s["scale"])
    live = s["ids"] >= 0
    at = s["ids"].long().clamp(min=0)
    t = torch.where(live, s["teacher"], -_INF)
    if s["renormalize"]:
        top = t.amax(1, keepdim=True)
        e = torch.where(live, torch.exp(t - torch.where(top > -_INF, top, 0.0)), 0.0)
        total = e.sum(1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
        log_p = t - top - torch.log(total)
    else:
        p, log_p = torch.exp(t), t
    term = p * (log_p - (z.gather(1, at) - lse[:, None]))
    loss = s["weight"] * torch.where(p > 0, term, 0.0).sum(1)
    out = {"loss": loss, "loss_sum": loss.sum().reshape(1), "lse": lse}
    if s["grad"]:
        d = torch.exp(z - lse[:, None]) * p.sum(1, keepdim=True)
        d.scatter_add_(1, at, -p)
        d *= (s["weight"] * (s["scale"] / s["T"]))[:, None]
        out["dlogits"] = d.to(_TYPES[s["grad_dtype"]])
    return out


def _plain(s):
    if s["op"] == "logprobs":
        return _plain_logprobs(s["logits"], s["targets"], s["scale"], s["K"])
    if s["op"] == "logprobs_grad":
        z = s["logits"].float() * s["scale"]
        d = _plain_logprobs_grad(z, s["targets"], s["lse"], s["entropy"], s["dlogprob"],
                                 s["dentropy"], s["scale"])
        return {"dlogits": d.to(_TYPES[s["grad_dtype"]])}
    if s["op"] == "distill":
        return _plain_distill(s)
    x = s["H"].float() @ s["E"].float().T
    out = _plain_logprobs(x, s["targets"], s["scale"], 0)
    if s["grad"]:
        d = _plain_logprobs_grad(x * s["scale"], s["targets"], out["lse"], out["entropy"],
                                 s["dlogprob"], s["dentropy"], s["scale"])
        out["dlogits"] = d.bfloat16()
    return out


# ------------------------------------------------------------ the operators
def _own(s):
    import linear_layers_b200 as tpl

    if s["op"] == "logprobs":
        r = tpl.vp_logprobs_fwd(s["logits"], s["targets"], s["N"], scale=s["scale"], top_k=s["K"])
        return {k: t for k, t in r.items() if t is not None}
    if s["op"] == "logprobs_grad":
        d = tpl.vp_logprobs_bwd(s["logits"], s["targets"], s["lse"], s["entropy"], s["dlogprob"],
                                s["dentropy"], s["N"], scale=s["scale"],
                                grad_dtype=_TYPES[s["grad_dtype"]])
        return {"dlogits": d}
    if s["op"] == "distill":
        r = tpl.vp_distill(s["logits"], s["ids"], s["teacher"], s["N"],
                           renormalize=s["renormalize"], weight=s["weight"], scale=s["scale"],
                           grad_scale=1.0 / s["T"], with_grad=s["grad"],
                           grad_dtype=_TYPES[s["grad_dtype"]])
        return {k: t for k, t in r.items() if t is not None}
    r = tpl.tp_linear_logprobs_fwd(s["H"], s["E"], s["targets"], s["N"], scale=s["scale"])
    out = {k: r[k] for k in ("logprob", "entropy", "lse")}
    if s["grad"]:
        out["dlogits"] = tpl.tp_linear_logprobs_dlogits(
            s["H"], s["E"], s["targets"], r["lse"], r["entropy"], s["dlogprob"], s["dentropy"],
            s["N"], scale=s["scale"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- work and truth
def work(case):
    T, v = case["T"], case["v"]
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "linear":
        products = 2.0 * T * case["h"] * v
        b = 2.0 * case["h"] * (T + v) + 8 * T + 12 * T
        if case["grad"]:
            b += 8 * T + 2.0 * T * v
        return {"bytes": b, "flops": products * (2 if case["grad"] else 1)}
    b = float(T) * v * size[case["dtype"]]
    if case["op"] == "logprobs":
        return {"bytes": b + T * (8 + 12 + 8 * case["K"]), "flops": 6.0 * T * v}
    if case["op"] == "logprobs_grad":
        return {"bytes": b + float(T) * v * size[case["grad_dtype"]] + T * 24, "flops": 8.0 * T * v}
    b += T * (8 * case["K"] + 12) + 4
    if case["grad"]:
        b += float(T) * v * size[case["grad_dtype"]]
    return {"bytes": b, "flops": (8.0 if case["grad"] else 4.0) * T * v}


def _exact_grad(lp, y, ent, dlogprob, dentropy, scale):
    """Σ over both outputs of upstream · ∂output/∂logit, by the softmax Jacobian."""
    p = lp.exp()
    d = torch.zeros_like(p).scatter_(1, y[:, None], dlogprob.double()[:, None])
    d -= dlogprob.double()[:, None] * p
    d -= dentropy.double()[:, None] * (torch.xlogy(p, p) + p * ent[:, None])
    return d * scale


def _exact_rows(s, x, r):
    """The outputs of rows r, whose logits are x (64 bits)."""
    scale = s["scale"]
    lse = torch.logsumexp(x * scale, dim=1)
    lp = x * scale - lse[:, None]
    ent = -torch.xlogy(lp.exp(), lp.exp()).sum(1)
    if s["op"] == "logprobs_grad":
        lse, ent = s["lse"][r].double(), s["entropy"][r].double()
        return {"dlogits": _exact_grad(x * scale - lse[:, None], s["targets"][r], ent,
                                       s["dlogprob"][r], s["dentropy"][r], scale)}
    if s["op"] == "distill":
        ids, t, w = s["ids"][r].long(), s["teacher"][r].double(), s["weight"][r].double()
        t = t.masked_fill(ids < 0, -_INF)
        if s["renormalize"]:
            t = torch.log_softmax(t, dim=1).masked_fill(ids < 0, -_INF)
        p = t.exp()
        q = lp.gather(1, ids.clamp(min=0))
        loss = w * (torch.xlogy(p, p) - torch.where(p > 0, p * q, 0.0)).sum(1)
        out = {"loss": loss, "lse": lse}
        if s["grad"]:
            teacher = torch.zeros_like(lp).scatter_add_(1, ids.clamp(min=0), p)
            out["dlogits"] = (lp.exp() * p.sum(1, keepdim=True) - teacher) * (w * scale / s["T"])[:, None]
        return out
    out = {"logprob": lp.gather(1, s["targets"][r][:, None])[:, 0], "entropy": ent, "lse": lse}
    if s["op"] == "linear" and s["grad"]:
        out["dlogits"] = _exact_grad(lp, s["targets"][r], ent, s["dlogprob"][r], s["dentropy"][r],
                                     scale)
    if s.get("K"):
        out["top_logprob"] = lp.sort(dim=1, descending=True).values[:, :s["K"]].clone()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    E = s["E"].double() if s["op"] == "linear" else None
    rows = []
    for r in _chunks(case["T"], case["v"]):
        x = s["H"][r].double() @ E.T if E is not None else s["logits"][r].double()
        rows.append(_exact_rows(s, x, r))
    out = {k: torch.cat([a[k] for a in rows]) for k in rows[0]}
    if s["op"] == "distill":
        out["loss_sum"] = out["loss"].sum().reshape(1)
    if s.get("K") and s["op"] == "logprobs":
        out["top_idx"] = None
    return out
