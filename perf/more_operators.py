"""Cases of the library's operators at the two ends of a layer stack, each with
a plain form in elementary torch operations and its definition in 64 bits.

* norm: the layer norm in front of a group of projections, with the residual
  add before it (forward; backward with the gradients of weight and bias),
* logprob: log probabilities of given tokens from the head's logits, their
  distribution's entropy and its top alternatives,
* distill: the distillation loss against a teacher's top alternatives, mixed
  with the cross entropy of given targets, and its gradient.

`own` selects what `run` computes with: False takes the plain form, True calls
the library.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
EPS = 1e-5

# the largest listed cases, in bytes: no drawn case costs more
MAX_NORM = 32768 * 4096 * 14
MAX_LOGPROB = 4096 * 131072 * 2
MAX_DISTILL = 8192 * 65536 * 4


def listed():
    return [
        # one token of 32 sequences in front of receptance / key / value: latency
        dict(name="norm_fwd_decode", op="norm_fwd", T=32, C=2048, x="bf16", a="bf16", y="bf16", stats=False),
        # a training batch of 16 sequences of 1024 tokens, d = 2048: fp32 residual
        # stream, the branch's fp32 output added, bf16 into the projections
        dict(name="norm_fwd_train", op="norm_fwd", T=16384, C=2048, x="f32", a="f32", y="bf16", stats=True),
        # a small block (8 x 256 tokens, d = 512), all bf16
        dict(name="norm_bwd_block", op="norm_bwd", T=2048, C=512, x="bf16", dy="bf16", dx="bf16", ds=False),
        # packed tokens and a width off the tiles, all fp32
        dict(name="norm_bwd_ragged", op="norm_bwd", T=5003, C=1032, x="f32", dy="f32", dx="f32", ds=True),
        # the widest layer: bf16 stream, dY is the fp32 dX of the projections,
        # the stream's own fp32 gradient added
        dict(name="norm_bwd_wide", op="norm_bwd", T=32768, C=4096, x="bf16", dy="f32", dx="f32", ds=True),
        # evaluation of a byte-level model: 8 x 256 tokens, fp32 logits, top 1
        dict(name="logprob_bytes", op="logprob", T=2048, V=256, z="f32", k=1, scale=1.0, pad=0),
        # 13 sequences decoding together, alternatives of each, an odd vocabulary
        dict(name="logprob_decode", op="logprob", T=13, V=50021, z="f32", k=20, scale=1.25, pad=0),
        # a teacher's pass over 4096 tokens at temperature 2, padded vocabulary
        dict(name="logprob_teacher", op="logprob", T=4096, V=131072, z="bf16", k=64, scale=0.5, pad=253),
        # a byte-level student: 8 x 256 tokens
        dict(name="distill_bytes", op="distill", T=2048, V=256, z="f32", K=16, alpha=0.5, tau=2.0, grad=True),
        # the loss alone of held-out tokens, an odd vocabulary
        dict(name="distill_eval", op="distill", T=1021, V=50021, z="bf16", K=32, alpha=0.1, tau=1.0, grad=False),
        # a training batch: loss and gradient
        dict(name="distill_train", op="distill", T=8192, V=65536, z="bf16", K=32, alpha=0.1, tau=2.0, grad=True),
        # few tokens, widest vocabulary, fp32
        dict(name="distill_wide", op="distill", T=61, V=131072, z="f32", K=64, alpha=0.0, tau=1.0, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mul8(x, lo=8):
    return max(lo, (int(x) + 4) // 8 * 8)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "logprob", "logprob", "distill", "distill"])
    t = lambda: rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        C = _mul8(_log(rng, 64, 16384))
        c = dict(op=op, T=1, C=C, x=t())
        if op == "norm_fwd":
            c.update(a=rng.choice(["none", "bf16", "f32"]), y=t(), stats=rng.random() < 0.5)
        else:
            c.update(dy=t(), dx="f32" if c["x"] == "f32" else t(), ds=rng.random() < 0.5)
        c["T"] = _log(rng, 1, max(1, min(65536, MAX_NORM // (work(c)["bytes"] + 1))))
        return c
    V = _log(rng, 64, 131072)
    if op == "logprob":
        z = t()
        return dict(op=op, T=_log(rng, 1, min(16384, MAX_LOGPROB // (V * ES[z]))), V=V, z=z,
                    k=rng.choice([0, 1, 5, rng.randint(2, 64)]), scale=rng.choice([1.0, 0.5, 1.25]),
                    pad=rng.choice([0, 0, V // 500]))
    z, grad = t(), rng.random() < 0.7
    return dict(op=op, T=_log(rng, 1, min(16384, MAX_DISTILL // (V * ES[z] * 2))), V=V, z=z, K=rng.randint(1, 64),
                alpha=rng.choice([0.0, 0.1, 0.5, 1.0]), tau=rng.choice([1.0, 2.0, 1.5]), grad=grad)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _logits(N, U, T, V, dt, pad, rows_at_once=512):
    """Logits of a head: some tokens are likelier everywhere, a few in each row
    stand out; rows start on 16 bytes (the row stride is a multiple of 8), and
    a padded vocabulary's last columns are masked out."""
    ld = (V + 7) // 8 * 8
    buf = torch.zeros(T, ld, dtype=dt, device="cuda")
    common = N(V)
    for t0 in range(0, T, rows_at_once):
        n = min(rows_at_once, T - t0)
        z = N(n, V) * 1.5 + common
        peak = (U(0.0, 1.0, n, 4) * V).long().clamp(max=V - 1)
        z.scatter_add_(1, peak, U(0.0, 10.0, n, 4))
        buf[t0:t0 + n, :V] = z
    if pad:
        buf[:, V - pad:V] = -math.inf
    return buf[:, :V]


def _data(case, seed):
    """The case's inputs as tensors (dict), from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = lambda *s: torch.randn(*s, generator=g, device="cuda")
    U = lambda lo, hi, *s: torch.rand(*s, generator=g, device="cuda") * (hi - lo) + lo
    op, d = case["op"], {}
    T = case["T"]
    if op.startswith("norm"):
        C = case["C"]
        # a residual stream: channels of different sizes, a few large ones
        size = torch.exp(N(C) * 0.5)
        d["w"], d["b"] = U(0.5, 1.5, C), N(C) * 0.1
        X = N(T, C) * size + N(C) * 0.3
        if op == "norm_fwd":
            d["X"] = X.to(DTYPES[case["x"]])
            if case["a"] != "none":
                d["A"] = (N(T, C) * 0.3).to(DTYPES[case["a"]])
            return d
        S = X.to(DTYPES[case["x"]])
        d["S"] = S
        d["dY"] = (N(T, C) * 0.01).to(DTYPES[case["dy"]])
        if case["ds"]:
            d["dS"] = (N(T, C) * 0.01).to(DTYPES[case["dx"]])
        return d
    V = case["V"]
    d["Z"] = _logits(N, U, T, V, DTYPES[case["z"]], case.get("pad", 0))
    d["tokens"] = (U(0.0, 1.0, T) * (V - case.get("pad", 0))).long().clamp(max=V - 1 - case.get("pad", 0))
    if op == "distill":
        # the teacher's alternatives: different tokens, falling probabilities
        # that do not sum to one (it kept its top K)
        K = case["K"]
        start, step = (U(0.0, 1.0, T, 1) * V).long(), max(1, V // 64 - 1)
        d["ids"] = (start + torch.arange(K, device="cuda") * step) % V
        d["lp"] = torch.log_softmax(N(T, K + 1) * 2.0, 1)[:, :K].contiguous()
        d["dloss"] = U(0.5, 1.5, T) / T
    return d


def prepare(case, seed):
    st = _data(case, seed)
    st["case"] = case
    op = case["op"]
    if op == "norm_bwd":
        # what the forward hands over: mean and 1 / deviation of each row
        S = st["S"].float()
        mean = S.mean(1)
        st["stats"] = torch.stack([mean, torch.rsqrt(((S - mean[:, None]) ** 2).mean(1) + EPS)], 1)
    if not own:
        return st
    import ternary_weight_linear_tern_amd as tl
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")
    f32, T = torch.float32, case["T"]
    if op == "norm_fwd":
        C = case["C"]
        st["Y"] = new((T, C), DTYPES[case["y"]])
        st["S"] = new((T, C), DTYPES[case["x"]]) if case["a"] != "none" else None
        st["stats"] = tl.empty_norm_stats(T) if case["stats"] else None
    elif op == "norm_bwd":
        C = case["C"]
        st["dX"] = new((T, C), DTYPES[case["dx"]])
        st["dw"], st["db"] = new((C,), f32), new((C,), f32)
        st["ws"] = tl.empty_norm_workspace(T, C)
    elif op == "logprob":
        for name in ("logp", "entropy", "lse"):
            st[name] = new((T,), f32)
        k = case["k"]
        st["top_ids"] = new((T, k), torch.int64) if k else None
        st["top_logp"] = new((T, k), f32) if k else None
        st["ws"] = tl.empty_logprob_workspace(T, case["V"], k)
    else:
        st["loss"] = new((T,), f32)
        st["dZ"] = torch.empty_like(torch.as_strided(st["Z"], (T, st["Z"].stride(0)), (st["Z"].stride(0), 1)))[
            :, :case["V"]] if case["grad"] else None
        st["ws"] = tl.empty_distill_workspace(T, case["V"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(st, case):
    import ternary_weight_linear_tern_amd as tl
    op = case["op"]
    if op == "norm_fwd":
        tl.tern_norm_fwd(st["X"], st["Y"], w=st["w"], b=st["b"], A=st.get("A"), S=st["S"], stats=st["stats"], eps=EPS)
        return [x for x in (st["Y"], st["S"], st["stats"]) if x is not None]
    if op == "norm_bwd":
        tl.tern_norm_bwd(st["S"], st["stats"], st["dY"], st["dX"], st["ws"], w=st["w"], dS=st.get("dS"), dw=st["dw"],
                         db=st["db"])
        return [st["dX"], st["dw"], st["db"]]
    if op == "logprob":
        tl.tern_logprob(st["Z"], st["ws"], tokens=st["tokens"], scale=case["scale"], logp=st["logp"],
                        entropy=st["entropy"], lse=st["lse"], top_ids=st["top_ids"], top_logp=st["top_logp"])
        out = [st["logp"], st["entropy"], st["lse"]]
        return out + [st["top_ids"], st["top_logp"]] if case["k"] else out
    tl.tern_distill(st["Z"], st["ws"], targets=st["tokens"], teacher_ids=st["ids"], teacher_logp=st["lp"],
                    alpha=case["alpha"], tau=case["tau"], loss=st["loss"], dloss=st["dloss"] if case["grad"] else None,
                    dZ=st["dZ"])
    return [st["loss"], st["dZ"]] if case["grad"] else [st["loss"]]


def _run_plain(st, case):
    op = case["op"]
    if op == "norm_fwd":
        out, x = [], st["X"]
        S = x.float()
        if "A" in st:
            kept = (S + st["A"].float()).to(x.dtype)     # the stream holds the sum in its own type
            out.append(kept)
            S = kept.float()
        mean = S.mean(1, keepdim=True)
        D = S - mean
        r = torch.rsqrt((D * D).mean(1, keepdim=True) + EPS)
        out.insert(0, (D * r * st["w"] + st["b"]).to(DTYPES[case["y"]]))
        if case["stats"]:
            out.append(torch.cat([mean, r], 1))
        return out
    if op == "norm_bwd":
        mean, r = st["stats"][:, :1], st["stats"][:, 1:]
        xh, dy = (st["S"].float() - mean) * r, st["dY"].float()
        g = dy * st["w"]
        dX = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if "dS" in st:
            dX = dX + st["dS"].float()
        return [dX.to(DTYPES[case["dx"]]), (dy * xh).sum(0), dy.sum(0)]
    rows = torch.arange(case["T"], device="cuda")
    if op == "logprob":
        z = st["Z"].float() * case["scale"]
        m = z.amax(1, keepdim=True)
        z -= m                                           # now at most 0
        e = torch.exp(z)
        s = e.sum(1)
        logs = torch.log(s)
        e *= z.clamp(min=-3e38)                          # a masked token: 0 times a finite number
        out = [z[rows, st["tokens"]] - logs, logs - e.sum(1) / s, m[:, 0] + logs]
        del e
        if case["k"]:
            # unique keys: the value's bits in ascending order, then the lower index first
            bits = (st["Z"].float() + 0.0).view(torch.int32)
            bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)
            last = (1 << 32) - 1
            key = (bits.long() << 32) + (last - torch.arange(case["V"], device="cuda"))
            ids = last - (torch.topk(key, case["k"], dim=1).values & last)
            out += [ids, torch.gather(z, 1, ids) - logs[:, None]]
        return out
    a, tau, T = case["alpha"], case["tau"], case["T"]
    z = st["Z"].float()
    z = z - z.amax(1, keepdim=True)
    y = st["tokens"]
    lp = st["lp"] - st["lp"].amax(1, keepdim=True)
    p = torch.exp(lp)
    ps = p.sum(1, keepdim=True)
    p, logp = p / ps, lp - torch.log(ps)
    e = torch.exp(z / tau)
    s = e.sum(1, keepdim=True)
    loss = tau * tau * (1.0 - a) * (p * (logp - torch.gather(z, 1, st["ids"]) / tau + torch.log(s))).sum(1)
    e1 = torch.exp(z) if a else None
    if a:
        s1 = e1.sum(1, keepdim=True)
        loss = loss + a * (torch.log(s1[:, 0]) - z[rows, y])
    if not case["grad"]:
        return [loss]
    del z
    e *= (1.0 - a) * tau / s
    e.scatter_add_(1, st["ids"], (a - 1.0) * tau * p)
    if a:
        e += e1 * (a / s1)
        e[rows, y] -= a
    return [loss, (e * st["dloss"][:, None]).to(st["Z"].dtype)]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "norm_fwd":
        n = T * case["C"]
        byt = ES[case["x"]] + ES[case["y"]]
        if case["a"] != "none":
            byt += ES[case["a"]] + ES[case["x"]]
        return {"bytes": n * byt + (8 * T if case["stats"] else 0) + 8 * case["C"], "flops": 8 * n}
    if op == "norm_bwd":
        n = T * case["C"]
        byt = ES[case["x"]] + ES[case["dy"]] + ES[case["dx"]] * (2 if case["ds"] else 1)
        return {"bytes": n * byt + 8 * T + 12 * case["C"], "flops": 16 * n}
    n = T * case["V"]
    if op == "logprob":
        return {"bytes": n * ES[case["z"]] + T * (20 + 12 * case["k"]), "flops": 8 * n}
    return {"bytes": n * ES[case["z"]] * (2 if case["grad"] else 1) + T * (16 + 12 * case["K"]),
            "flops": (14 if case["grad"] else 6) * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _by_rows(f, T, per_row):
    """f(rows) over slices of rows that hold about 2^27 numbers each."""
    n = max(1, (1 << 27) // per_row)
    parts = [f(slice(t, min(t + n, T))) for t in range(0, T, n)]
    return [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]))]


def exact(case, seed):
    d = _data(case, seed)
    op, T = case["op"], case["T"]
    f64 = torch.float64
    if op == "norm_fwd":
        def rows(s):
            X, kept = d["X"][s].to(f64), []
            if "A" in d:
                X = (X + d["A"][s].to(f64)).to(d["X"].dtype)
                kept = [X]
                X = X.to(f64)
            var, mean = torch.var_mean(X, dim=1, correction=0, keepdim=True)
            dev = torch.sqrt(var + EPS)
            out = [(X - mean) / dev * d["w"].to(f64) + d["b"].to(f64)] + kept
            return out + [torch.cat([mean, 1.0 / dev], 1)] if case["stats"] else out
        return _by_rows(rows, T, case["C"])
    if op == "norm_bwd":
        dw, db = (torch.zeros(case["C"], dtype=f64, device="cuda") for _ in range(2))

        def rows(s):
            S, dY = d["S"][s].to(f64), d["dY"][s].to(f64)
            var, mean = torch.var_mean(S, dim=1, correction=0, keepdim=True)
            dev = torch.sqrt(var + EPS)
            hat = (S - mean) / dev
            dw.add_((dY * hat).sum(0))
            db.add_(dY.sum(0))
            # through the mean and the deviation
            u = dY * d["w"].to(f64)
            dX = (u - (u.sum(1, keepdim=True) + hat * (u * hat).sum(1, keepdim=True)) / case["C"]) / dev
            return [dX + d["dS"][s].to(f64) if "dS" in d else dX]
        return _by_rows(rows, T, case["C"]) + [dw, db]
    if op == "logprob":
        def rows(s):
            Z = d["Z"][s]
            L = torch.log_softmax(Z.to(f64) * case["scale"], 1)
            lse = torch.logsumexp(Z.to(f64) * case["scale"], 1)
            H = -torch.where(L > -math.inf, L.exp() * L, 0.0).sum(1)
            out = [L.gather(1, d["tokens"][s, None])[:, 0], H, lse]
            if case["k"]:
                ids = torch.sort(Z.float(), dim=1, descending=True, stable=True).indices[:, :case["k"]]
                out += [ids, L.gather(1, ids)]
            return out
        return _by_rows(rows, T, case["V"])
    a, tau = case["alpha"], case["tau"]

    def rows(s):
        Z = d["Z"][s].to(f64)
        hard, soft = torch.log_softmax(Z, 1), torch.log_softmax(Z / tau, 1)
        y, ids = d["tokens"][s, None], d["ids"][s]
        lp = torch.log_softmax(d["lp"][s].to(f64), 1)
        kl = (lp.exp() * (lp - soft.gather(1, ids))).sum(1)
        loss = (1.0 - a) * tau ** 2 * kl - a * hard.gather(1, y)[:, 0]
        if not case["grad"]:
            return [loss]
        G = a * hard.exp() + (1.0 - a) * tau * soft.exp()
        G.scatter_add_(1, y, torch.full_like(y, -a, dtype=f64))
        G.scatter_add_(1, ids, -(1.0 - a) * tau * lp.exp())
        return [loss, G * d["dloss"][s, None].to(f64)]
    return _by_rows(rows, T, case["V"])
