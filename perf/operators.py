"""Cases of the library's sequence, serving and update operators, each with a
plain form in elementary torch operations and its definition in 64 bits.

* recur: the gated linear recurrence between the receptance / key / value
  projections and the output projection (forward, backward, one token),
* q4: products of a few rows with 4-bit weights and group scales,
* ortho: an update matrix orthogonalised by Newton-Schulz products.

`own` selects what `run` computes with: False takes the plain form, True calls
the library.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
NS_EPS = 1e-7

# the largest listed cases: no drawn case costs more
MAX_RECUR = 32768 * 4096       # tokens x channels
MAX_STEP = 4096 * 4096         # sequences x channels of a single-token step
MAX_Q4 = 16384 * 4096          # weights
MAX_ORTHO = 4096 * 4096 * 16384


def listed():
    return [
        # one generated token of 32 sequences
        dict(name="recur_step_32", op="recur_step", B=32, C=2048, act="bf16"),
        # a small training block: batch 8 x context 256, d = 512; the three
        # inputs are column slices of one grouped projection's output
        dict(name="recur_fwd_block", op="recur_fwd", T=2048, C=512, seqs=8, ragged=False, act="bf16", grouped=True),
        # a training batch of 16 sequences of 1024 tokens, d = 2048
        dict(name="recur_fwd_train", op="recur_fwd", T=16384, C=2048, seqs=16, ragged=False, act="bf16",
             grouped=True),
        # packed sequences of uneven lengths (some empty) in fp32, a width off the tiles
        dict(name="recur_bwd_ragged", op="recur_bwd", T=5003, C=1032, seqs=37, ragged=True, act="f32", dy="f32",
             grouped=False),
        # one long document, the widest layer; dY is the fp32 dX of the output projection
        dict(name="recur_bwd_long", op="recur_bwd", T=32768, C=4096, seqs=1, ragged=False, act="bf16", dy="f32",
             grouped=True),
        # one token through a small projection: latency
        dict(name="q4_one_small", op="q4", T=1, n_in=512, n_out=512, n=1, group=32, act="bf16", y="bf16",
             scale="bf16"),
        # one token through receptance, key and value at d = 2048: one call
        dict(name="q4_one_rkv", op="q4", T=1, n_in=2048, n_out=2048, n=3, group=64, act="bf16", y="bf16",
             scale="f32"),
        # one token through the widest ffn matrix: bandwidth
        dict(name="q4_one_ffn", op="q4", T=1, n_in=4096, n_out=16384, n=1, group=128, act="bf16", y="f32",
             scale="f32"),
        # 13 sequences decoding together, fp32 activations
        dict(name="q4_batch_ffn", op="q4", T=13, n_in=16384, n_out=4096, n=1, group=64, act="f32", y="f32",
             scale="bf16"),
        # the six gradients of a small layer in one call
        dict(name="ortho_layer_512", op="ortho", shape="layer", rows=512, cols=2048, grad="f32", steps=5),
        # one matrix off the tiles, bf16 momentum
        dict(name="ortho_odd", op="ortho", shape="single", rows=2600, cols=1000, grad="bf16", steps=5),
        # the widest layer's ffn matrix
        dict(name="ortho_ffn_4096", op="ortho", shape="single", rows=4096, cols=16384, grad="f32", steps=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mul8(x, lo=8):
    return max(lo, (int(x) + 4) // 8 * 8)


def draw(rng):
    op = rng.choice(["recur_fwd", "recur_bwd", "recur_step", "q4", "q4", "ortho"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if op in ("recur_fwd", "recur_bwd"):
        C = _mul8(_log(rng, 64, 4096))
        # an fp32 pass moves twice the bytes
        T = _log(rng, 1, min(32768, MAX_RECUR // (C * (2 if act == "f32" else 1))))
        c = dict(op=op, T=T, C=C, seqs=min(T, _log(rng, 1, 64)), ragged=rng.random() < 0.6, act=act,
                 grouped=rng.random() < 0.5)
        if not c["ragged"]:
            while T % c["seqs"]:
                c["seqs"] -= 1
        if op == "recur_bwd":
            c["dy"] = "f32" if act == "f32" else rng.choice(["bf16", "f32"])
        return c
    if op == "recur_step":
        C = _mul8(_log(rng, 64, 4096))
        return dict(op=op, B=_log(rng, 1, min(4096, MAX_STEP // C)), C=C, act=act)
    if op == "q4":
        n_in, n_out = _mul8(_log(rng, 64, 16384)), _mul8(_log(rng, 64, 16384))
        while n_in * n_out > MAX_Q4:
            n_in, n_out = _mul8(n_in * 0.7), _mul8(n_out * 0.7)
        n = rng.choice([1, 1, 2, 3])
        while n * n_in * n_out > MAX_Q4:
            n -= 1
        return dict(op=op, T=_log(rng, 1, 13), n_in=n_in, n_out=n_out, n=n, group=rng.choice([32, 64, 128]),
                    act=act, y="f32" if act == "f32" else rng.choice(["bf16", "f32"]),
                    scale=rng.choice(["bf16", "f32"]))
    shape = rng.choice(["single", "single", "layer"])
    grad = rng.choice(["bf16", "f32"])
    if shape == "layer":
        d = _mul8(_log(rng, 64, 1024))
        return dict(op=op, shape=shape, rows=d, cols=d * rng.choice([2, 4]), grad=grad, steps=5)
    rows, cols = _mul8(_log(rng, 64, 4096)), _mul8(_log(rng, 64, 4096))
    return dict(op=op, shape=shape, rows=rows, cols=cols, grad=grad, steps=5)


def _ortho_shapes(case):
    d, f = case["rows"], case["cols"]
    return [(d, d)] * 4 + [(d, f), (f, d)] if case["shape"] == "layer" else [(d, f)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case, seed):
    """Host lengths of the case's sequences (ragged: uneven, some empty)."""
    T, S = case["T"], case["seqs"]
    if not case["ragged"]:
        return [T // S] * S
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    w = torch.rand(S, generator=g, dtype=torch.float64) ** 2 + 1e-3
    if S > 3:
        w[torch.randperm(S, generator=g)[: max(1, S // 8)]] = 0.0
    cuts = [int(x) for x in torch.round(torch.cumsum(w, 0) / w.sum() * T)]
    cuts[-1] = T
    return [b - a for a, b in zip([0] + cuts[:-1], cuts)]


def _data(case, seed, device="cuda"):
    """The case's inputs as tensors (dict), from the seed alone."""
    g = torch.Generator(device=device).manual_seed(seed)
    N = lambda *s: torch.randn(*s, generator=g, device=device)
    U = lambda lo, hi, *s: torch.rand(*s, generator=g, device=device) * (hi - lo) + lo
    op = case["op"]
    d = {}
    if op.startswith("recur"):
        rows, C, dt = case.get("T", case.get("B")), case["C"], DTYPES[case["act"]]
        # per-channel gate bias: memories of a few tokens to a few hundred
        bias = U(-6.0, 1.0, C)
        if case.get("grouped"):
            buf = torch.empty(rows, 3 * C, dtype=dt, device=device)
            d["R"], d["K"], d["V"] = buf[:, :C], buf[:, C:2 * C], buf[:, 2 * C:]
        else:
            d["R"], d["K"], d["V"] = (torch.empty(rows, C, dtype=dt, device=device) for _ in range(3))
        d["R"].copy_(N(rows, C))
        d["K"].copy_(N(rows, C) + bias)
        d["V"].copy_(N(rows, C))
        if op == "recur_step":
            d["h"] = N(rows, C) * 0.5
            return d
        lens = _lengths(case, seed)
        off = [0]
        for n in lens:
            off.append(off[-1] + n)
        d["longest"] = max(lens)
        d["offsets"] = torch.tensor(off, dtype=torch.int64).to(device)
        d["h0"] = N(len(lens), C) * 0.5
        if op == "recur_bwd":
            d["dY"] = (N(rows, C) * 0.01).to(DTYPES[case["dy"]])
            d["dhT"] = N(len(lens), C) * 0.01
    elif op == "q4":
        n_in, n_out = case["n_in"], case["n_out"]
        d["X"] = N(case["T"], n_in).to(DTYPES[case["act"]])
        ng = -(-n_in // case["group"])
        d["q"] = [torch.randint(-7, 8, (n_in, n_out), generator=g, device=device, dtype=torch.int8)
                  for _ in range(case["n"])]
        d["gscale"] = [U(0.01, 0.1, ng, n_out).to(DTYPES[case["scale"]]) for _ in range(case["n"])]
    else:
        d["G"] = []
        for rows, cols in _ortho_shapes(case):
            # a weight gradient X^T . dY * scale over a batch of tokens
            T = 2 * max(rows, cols)
            G = torch.zeros(rows, cols, device=device)
            for t0 in range(0, T, 8192):
                n = min(8192, T - t0)
                G += N(n, rows).bfloat16().t().contiguous() @ (N(n, cols) * 0.01).bfloat16()
            d["G"].append((G * U(0.01, 0.1, cols)).to(DTYPES[case["grad"]]))
    return d


def prepare(case, seed):
    st = _data(case, seed)
    st["case"] = case
    if not own:
        return st
    import ternary_weight_linear_tern_amd as tl
    op = case["op"]
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")
    if op.startswith("recur"):
        shape, dt = tuple(st["K"].shape), DTYPES[case["act"]]
    if op == "recur_step":
        st["Y"], st["h_out"] = new(shape, dt), torch.empty_like(st["h"])
    elif op == "recur_fwd":
        st["Y"], st["hT"] = new(shape, dt), torch.empty_like(st["h0"])
        st["ws"] = tl.empty_recur_workspace(*shape)
    elif op == "recur_bwd":
        st["ws"] = tl.empty_recur_workspace(*shape)
        st["states"] = tl.empty_recur_states(*shape)
        tl.tern_recur_fwd(st["K"], st["V"], st["R"], new(shape, dt), st["ws"], h0=st["h0"], offsets=st["offsets"],
                          states=st["states"])
        buf = new((shape[0], 3 * shape[1]), dt)
        C = shape[1]
        st["dR"], st["dK"], st["dV"] = buf[:, :C], buf[:, C:2 * C], buf[:, 2 * C:]
        st["dh0"] = torch.empty_like(st["h0"])
    elif op == "q4":
        st["projs"] = []
        for q, s in zip(st["q"], st["gscale"]):
            pk = tl.empty_q4_packed(case["n_in"], case["n_out"])
            tl.tern_q4_pack(q, pk)
            st["projs"].append(dict(n_in=case["n_in"], n_out=case["n_out"], group=case["group"], packed=pk, gscale=s,
                                    X=st["X"], Y=new((case["T"], case["n_out"]), DTYPES[case["y"]])))
    else:
        shapes = _ortho_shapes(case)
        st["mats"] = [dict(G=G, O=new(tuple(G.shape), torch.bfloat16)) for G in st["G"]]
        st["ws"] = tl.empty_ortho_workspace(shapes)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(state, case)


def _run_own(st, case):
    import ternary_weight_linear_tern_amd as tl
    op = case["op"]
    if op == "recur_step":
        tl.tern_recur_step(st["K"], st["V"], st["R"], st["h"], st["Y"], st["h_out"])
        return st["Y"], st["h_out"]
    if op == "recur_fwd":
        tl.tern_recur_fwd(st["K"], st["V"], st["R"], st["Y"], st["ws"], h0=st["h0"], offsets=st["offsets"],
                          hT=st["hT"])
        return st["Y"], st["hT"]
    if op == "recur_bwd":
        tl.tern_recur_bwd(st["K"], st["V"], st["R"], st["dY"], st["states"], st["dK"], st["dV"], st["dR"], st["ws"],
                          h0=st["h0"], offsets=st["offsets"], dhT=st["dhT"], dh0=st["dh0"])
        return st["dK"], st["dV"], st["dR"], st["dh0"]
    if op == "q4":
        tl.tern_layer_q4_matvec(st["projs"])
        return [p["Y"] for p in st["projs"]]
    tl.tern_layer_orthogonalize(st["mats"], st["ws"], steps=case["steps"])
    return [m["O"] for m in st["mats"]]


def _scan(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] along dim 0 by doubling (a is 0 where a
    sequence starts; no sequence is longer than `longest`)."""
    d = 1
    while d < longest:
        b2, a2 = b.clone(), a.clone()
        b2[d:] += a[d:] * b[:-d]
        a2[d:] *= a[:-d]
        a, b, d = a2, b2, 2 * d
    return b


def _sequences(st):
    """First and last token of the non-empty sequences, and their indices."""
    off = st["offsets"]
    live = torch.nonzero(off[1:] > off[:-1])[:, 0]
    return off[:-1][live], off[1:][live] - 1, live


def _run_plain(st, case):
    op = case["op"]
    if op == "recur_step":
        w = torch.sigmoid(st["K"].float())
        h = st["h"] + w * (st["V"].float() - st["h"])
        return (torch.sigmoid(st["R"].float()) * h).to(st["R"].dtype), h
    if op in ("recur_fwd", "recur_bwd"):
        dt = st["K"].dtype
        first, last, live = _sequences(st)
        w, v, s = torch.sigmoid(st["K"].float()), st["V"].float(), torch.sigmoid(st["R"].float())
        keep = torch.sigmoid(-st["K"].float())
        a, b = keep.clone(), w * v
        b[first] += a[first] * st["h0"][live]
        a[first] = 0.0
        h = _scan(a, b, st["longest"])
        if op == "recur_fwd":
            hT = st["h0"].clone()
            hT[live] = h[last]
            return (s * h).to(dt), hT
        del a, b
        prev = torch.zeros_like(h)
        prev[1:] = h[:-1]
        prev[first] = st["h0"][live]
        dy = st["dY"].float()
        dr = dy * h * s * (1.0 - s)
        u = dy * s
        del dy, s, h
        # g[t] = u[t] + keep[t+1] g[t+1], the last token of a sequence taking dhT
        u[last] += st["dhT"][live]
        c = torch.zeros_like(keep)
        c[:-1] = keep[1:]
        c[last] = 0.0
        grad = _scan(c.flip(0), u.flip(0), st["longest"]).flip(0)
        del c, u
        dh0 = st["dhT"].clone()
        dh0[live] = keep[first] * grad[first]
        return (grad * (v - prev) * w * keep).to(dt), (grad * w).to(dt), dr.to(dt), dh0
    if op == "q4":
        X, g = st["X"].float(), case["group"]
        out = []
        for q, s in zip(st["q"], st["gscale"]):
            W = q.float() * s.float().repeat_interleave(g, 0)[: q.shape[0]]
            out.append((X @ W).to(DTYPES[case["y"]]))
        return out
    out = []
    for G in st["G"]:
        X = G.float()
        tall = X.shape[0] > X.shape[1]
        if tall:
            X = X.t().contiguous()
        X = X / (torch.sqrt((X * X).sum()) + NS_EPS)
        for _ in range(case["steps"]):
            A = X @ X.t()
            X = NS_A * X + (NS_B * A + NS_C * (A @ A)) @ X
        out.append((X.t() if tall else X).contiguous().to(torch.bfloat16))
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "q4":
        nw = case["n_in"] * case["n_out"]
        ng = -(-case["n_in"] // case["group"])
        byt = case["n"] * (nw // 2 + ng * case["n_out"] * (2 if case["scale"] == "bf16" else 4)
                           + case["T"] * case["n_out"] * (2 if case["y"] == "bf16" else 4))
        byt += case["T"] * case["n_in"] * (2 if case["act"] == "bf16" else 4)
        return {"bytes": byt, "flops": 2 * case["n"] * case["T"] * nw}
    if op == "ortho":
        byt = flops = 0
        for r, c in _ortho_shapes(case):
            m, n = min(r, c), max(r, c)
            byt += r * c * ((2 if case["grad"] == "bf16" else 4) + 2)
            # two symmetric products (half of each) and one full product a step
            flops += case["steps"] * (m * m * n + m * m * m + 2 * m * m * n)
        return {"bytes": byt, "flops": flops}
    es = 2 if case["act"] == "bf16" else 4
    C = case["C"]
    if op == "recur_step":
        return {"bytes": case["B"] * C * (4 * es + 8), "flops": 12 * case["B"] * C}
    n, ends = case["T"] * C, case["seqs"] * C * 4
    if op == "recur_fwd":
        return {"bytes": 4 * n * es + 2 * ends, "flops": 12 * n}
    dy = 2 if case["dy"] == "bf16" else 4
    return {"bytes": n * (6 * es + dy) + 3 * ends, "flops": 30 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    d = _data(case, seed)
    op = case["op"]
    f64 = torch.float64
    gate = lambda x: 1.0 / (1.0 + torch.exp(-x.to(f64)))
    if op == "recur_step":
        w = gate(d["K"])
        h = (1.0 - w) * d["h"].to(f64) + w * d["V"].to(f64)
        return gate(d["R"]) * h, h
    if op in ("recur_fwd", "recur_bwd"):
        off = d["offsets"].tolist()
        seqs = [(s, a, b) for s, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a]
        write = gate(d["K"])
        H = write * d["V"].to(f64)               # becomes h, token after token
        before = torch.empty_like(H)             # h of the token before
        end = d["h0"].to(f64).clone()
        for s, a, b in seqs:
            h = d["h0"][s].to(f64)
            for t in range(a, b):
                before[t] = h
                h = torch.addcmul(H[t], 1.0 - write[t], h)
                H[t] = h
            end[s] = h
        if op == "recur_fwd":
            return gate(d["R"]) * H, end
        # 1 - w of a wide-open gate is lost to cancellation: the gate of -k instead
        shut = gate(-d["K"].to(f64))
        rec = gate(d["R"])
        dy = d["dY"].to(f64)
        dR = dy * H * rec * gate(-d["R"].to(f64))
        del H
        grad = dy.mul_(rec)
        del rec
        dh0 = d["dhT"].to(f64).clone()
        for s, a, b in seqs:
            back = dh0[s].clone()
            for t in range(b - 1, a - 1, -1):
                grad[t] += back
                back = shut[t] * grad[t]
            dh0[s] = back
        dK = (d["V"].to(f64) - before).mul_(grad).mul_(write).mul_(shut)
        return dK, grad * write, dR, dh0
    if op == "q4":
        X = d["X"].to(f64)
        out = []
        for q, s in zip(d["q"], d["gscale"]):
            Y = torch.zeros(case["T"], case["n_out"], dtype=f64, device=X.device)
            for j in range(s.shape[0]):
                rows = slice(j * case["group"], min((j + 1) * case["group"], case["n_in"]))
                Y += (X[:, rows] @ q[rows].to(f64)) * s[j].to(f64)
            out.append(Y)
        return out
    out = []
    for G in d["G"]:
        X = G.to(f64)
        X = X / (torch.linalg.vector_norm(X) + NS_EPS)
        if X.shape[0] <= X.shape[1]:
            for _ in range(case["steps"]):
                P = X @ X.T.contiguous()
                X = NS_A * X + NS_B * (P @ X) + NS_C * (P @ (P @ X))
        else:
            for _ in range(case["steps"]):
                P = X.T.contiguous() @ X
                X = NS_A * X + NS_B * (X @ P) + NS_C * ((X @ P) @ P)
        out.append(X)
    return out
