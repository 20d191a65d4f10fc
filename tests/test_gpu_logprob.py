"""Log probabilities, entropies and top alternatives of tokens on the GPU against
the formulas in 64 bits (tests/rows_ref.py); the alternatives' ids are exact."""
import math

import pytest
import torch

import rows_ref as ref
import ternary_weight_linear_tern_amd as tl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


def logits(T, V, seed, dt=F32, size=2.0, extra=0):
    """[T, V] in rows that start on 16 bytes; what stands between V and the stride
    (`extra` more columns of it) is NaN, which nothing may read into a result."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = (V + 7) // 8 * 8 + extra
    buf = torch.full((T, ld), math.nan, dtype=dt, device="cuda")
    buf[:, :V] = (torch.randn(T, V, generator=g, device="cuda") * size).to(dt)
    return buf[:, :V]


def run(Z, k=0, scale=1.0, tokens=None, ws=None):
    T, V = Z.shape
    new = lambda *s: torch.full(s, 77.0, device="cuda")
    o = dict(entropy=new(T), lse=new(T))
    if tokens is not None:
        o["logp"] = new(T)
    if k:
        o["top_ids"], o["top_logp"] = torch.full((T, k), -7, device="cuda"), new(T, k)
    tl.tern_logprob(Z, tl.empty_logprob_workspace(T, V, k) if ws is None else ws, tokens=tokens, scale=scale, **o)
    return o


def check(Z, k=0, scale=1.0, tokens=None, tag=""):
    T, V = Z.shape
    if tokens is None:
        g = torch.Generator(device="cuda").manual_seed(V)
        tokens = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    got, want = run(Z, k, scale, tokens), ref.logprob(Z, scale, tokens, k)
    nan = torch.isnan(want["lse"][0])
    for name, w in want.items():
        if name == "top_ids":
            assert bool(((got[name] >= 0) & (got[name] < V)).all()), tag
            assert torch.equal(got[name][~nan], w[~nan]), f"{tag} top_ids"
        else:
            ref.assert_within(got[name], *w, tag=f"{tag} {name}")
    return got


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 64, 65, 255, 256, 257, 511, 513, 1000, 2047, 2048, 4100, 8191, 16384,
                               32771, 50021, 65536, 65544, 131072, 131077, 262147, 1048576])
@pytest.mark.parametrize("dt", [F32, BF])
def test_sizes(V, dt):
    for T in (1, 3, 19 if V < 70000 else 2):
        check(logits(T, V, V + T, dt), k=min(V, 20), tag=f"{T} x {V} {dt}")
    check(logits(2, V, 5, dt), k=min(V, 64), tag=f"2 x {V} {dt} top 64")
    check(logits(2, V, 6, dt, extra=24), k=1, tag=f"2 x {V} {dt} strided")


@pytest.mark.parametrize("T,V", [(300, 256), (1500, 1000), (700, 8200), (600, 65536), (260, 131072), (20000, 64)])
@pytest.mark.parametrize("k", [0, 1, 5, 33])
def test_many_rows(T, V, k):
    check(logits(T, V, k, BF), k=k, scale=0.5, tag=f"{T} x {V} k {k}")


@pytest.mark.parametrize("V", [8, 64, 100, 127, 128, 250, 256, 512, 1000, 2000, 4000])
@pytest.mark.parametrize("dt", [F32, BF])
def test_alternatives_of_short_rows(V, dt):
    """Rows of one wave (2100 of them): from few of its lanes' elements to most of the row."""
    Z = logits(2100, V, V, dt)
    Z[::5] = torch.round(Z[::5])                       # ties
    Z[1::5, V // 3:] = -INF                            # a third is allowed
    Z[2::5, 1:] = -INF
    for k in sorted({min(V, k) for k in (2, 4, 15, 16, 17, 31, 32, 33, 50, 63, 64)}):
        check(Z, k=k, tag=f"{V} {dt} top {k}")
    check(hard_rows(V, dt, 150), k=min(V, 64), tag=f"{V} {dt} hard")


@pytest.mark.parametrize("scale", [1.0, 0.125, 1.7, 30.0])
def test_scales(scale):
    check(logits(7, 5000, 1), k=9, scale=scale, tag=str(scale))
    check(logits(7, 70000, 2, BF, size=5.0), k=9, scale=scale, tag=str(scale))


def hard_rows(V, dt, times=1):
    """Rows that are hard to choose from or to sum: ties, runs, few allowed, none."""
    g = torch.Generator(device="cuda").manual_seed(3)
    i = torch.arange(V, device="cuda")
    rows = [torch.zeros(V, device="cuda"),                                  # all alike
            torch.full((V,), -INF, device="cuda"),                          # nothing allowed
            i / V * 8, (V - i) / V * 8,                                     # rising, falling
            (i % 7).float(), (i % 2048 < 40).float() * 3,                   # many ties, a period of the tiles
            torch.where(i == V - 1, 5.0, -INF), torch.where(i % 97 == 3, 1.0, -INF),   # few allowed
            torch.where(i < V // 2, -3.3e38, 0.0), torch.full((V,), -3.3e38, device="cuda"),
            torch.where(i % 2 == 0, 0.0, -0.0),                             # -0 ties with +0
            torch.randn(V, generator=g, device="cuda") * 1e-3 + 90.0,
            torch.where(i // 8 % 1024 < 3, 4.0, 0.0) + torch.randn(V, generator=g, device="cuda") * 1e-2,
            torch.where(i == V // 3, 200.0, 0.0)]
    ld = (V + 7) // 8 * 8
    buf = torch.zeros(len(rows), ld, dtype=dt, device="cuda")
    for t, r in enumerate(rows):
        buf[t, :V] = r.to(dt)
    return buf.repeat(times, 1)[:, :V]


@pytest.mark.parametrize("V", [64, 256, 1000, 5003, 40000, 131072, 300000])
@pytest.mark.parametrize("dt", [F32, BF])
def test_hard_rows(V, dt):
    Z = hard_rows(V, dt)
    for k in (1, 20, 64):
        check(Z, k=k, tag=f"{V} {dt} top {k}")
    # enough rows that none is cut among workgroups
    check(hard_rows(V, dt, 40), k=20, tag=f"{V} {dt} many")


@pytest.mark.parametrize("V", [2000, 30000, 131072, 500000])
@pytest.mark.parametrize("dt", [F32, BF])
def test_alternatives_close_together(V, dt):
    """The large values stand in few places of every stride of 2048 (or 512), where the
    lanes' largest elements say little of the others'; values that repeat; a few
    tokens allowed among them."""
    g = torch.Generator(device="cuda").manual_seed(8)
    i = torch.arange(V, device="cuda")
    R = lambda: torch.randn(V, generator=g, device="cuda")
    rows = [torch.where(i % 2048 < 512, R(), R() - 20), torch.where(i % 512 < 64, R(), R() - 20),
            torch.where(i % 2048 < 8, R(), -INF), torch.where(i % 2048 < 512, torch.round(R() * 2), -3.0),
            torch.where(i // 8 % 256 < 66, i / V, -1.0), torch.where(i % 3 == 0, torch.round(R()), -INF)]
    ld = (V + 7) // 8 * 8
    buf = torch.zeros(len(rows), ld, dtype=dt, device="cuda")
    for t, r in enumerate(rows):
        buf[t, :V] = r.to(dt)
    for k in (1, 2, 33, 64):
        check(buf[:, :V], k=k, tag=f"{V} {dt} top {k}")
        check(buf.repeat(100, 1)[:, :V], k=k, tag=f"{V} {dt} top {k}, many")


@pytest.mark.parametrize("V", [256, 50021, 200000])
def test_certain_rows(V):
    """One token has next to all probability: no log probability above 0, no entropy below."""
    for gap in (5.0, 15.0, 30.0, 100.0):
        Z = logits(5, V, 3, size=1e-3)
        Z += 37.123
        Z[:, V // 2] += gap
        o = check(Z, k=3, tokens=torch.full((5,), V // 2, device="cuda"), tag=f"{V} {gap}")
        assert bool((o["logp"] <= 0).all()) and bool((o["top_logp"] <= 0).all()) and bool((o["entropy"] >= 0).all())


@pytest.mark.parametrize("V", [100, 3000, 131072])
def test_non_finite_rows_stay_alone(V):
    Z = logits(7, V, 4)
    good = run(Z, k=10)
    Z[1, 5], Z[3, V - 1], Z[5] = math.nan, INF, math.nan
    got = check(Z, k=10, tag=str(V))
    for t in (0, 2, 4, 6):
        for name in got:
            if name != "logp":
                assert torch.equal(got[name][t], good[name][t])


def test_nothing_allowed():
    Z = torch.full((3, 1000), -INF, device="cuda")
    Z[1] = 0.0
    o = run(Z, k=3, tokens=torch.tensor([5, 5, -1], device="cuda"))
    assert o["lse"].tolist()[0] == -INF and o["entropy"].tolist()[0] == 0 and o["logp"].tolist()[0] == -INF
    assert o["logp"].tolist()[2] == 0
    assert o["top_ids"].tolist()[0] == [0, 1, 2] and o["top_logp"].tolist()[0] == [-INF] * 3


def test_outputs_are_optional():
    Z = logits(5, 3001, 1)
    tok = torch.tensor([0, 3000, 17, 3001, -1], device="cuda")
    want = run(Z, k=4, tokens=tok)
    for names in (("lse",), ("entropy",), ("logp",), ("top_ids", "top_logp")):
        o = {n: torch.empty_like(want[n]) for n in names}
        tl.tern_logprob(Z, tl.empty_logprob_workspace(5, 3001, 4), tokens=tok if "logp" in names else None, **o)
        assert all(torch.equal(o[n], want[n]) for n in names)
    tl.tern_logprob(torch.empty(0, 64, device="cuda"), lse=torch.empty(0, device="cuda"))


def test_far_rows():
    """Offsets past 2^31 elements: the last rows of a matrix of 2.3e9 logits."""
    T, V = 17600, 131072
    Z = torch.zeros(T, V, dtype=BF, device="cuda")
    tail = logits(3, V, 9, BF)
    Z[-3:] = tail
    a, b = run(Z, k=2), run(tail, k=2)
    ids = ref.top(tail, 2)
    assert torch.equal(a["top_ids"][-3:], ids) and torch.equal(b["top_ids"], ids)
    want = ref.logprob(tail, 1.0, None, 0)
    ref.assert_within(a["lse"][-3:], *want["lse"], tag="lse")
    assert torch.equal(a["top_ids"][0], torch.tensor([0, 1], device="cuda"))


@pytest.mark.parametrize("T,V", [(300000, 64), (70000, 5003), (66000, 8200), (65600, 40000)])
def test_more_rows_than_workgroups(T, V):
    """Workgroups go on to further rows: equal rows but for the last ones."""
    ld = (V + 7) // 8 * 8
    tail = logits(5, V, 2, BF)
    Z = logits(1, V, 3, BF).repeat(T, 1) if V % 8 == 0 else torch.zeros(T, ld, dtype=BF, device="cuda")[:, :V]
    Z[-5:] = tail
    a, b = run(Z, k=3), run(tail, k=3)
    want = ref.logprob(tail, 1.0, None, 3)
    assert torch.equal(a["top_ids"][-5:], want["top_ids"])
    for name in ("lse", "entropy", "top_logp"):
        ref.assert_within(a[name][-5:], *want[name], tag=name)
        assert bool((a[name][:-5] == a[name][:1]).all())
    assert bool((a["top_ids"][:-5] == a["top_ids"][:1]).all())


@pytest.mark.parametrize("T,V", [(3, 131072), (700, 50024), (4000, 256)])
def test_repeats_bitwise(T, V):
    Z = logits(T, V, 1, BF)
    first = run(Z, k=20)
    for _ in range(3):
        again = run(Z, k=20)
        assert all(torch.equal(first[n], again[n]) for n in first)
