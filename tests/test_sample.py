"""Sampling with temperature, top-k, top-p and min-p: the CUDA path against
the definition in 64 bits, and the calls that are refused.

Tokens and kept sets have to be equal.  The kernel's weights are multiples of
2^-43 of the largest, each within 2^-43 of the exact one, so a sum of n weights
is within n 2^-43; a draw, or a border of the kept set, that lies closer than
that to another outcome is left out (with n = 250,000 a few draws in 100,000).
A probability is off by exp2 (2^-22) and the roundings of the sum to fp32 and
their product, below 2^-21 of its value; a weight 2^-y below 2^-19 of the
largest is exp2 of an fp32 argument made in three roundings, which adds
3 y 2^-24 ln 2."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_target_gb300 as sv
from speculative_decoding_target_gb300 import _native, build

DEV = "cuda"
gpu = pytest.mark.gpu


def reference(x, t, k, p, m, u):
    """One row in float64: (token, kept ids in order, probabilities over the
    vocabulary, the smallest distance of a decision in weights of which the
    largest is 1, as the bound is)."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    V = len(x)
    if not (t >= 0) or not np.isfinite(x).any():
        return -1, np.array([], int), np.zeros(V), 1.0
    order = np.lexsort((np.arange(V), -x))
    order = order[np.isfinite(x[order])]
    n, margin = len(order), 1.0
    if t == 0 or k == 1 or p <= 0 or m > 1:
        pr = np.zeros(V)
        pr[order[0]] = 1.0
        return int(order[0]), order[:1], pr, 1.0
    with np.errstate(over="ignore"):
        w = np.exp((x[order] - x[order[0]]) / t)
    if 0 < k < n:
        n = k
    w = w[:n]
    if p < 1:
        c = np.concatenate([[0.0], np.cumsum(w)])
        keep = c[:-1] < p * c[-1]
        keep[0] = True
        margin = min(margin, np.abs(c[1:-1] - p * c[-1]).min(initial=1.0))
        w, n = w[:int(keep.sum())], int(keep.sum())
    if m > 0:
        # one weight, not a sum of V of them, is off by 2^-43 at most (and
        # the largest, 1, by nothing): its distance counts V times
        margin = min(margin, V * np.abs(w - m)[w < 1].min(initial=1.0))
        keep = w >= m
        keep[0] = True
        w, n = w[:int(keep.sum())], int(keep.sum())
    ids = order[:n]
    full = np.zeros(V)
    full[ids] = w
    c = np.cumsum(full)
    target = float(u) * c[-1]
    tok = int(np.searchsorted(c, target, side="right"))
    near = c[ids.min():]
    margin = min(margin, np.abs(near - target).min())
    tok = min(tok, int(ids[w > 0].max()))
    return tok, ids, full / c[-1], margin


def run(x, t=None, k=None, p=None, m=None, u=None, **kw):
    build.build()
    f = lambda a, d: None if a is None else torch.as_tensor(
        a, dtype=d, device=DEV)
    x = x if torch.is_tensor(x) else torch.as_tensor(x, device=DEV)
    shape = x.shape
    probs = torch.full(shape, float("nan"), device=DEV)
    filt = torch.full(shape, float("nan"), device=DEV)
    args = dict(temperature=f(t, torch.float32), top_k=f(k, torch.int32),
                top_p=f(p, torch.float32), min_p=f(m, torch.float32))
    u = f(u, torch.float32)
    tok = sv.sample(x, u, probs=probs, filtered=filt, **args, **kw)
    alone = sv.sample(x, u, **args, **kw)
    assert torch.equal(tok, alone)         # the same without the outputs
    return tok.cpu().numpy(), probs.cpu().numpy(), filt.cpu().numpy()


def check(x, t, k, p, m, u, out=None):
    """Every row against the reference; returns how many were left out."""
    tok, probs, filt = out or run(x, t, k, p, m, u)
    xs = x.float().cpu().numpy() if torch.is_tensor(x) else np.asarray(x)
    rows, V = xs.shape
    left = 0
    one = lambda a, r, d: d if a is None else float(np.float32(a[r]))
    for r in range(rows):
        ref, ids, pr, margin = reference(
            xs[r], one(t, r, 1.0), 0 if k is None else int(k[r]),
            one(p, r, 1.0), one(m, r, 0.0), np.float32(u[r]))
        kept = np.isfinite(filt[r])
        if margin < V * 2.0 ** -43:
            left += 1
            continue
        assert tok[r] == ref, (r, tok[r], ref, margin)
        want = np.zeros(V, bool)
        want[ids] = True
        # a token whose weight rounds to nothing is kept or not by the
        # cumulative cuts alone
        assert np.array_equal(kept, want), (r, kept.sum(), want.sum())
        assert np.array_equal(filt[r][kept], xs[r][kept].clip(
            -np.inf, np.finfo(np.float32).max))
        top = max(pr.max(), 1e-300)
        y = np.log2(top / np.maximum(pr, 1e-300))
        tol = (np.where(y > 19, 3 * y * 2.0 ** -24 * np.log(2), 0)
               + 2.0 ** -21) * pr + 1e-37
        assert np.all(np.abs(probs[r] - pr) <= tol), (
            r, np.abs(probs[r] - pr).max())
    return left


def uniforms(n, seed):
    return np.random.default_rng(seed).random(n).astype(np.float32)


@gpu
@pytest.mark.parametrize("vocab", [1, 2, 7, 511, 4097, 32003, 248320])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_cut(vocab, dtype):
    g = torch.Generator(device=DEV).manual_seed(vocab)
    n = 24
    x = (torch.randn((n, vocab), generator=g, device=DEV) * 2).to(dtype)
    rng = np.random.default_rng(vocab)
    t = rng.choice([0.0, 0.3, 0.7, 1.0, 1.4, 5.0], n)
    k = rng.choice([0, 1, 2, 50, 1000, vocab - 1, vocab, vocab + 5], n)
    p = rng.choice([1.0, 0.01, 0.5, 0.9, 0.999, 2.0], n)
    m = rng.choice([0.0, 0.001, 0.1, 0.7, 1.0, -1.0], n)
    u = uniforms(n, vocab)
    assert check(x, t, k, p, m, u) <= 1
    for a in ((None, None, None, None), (t, None, None, None),
              (None, k, None, None), (None, None, p, None),
              (None, None, None, m), (t, k, p, None)):
        assert check(x[:8], *[v if v is None else v[:8] for v in a],
                     u[:8]) <= 1


@gpu
@pytest.mark.parametrize("vocab", [262144, 262145, 300007, 524288])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 10])
def test_largest_vocabularies(vocab, dtype, rows):
    # wide kept sets, drawn over the whole row: each CTA's share at its largest
    g = torch.Generator(device=DEV).manual_seed(vocab + rows)
    x = torch.randn((rows, vocab), generator=g, device=DEV).to(dtype)
    u = (np.arange(rows) + uniforms(rows, vocab)).astype(np.float32) / rows
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    assert check(x, [1.3] * rows, None, None, None, u) <= 1
    assert check(x, [0.9] * rows, None, [0.97] * rows, None, u) <= 1


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_top_k_where_few_threads_hold_the_values(dtype):
    # the threads' maxima tell little: finite values in few columns of 512,
    # one value in most of the row, fewer finite values than k
    V, n = 60000, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((n, V), generator=g, device=DEV) * 2
    few = torch.full_like(x, -float("inf"))
    few[:, 5::512] = x[:, 5::512]
    few[1, 5::512] = 1.25
    flat = torch.where(x > 6, x, torch.full_like(x, -1.0))
    flat[2] = torch.where(x[2] > 4, torch.full_like(x[2], 3.0), x[2] * 0)
    some = torch.full_like(x, -float("inf"))
    some[:, 1000:1030] = x[:, 1000:1030]
    dense = x.clone()                       # the largest values side by side
    dense[:, 7000:12000] = 9 + x[:, 7000:12000].abs() / 8
    k = [1, 2, 20, 50, 117, 118, 500, 1024]
    for i, y in enumerate((few, flat, some, dense)):
        y = y.to(dtype)
        u = uniforms(n, i)
        assert check(y, None, k, None, None, u) <= 1
        assert check(y, [0.8] * n, k, [0.9] * n, [0.01] * n, u) <= 1


@gpu
@pytest.mark.parametrize("vocab", [20011, 140009])
def test_many_rows_of_mixed_settings(vocab):
    # more clusters than are resident, rows that end at different steps, with
    # and without distributions, twice on two streams at once
    n = 230
    g = torch.Generator(device=DEV).manual_seed(vocab)
    x = torch.randn((n, vocab), generator=g, device=DEV) * 2.5
    rng = np.random.default_rng(vocab)
    t = rng.choice([0.0, 0.6, 1.0, 1.3, -1.0], n)
    k = rng.choice([0, 0, 1, 40, 300, 900, 5000], n)
    p = rng.choice([1.0, 0.5, 0.9, 0.99], n)
    m = rng.choice([0.0, 0.0, 0.02], n)
    u = uniforms(n, vocab)
    assert check(x, t, k, p, m, u) <= 1
    f = lambda a, d=torch.float32: torch.as_tensor(a, dtype=d, device=DEV)
    args = dict(temperature=f(t), top_k=f(k, torch.int32), top_p=f(p),
                min_p=f(m))
    want = sv.sample(x, f(u), **args)
    torch.cuda.synchronize()
    uu = f(u)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(sv.sample(x, uu, **args))
    torch.cuda.synchronize()
    for y in got:
        assert torch.equal(y, want)


@gpu
def test_peaked_rows_and_wide_ranges():
    rng = np.random.default_rng(1)
    n, V = 16, 50000
    x = rng.normal(size=(n, V)).astype(np.float32) * 2
    for r in range(n):
        x[r, rng.integers(0, V, 20)] += rng.uniform(5, 20, 20).astype(
            np.float32)
    x[3] *= 1000                      # one token holds nearly everything
    x[4] *= 1e30
    x[5] *= 1e-30                     # nearly equal weights
    x[6, :] = -np.inf
    x[6, 77] = -5.0                   # one finite logit
    x[7, ::2] = -np.inf
    p = rng.choice([0.3, 0.9, 0.99], n)
    t = rng.uniform(0.5, 1.5, n)
    u = uniforms(n, 2)
    assert check(x, t, None, p, None, u) <= 1
    assert check(x, t, [40] * n, p, [0.01] * n, u) <= 1
    assert check(x, t, None, None, None, u) <= 1


@gpu
def test_ties():
    # equal logits: the cuts take the lowest ids; exact at dyadic fractions
    V = 4096
    x = np.zeros((6, V), np.float32)
    x[1, 100:200] = 1.0
    x[2] = np.repeat(np.arange(64), 64)[::-1].astype(np.float32) / 8
    x[3] = -0.0
    x[3, ::3] = 0.0
    u = np.array([0.0, 0.5, 0.25, 0.999, 0.75, 0.1], np.float32)
    tok, probs, filt = run(x, None, [10, 150, 100, 7, 0, 0],
                           [1, 1, 1, 1, 0.5, 0.25], None, u)
    assert np.array_equal(np.flatnonzero(probs[0]), np.arange(10))
    assert tok[0] == 0 and np.allclose(probs[0][:10], 0.1)
    want1 = np.r_[0:50, 100:200]
    assert np.array_equal(np.flatnonzero(probs[1]), want1)
    assert np.array_equal(np.flatnonzero(probs[2]), np.arange(100))
    assert np.array_equal(np.flatnonzero(probs[3]), np.arange(7))
    assert tok[3] == 6                        # -0 and 0 are the same
    assert np.array_equal(np.flatnonzero(probs[4]), np.arange(V // 2))
    assert tok[4] == 3 * V // 8
    assert np.array_equal(np.flatnonzero(probs[5]), np.arange(V // 4))
    # bf16 rows with few distinct values, a border inside each
    g = torch.Generator(device=DEV).manual_seed(3)
    xb = (torch.randn((12, 100003), generator=g, device=DEV) * 0.02).to(
        torch.bfloat16)
    assert check(xb, None, [5000 * r + 3 for r in range(12)], None, None,
                 uniforms(12, 4)) <= 1
    assert check(xb, None, None, np.linspace(0.05, 0.95, 12), None,
                 uniforms(12, 5)) <= 1


@gpu
def test_one_value_and_wide_borders():
    # more equal logits at the border than one CTA sorts: the lowest ids
    V = 200000
    x = np.zeros((5, V), np.float32)
    x[1, 5000:5100] = 0.5
    x[2] = (np.arange(V) % 3).astype(np.float32)
    x[3] = -np.inf
    x[3, ::2] = 1.25
    x[4] = np.where(np.arange(V) < 100000, 2.0, 1.0)
    u = np.array([0.5, 0.999, 0.25, 0.75, 0.3], np.float32)
    tok, probs, _ = run(x, None, [70001, 3000, 66700, 50000, 150000], None,
                        None, u)
    zero = np.flatnonzero(x[1] == 0)[:2900]
    want = [np.arange(70001), np.sort(np.r_[np.arange(5000, 5100), zero]),
            np.sort(np.r_[np.flatnonzero(x[2] == 2),
                          np.flatnonzero(x[2] == 1)[:66700 - 66666]]),
            np.arange(0, 100000, 2), np.arange(150000)]
    for r in range(5):
        assert np.array_equal(np.flatnonzero(probs[r]), want[r]), r
    assert tok[0] == 35000 and tok[3] == 75000
    tok, probs, _ = run(x[:1], None, None, [0.5], None, u[:1])
    assert np.array_equal(np.flatnonzero(probs[0]), np.arange(V // 2))
    assert tok[0] == V // 4


@gpu
def test_idle_empty_and_special_rows():
    V = 1000
    rng = np.random.default_rng(6)
    x = rng.normal(size=(9, V)).astype(np.float32)
    t = np.ones(9, np.float32)
    t[0], t[1], t[2], t[3] = -1.0, np.nan, 0.0, np.inf
    x[2, [5, 700]] = 9.0                      # greedy: the lower id
    x[4] = -np.inf
    x[5, 10] = np.nan
    x[5, 20] = np.inf
    x[6, :] = np.nan
    x[7, [3, 8]] = np.inf                     # two largest values
    u = uniforms(9, 7)
    u[8] = 1.0                                # clamped below one
    tok, probs, filt = run(x, t, None, None, None, u)
    assert tok[0] == tok[1] == tok[4] == tok[6] == -1
    for r in (0, 1, 4, 6):
        assert not probs[r].any() and np.isneginf(filt[r]).all()
    assert tok[2] == 5 and probs[2][5] == 1 and probs[2].sum() == 1
    assert np.allclose(probs[3], 1 / V, rtol=1e-6)
    assert tok[5] == 20 and probs[5][10] == 0
    assert tok[7] in (3, 8) and probs[7][3] == probs[7][8] == 0.5
    assert tok[8] == V - 1
    assert check(x, t, None, None, None, u, (tok, probs, filt)) <= 2
    # bf16: +inf is the largest finite bf16
    xb = torch.zeros((2, 3000), dtype=torch.bfloat16, device=DEV)
    xb[0, [7, 2000]] = float("inf")
    xb[1, 5], xb[1, 6] = float("nan"), -float("inf")
    tok, probs, filt = run(xb, None, None, None, None, [0.9, 0.0])
    assert tok.tolist() == [2000, 0]
    assert probs[0][7] == probs[0][2000] == 0.5
    assert filt[0][7] == torch.finfo(torch.bfloat16).max
    assert probs[1][5] == probs[1][6] == 0 and np.isneginf(filt[1][[5, 6]]).all()


@gpu
def test_strides_shapes_alignment_and_streams():
    g = torch.Generator(device=DEV).manual_seed(8)
    big = torch.randn((5, 3001), generator=g, device=DEV)
    u = torch.rand(5, generator=g, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        b = big.to(dtype)
        for off in (0, 1, 3):
            view = b[:, off:off + 2990]
            tok = sv.sample(view, u)
            assert torch.equal(tok, sv.sample(view.contiguous(), u))
    # leading dimensions, on another stream, filtered in place
    x = torch.randn((2, 3, 5000), generator=g, device=DEV)
    u = torch.rand((2, 3), generator=g, device=DEV)
    p = torch.full((2, 3), 0.8, device=DEV)
    want = sv.sample(x, u, top_p=p)
    filt = torch.empty_like(x)
    sv.sample(x, u, top_p=p, filtered=filt)
    y = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.sample(y, u, top_p=p, filtered=y, stream=s)
    s.synchronize()
    assert want.shape == (2, 3) and torch.equal(got, want)
    assert torch.equal(y, filt)


@gpu
def test_captured_graph():
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn((7, 60000), generator=g, device=DEV) * 2
    u = torch.rand(7, generator=g, device=DEV)
    k = torch.full((7,), 100, dtype=torch.int32, device=DEV)
    tok = torch.empty(7, dtype=torch.int32, device=DEV)
    probs = torch.empty_like(x)
    sv.sample(x, u, top_k=k, token=tok, probs=probs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sample(x, u, top_k=k, token=tok, probs=probs)
    for seed in range(3):
        x.copy_(torch.randn((7, 60000), generator=g, device=DEV))
        u.copy_(torch.rand(7, generator=g, device=DEV))
        k.fill_(10 * seed + 1)
        graph.replay()
        p2 = torch.empty_like(x)
        assert torch.equal(tok, sv.sample(x, u, top_k=k, probs=p2))
        assert torch.equal(probs, p2)
        assert int((probs > 0).sum()) == 7 * (10 * seed + 1)


@gpu
def test_draws_follow_the_distribution():
    # one row, many uniforms on a grid: token counts are the probabilities
    # times the grid, off by at most one at each border
    g = torch.Generator(device=DEV).manual_seed(10)
    n = 4096
    row = torch.randn(300, generator=g, device=DEV) * 1.5
    x = row.expand(n, 300).contiguous()
    u = (torch.arange(n, device=DEV).float() + 0.5) / n
    p = torch.full((n,), 0.9, device=DEV)
    probs = torch.empty_like(x)
    tok = sv.sample(x, u, top_p=p, probs=probs)
    count = torch.bincount(tok.long(), minlength=300).double()
    assert bool(((count - probs[0].double() * n).abs() <= 1.001).all())
    assert bool((tok[1:] >= tok[:-1]).all())   # in id order


@gpu
def test_drafts_and_filtered_targets_in_stochastic_verify():
    # drafts drawn here with their distributions, and targets filtered here,
    # go through the stochastic verify: every committed token lies in the
    # target's kept set, and a drafter that equals the target is accepted
    B, q_len, V = 16, 5, 4000
    g = torch.Generator(device=DEV).manual_seed(11)
    target = torch.randn((B, q_len, V), generator=g, device=DEV) * 2
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)
    p = torch.full((B, q_len), 0.8, device=DEV)
    filt, probs = torch.empty_like(target), torch.empty_like(target)
    sv.sample(target, rand(B, q_len), top_p=p, filtered=filt, probs=probs)
    drafts = torch.zeros((B, q_len), dtype=torch.int32, device=DEV)
    q = torch.empty((B, q_len - 1, V), device=DEV)
    drafts[:, 1:] = sv.sample(target[:, :-1].contiguous(), rand(B, q_len - 1),
                              top_p=p[:, 1:].contiguous(), probs=q)
    acc, nxt, toks, _ = sv.stochastic_accept(
        filt.view(B * q_len, V), drafts, torch.ones(B, device=DEV),
        rand(B, q_len - 1) * 0.999, rand(B), draft_probs=q)
    assert bool((acc == q_len - 1).all())
    kept = torch.isfinite(filt)
    for j in range(q_len):
        assert bool(kept[torch.arange(B), j, toks[:, j].long()].all())


# Two neighbouring logits whose integer weights fall the other way round: the
# larger logit's is one step of 2^-43 below min_p, the smaller's is min_p.
# (temperature, largest logit, the larger, the smaller, min_p)
TURNED = [
    ("0x1.83611ap+0", "0x1.3edb4cp-2", "-0x1p-26", "-0x1.000002p-26",
     "0x1.a0c668p-1"),
    ("0x1.651896p+1", "0x1.1e31f6p+0", "-0x1.fffffep-25", "-0x1p-24",
     "0x1.56f472p-1"),
    ("0x1.b660e4p+1", "0x1.f744fcp+0", "-0x1p-24", "-0x1.000002p-24",
     "0x1.2063b8p-1"),
    ("0x1.0ebccp-1", "0x1.6b97cp-3", "-0x1p-27", "-0x1.000002p-27",
     "0x1.6dfb24p-1"),
]


@gpu
@pytest.mark.parametrize("cut", ["top-k", "top-p", "both", "none"])
def test_min_p_between_neighbouring_logits(cut):
    # whichever of the two min-p keeps, the token, the distribution and the
    # filtered logits are those of one kept set
    build.build()
    V, rows = 6000, len(TURNED)
    vals = [[float.fromhex(a) for a in r] for r in TURNED]
    x = torch.full((rows, V), -float("inf"))
    for r, (_, top, more, less, _) in enumerate(vals):
        x[r, 4000], x[r, 3000], x[r, 17] = top, more, less
        x[r, 5000] = top - 1000.0           # no weight: never kept
    x = x.to(DEV)
    f = lambda a, d=torch.float32: torch.tensor(a, dtype=d, device=DEV)
    kw = dict(temperature=f([v[0] for v in vals]),
              min_p=f([v[4] for v in vals]))
    if cut in ("top-k", "both"):
        kw["top_k"] = f([3] * rows, torch.int32)
    if cut in ("top-p", "both"):
        kw["top_p"] = f([0.9999999] * rows)
    for u in (0.0, 0.2, 0.35, 0.5, 0.75, 0.99):
        uu = f([u] * rows)
        probs = torch.full_like(x, float("nan"))
        filt = torch.full_like(x, float("nan"))
        tok = sv.sample(x, uu, probs=probs, filtered=filt, **kw)
        alone = sv.sample(x, uu, **kw)
        assert torch.equal(tok, alone)
        kept = torch.isfinite(filt)
        assert torch.equal(kept, probs > 0)
        assert bool(kept[:, 4000].all())
        # the smaller logit of the two is at the border, not below it
        assert bool(kept[:, 17].all())
        assert int(kept.sum(1).max()) <= 3
        p = probs.double()
        assert bool(((p.sum(1) - 1).abs() < 2.0 ** -20).all())
        run = p.cumsum(1)
        want = (run > u * run[:, -1:]).int().argmax(1)
        assert torch.equal(tok.long(), want)


# ---------------------------------------------------------------- CPU tests

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: checks come first


def _raw(rows=2, vocab=1000, dtype=0, stride=None, logits=FAKE, u=FAKE,
         token=FAKE, probs=None, t=None):
    build.build()
    d = _native.SampleDesc(rows, vocab, dtype,
                           vocab if stride is None else stride)
    return _native.load().spec_sample(ctypes.byref(d), logits, t, None, None,
                                      None, u, token, probs, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), _native.SPEC_ERR_ARG),
    (dict(rows=(1 << 24) + 1), _native.SPEC_ERR_ARG),
    (dict(vocab=0), _native.SPEC_ERR_ARG),
    (dict(vocab=524289), _native.SPEC_ERR_UNSUPPORTED),
    (dict(dtype=2), _native.SPEC_ERR_ARG),
    (dict(stride=999), _native.SPEC_ERR_ARG),
    (dict(logits=None), _native.SPEC_ERR_ARG),
    (dict(u=None), _native.SPEC_ERR_ARG),
    (dict(token=None), _native.SPEC_ERR_ARG),
    (dict(logits=ctypes.c_void_p(0x100002)), _native.SPEC_ERR_ALIGN),
    (dict(dtype=1, logits=ctypes.c_void_p(0x100001)), _native.SPEC_ERR_ALIGN),
    (dict(probs=ctypes.c_void_p(0x100002)), _native.SPEC_ERR_ALIGN),
    (dict(t=ctypes.c_void_p(0x100001)), _native.SPEC_ERR_ALIGN),
])
def test_refusals(kw, code):
    assert _raw(**kw) == code
    assert _native.load().spec_last_error()


def test_no_rows_is_a_noop():
    assert _raw(rows=0, logits=None) == _native.SPEC_OK


def test_binding_refuses_wrong_tensors():
    x, u = torch.zeros((2, 100)), torch.zeros(2)
    for a, kw in ((x.double(), {}), (x.half(), {}), (x[:, ::2], {}),
                  (x, dict(top_k=torch.zeros(2))),
                  (x, dict(top_p=torch.zeros(3))),
                  (x, dict(temperature=torch.ones(2).double())),
                  (x, dict(probs=torch.zeros(2, 99))),
                  (torch.zeros(100).expand(2, 100), {}), (x, {})):
        with pytest.raises(sv.SpecError):
            sv.sample(a, u, **kw)
    with pytest.raises(sv.SpecError):
        sv.sample(x, torch.zeros(3))
