"""Log probabilities, entropy and alternatives: the CUDA path against the
definition in 64 bits, and the calls that are refused.

Tolerances.  With z = (x - max) / T, E the mean of |z| under p: the factor
log2(e) / T is off by 2^-24 and its constant by 2^-25, t by two more roundings:
3.5 2^-24 of z in every weight: 2.1e-7 E; a token's own z by two, 2^-23 |z|.  A
weight is off by ex2's 2^-22.  A sum passes at most 16 + 2 additions in its
batch, 128 batches and 5 + 5 + 4 inside the warp, the CTA and the cluster, 160
2^-24.  A change of the reference (two roundings and an ex2, 2^-23 + 2^-22) makes
what it touches 2^-8 of itself or less, so all of them count for 1.01 such errors;
the joins change it twice more: 1.1e-5, below 1.5e-5 of S.
ln S is off by 2^-22 of itself, at most 3.2e-6 more with S < 2^19.  So log p is
off by 1.9e-5 + 2.1e-7 (|z| + E) and its own rounding, 2^-24 of it; the entropy,
of which both ln S and a mean of z have that error, by 1.9e-5 (1 + E) + 2.1e-7 E
and 2^-24 of itself."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_target_gb300 as sv
from speculative_decoding_target_gb300 import _native, build

DEV = "cuda"
MOST = {t: torch.finfo(t).max for t in (torch.float32, torch.bfloat16)}


def reference(x, token, t, top, most):
    """One row in 64 bits: (logprob, entropy, ids, their log p, E, z)."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x.astype(np.float64), most))
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    lp = np.full(len(x), -np.inf)
    if len(order) == 0:
        H, E = 0.0, 0.0
    elif t == 0:
        lp[order[0]], H, E = 0.0, 0.0, 0.0
    else:
        z = (x - x[order[0]]) / t
        e = np.exp(z)
        S = e.sum()
        lp = z - np.log(S)
        p = e / S
        E = -(p[order] * np.maximum(z[order], -1e300)).sum()
        H = np.log(S) + E
    ids = np.full(top, -1)
    n = min(top, len(order))
    ids[:n] = order[:n]
    best = np.full(top, -np.inf)
    best[:n] = lp[order[:n]]
    return (lp[token] if token is not None else None), H, ids, best, E


def check(x, out, token, t, top):
    rows = x.shape[0]
    xs = x.float().cpu().numpy()
    got = {k: v.double().cpu().numpy() for k, v in out.items()}
    for r in range(rows):
        tok = None if token is None else int(token[r])
        tr = 1.0 if t is None else float(t[r])
        idle = (tok is not None and not 0 <= tok < x.shape[1]) or not (
            0 <= tr < np.inf)
        if idle:
            assert got["entropy"][r] == 0
            assert token is None or got["logprob"][r] == 0
            if top:
                assert (got["top_ids"][r] == -1).all()
                assert (got["top_logprobs"][r] == -np.inf).all()
            continue
        lp, H, ids, best, E = reference(xs[r], tok, tr, top, MOST[x.dtype])

        def near(a, b, tol):
            fin = np.isfinite(b)
            assert np.array_equal(np.isfinite(a), fin), (r, a, b)
            assert np.all(np.abs(a[fin] - b[fin]) <= tol[fin]), (r, a, b)
        lp_tol = lambda v: (1.9e-5 + 2.1e-7 * (np.abs(v) + H + E)
                            + 2.0 ** -24 * np.abs(v))
        if token is not None:
            v = np.array([lp])
            near(got["logprob"][r:r + 1], v, lp_tol(v))
        assert abs(got["entropy"][r] - H) <= (
            1.9e-5 * (1 + E) + 2.1e-7 * E + 2.0 ** -24 * H), (r, H)
        if top:
            assert np.array_equal(got["top_ids"][r], ids), (
                r, got["top_ids"][r], ids)
            near(got["top_logprobs"][r], best, lp_tol(best))


def run(x, token=None, t=None, top=0, **kw):
    build.build()
    i32 = lambda v: None if v is None else torch.as_tensor(
        v, dtype=torch.int32, device=DEV)
    f32 = lambda v: None if v is None else torch.as_tensor(
        v, dtype=torch.float32, device=DEV)
    return sv.logprobs(x, i32(token), temperature=f32(t), top=top, **kw)


def logits(rows, vocab, dtype, seed=0, spread=2.0, peaks=4):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((rows, vocab), generator=g, device=DEV) * spread
    if peaks and vocab > 8:
        at = torch.randint(0, vocab, (rows, peaks), generator=g, device=DEV)
        x.scatter_add_(1, at, torch.full(at.shape, 9.0, device=DEV))
    return x.to(dtype)


# ---------------------------------------------------------------- GPU tests

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (3, 2, 5), (2, 7, 32), (5, 31, 20), (9, 900, 1), (4, 5003, 32),
    (17, 50001, 8), (1, 248320, 20), (40, 248320, 5), (3, 524288, 32),
    (400, 4099, 3), (700, 33000, 0)])
def test_sizes(dtype, rows, vocab, top):
    x = logits(rows, vocab, dtype, seed=vocab)
    r = np.random.default_rng(rows)
    token = r.integers(0, vocab, rows)
    t = r.uniform(0.3, 2.0, rows).astype(np.float32)
    check(x, run(x, token, t, top), token, t, top)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,stride", [(0, 5003), (1, 5001), (3, 5007),
                                        (7, 5000), (5, 9001)])
def test_strides_and_alignment(dtype, off, stride):
    buf = logits(1, 8 * stride + 16, dtype, seed=off, peaks=40)[0]
    x = buf[off:off + 8 * stride].view(8, stride)[:, :5000]
    token = np.arange(8) * 600
    check(x, run(x, token, None, 9), token, None, 9)
    # the largest in front of the first and behind the last whole vector
    buf[off], buf[off + 4999] = 30.0, 30.0
    buf[off + stride], buf[off + stride + 1] = 30.0, 31.0
    check(x, run(x, token, None, 3), token, None, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(6, 60000), (400, 20011)])
def test_equal_logits(dtype, rows, vocab):
    # rows of one value; two values, the larger behind; few values; equals
    # that lie in one thread's vectors
    x = torch.zeros((rows, vocab), device=DEV)
    x[1] = -3.5
    x[2, vocab // 2:] = 1.0
    g = torch.Generator(device=DEV).manual_seed(1)
    x[3] = torch.randint(0, 3, (vocab,), generator=g, device=DEV).float()
    x[4, ::4096] = 2.0
    x[5, 8 * 512 * torch.arange(vocab // 4096, device=DEV) + 17] = 5.0
    x = x.to(dtype)
    token = np.arange(rows) % vocab
    check(x, run(x, token, None, 32), token, None, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [700, 40000])
def test_one_thread_holds_the_best(dtype, vocab):
    # sorted rows, and rows whose best lie in the same few vectors
    x = logits(4, vocab, dtype, peaks=0)
    x[0] = x[0].sort()[0]
    x[1] = x[1].sort(descending=True)[0]
    x[2, 64:104] += 50.0
    for v in range(0, vocab, 4096):
        x[3, v:v + 8] += 40.0
    token = [3, 600, 70, 0]
    check(x, run(x, token, None, 32), token, None, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [65, 30011])
def test_values_that_are_not_finite(dtype, vocab):
    inf, nan = float("inf"), float("nan")
    x = logits(9, vocab, dtype, seed=3)
    x[0] = -inf
    x[1] = nan
    x[2, 1:] = -inf
    x[2, 0] = -3e38
    x[3, ::2] = -inf
    x[3, 1::4] = nan
    x[4, 60], x[4, 61] = inf, MOST[dtype]
    x[5] = torch.finfo(dtype).min
    x[5, 64] = nan
    x[6, 5:] = torch.finfo(dtype).min
    x[7, :60] = -1e30
    x[8, 7] = 3e38
    token = [4, 5, 0, 2, 61, 3, 60, 1, 7]
    check(x, run(x, token, None, 7), token, None, 7)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(12, 30000), (330, 9001)])
def test_temperatures_and_idle_rows(dtype, rows, vocab):
    x = logits(rows, vocab, dtype, seed=4)
    t = np.ones(rows, np.float32)
    t[:12] = [0, 0, 1e-3, 100.0, -1, np.nan, np.inf, 1, 1, 1, 1e30, 0]
    token = np.arange(rows) * 7
    first = x.float().argmax(1).cpu().numpy()
    token[1] = first[1]
    token[7:10] = [-1, vocab, -(2 ** 31)]
    for top in (0, 4):
        check(x, run(x, token, t, top), token, t, top)
    check(x, run(x, None, t, 2), None, t, 2)


@pytest.mark.gpu
def test_against_a_long_tail():
    # one weight of one beside half a million of 2^-26: their sum counts
    x = torch.zeros((2, 524288), device=DEV)
    x[:, 77] = 26 * np.log(2)
    x[1, ::2] = -1.0
    x[1, 77] = 26 * np.log(2)
    check(x, run(x, [77, 3], None, 3), [77, 3], None, 3)


@pytest.mark.gpu
def test_shapes_streams_graphs_and_repeats():
    build.build()
    x = logits(64, 30000, torch.float32, seed=6).view(8, 8, 30000)
    token = torch.randint(-1, 30000, (8, 8), dtype=torch.int32, device=DEV)
    out = sv.logprobs(x, token, top=3)
    assert out["top_ids"].shape == (8, 8, 3) and out["logprob"].shape == (8, 8)
    check(x.view(64, -1), {k: v.flatten(0, 1) for k, v in out.items()},
          token.flatten().tolist(), None, 3)
    again = sv.logprobs(x, token, top=3)
    assert all(torch.equal(out[k], again[k]) for k in out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.logprobs(x, token, top=3, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(out[k], got[k]) for k in out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = sv.logprobs(x, token, top=3)
    x.mul_(0.5)
    token.fill_(5)
    g.replay()
    check(x.view(64, -1), {k: v.flatten(0, 1) for k, v in held.items()},
          [5] * 64, None, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 300000), (4870, 9001)])
def test_infinities_in_many_vectors(dtype, rows, vocab):
    # all count alike, so the first are the best; ends of threads differ
    inf = float("inf")
    x = logits(rows, vocab, dtype, seed=9)
    x[0] = inf
    x[0, 0] = -inf
    if rows > 1:
        x[1, 100::3] = inf
        x[1, 105] = MOST[dtype]
        token = np.full(rows, 101)
        token[5:] = -1
        token[0] = 7
    else:
        token = [3]
    check(x, run(x, token, None, 32), token, None, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_their_own(dtype):
    # several rows a CTA, idle ones and rows without mass between
    rows, vocab = 5003, 517
    x = logits(rows, vocab, dtype, seed=10)
    x[40] = -float("inf")
    token = np.arange(rows) % vocab
    token[::7] = -1
    t = np.where(np.arange(rows) % 5 == 0, 0.0, 0.7).astype(np.float32)
    for top in (0, 3):
        check(x, run(x, token, t, top), token, t, top)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 70])
def test_parts_with_many_large_logits(dtype, rows):
    # 31 large logits in each of a row's parts, however it is cut, and no 32nd
    # that a part's last place could rule them out by
    vocab = 60 * 4096
    x = logits(rows, vocab, dtype, seed=11, peaks=0)
    live = rows // 2
    at = torch.arange(60, device=DEV)[:, None] * 4096 + 64 * torch.arange(
        31, device=DEV)
    x[live, at.flatten()] = 100 + torch.randint(
        0, 64, (at.numel(),), device=DEV).to(dtype) / 2
    token = np.full(rows, -1)
    token[live] = 64 * 7
    check(x, run(x, token, None, 32), token, None, 32)


@pytest.mark.gpu
def test_long_rows_whole():
    # half a million fp32 tokens a CTA, values that rise through the row
    x = torch.zeros((310, 524288), device=DEV)
    x[5] = logits(1, 524288, torch.float32, seed=14)[0]
    x[5] += torch.linspace(0, 60, 524288, device=DEV)
    x[9, 77] = 26 * np.log(2)
    x[200] = torch.linspace(40, 0, 524288, device=DEV)
    token = np.full(310, -1)
    token[[5, 9, 200]] = [524287, 77, 100000]
    check(x, run(x, token, None, 3), token, None, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [9, 90])
def test_two_calls_at_once(rows):
    x = [logits(rows, 120000, torch.bfloat16, seed=12 + k) for k in range(2)]
    token = torch.arange(rows, dtype=torch.int32, device=DEV)
    want = [sv.logprobs(v, token, top=9) for v in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    got = [[sv.logprobs(v, token, top=9, stream=s) for v, s in zip(x, streams)]
           for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.gpu
def test_agrees_with_the_sampler():
    # the drawn token's log p is the log of the probability it was drawn with
    build.build()
    x = logits(20, 50000, torch.bfloat16, seed=8)
    t = torch.linspace(0.5, 1.5, 20, device=DEV)
    t[3] = 0
    u = torch.rand(20, device=DEV)
    probs = torch.empty((20, 50000), device=DEV)
    token = sv.sample(x, u, temperature=t, probs=probs)
    out = sv.logprobs(x, token, temperature=t, top=1)
    p = probs.gather(1, token.long()[:, None])[:, 0]
    # a weight of the sampler is a multiple of 2^-43 of the largest
    assert torch.allclose(out["logprob"].exp(), p, rtol=1e-4, atol=1e-11)
    assert torch.equal(out["top_ids"][:, 0].long(),
                       x.float().argmax(1)) and int(token[3]) == int(
        out["top_ids"][3, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(4, 70), (3, 60000), (400, 9001)])
def test_subnormal_logits_keep_their_order(dtype, rows, vocab):
    # the best logits are subnormals and zeros of both signs, single ones and
    # a thread's worth of neighbours
    x = logits(rows, vocab, dtype, seed=15, peaks=0) - 40
    whole = torch.int32 if dtype == torch.float32 else torch.int16
    g = torch.Generator(device=DEV).manual_seed(16)
    at = torch.stack([torch.randperm(vocab, generator=g, device=DEV)[:44]
                      for _ in range(rows)])
    at[:, 8:20] = vocab // 2 + torch.arange(12, device=DEV)
    most = 0x7fffff if dtype == torch.float32 else 0x7f
    small = torch.randint(1, most + 1, (rows, 44), generator=g, device=DEV)
    small[:, :4] = 0
    small = small.to(whole).view(dtype)
    small[:, 1::3] = -small[:, 1::3]
    x.scatter_(1, at, small)
    token = at[:, 9].tolist()
    t = np.where(np.arange(rows) % 2, 0.0, 1.0).astype(np.float32)
    check(x, run(x, token, t, 32), token, t, 32)
    check(x, run(x, token, t, 1), token, t, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(4, 70), (3, 60000), (400, 9001)])
def test_subnormal_logits_keep_their_order(dtype, rows, vocab):
    # the best logits are subnormals and zeros of both signs, single ones and
    # a thread's worth of neighbours
    x = logits(rows, vocab, dtype, seed=15, peaks=0) - 40
    whole = torch.int32 if dtype == torch.float32 else torch.int16
    g = torch.Generator(device=DEV).manual_seed(16)
    at = torch.stack([torch.randperm(vocab, generator=g, device=DEV)[:44]
                      for _ in range(rows)])
    at[:, 8:20] = vocab // 2 + torch.arange(12, device=DEV)
    most = 0x7fffff if dtype == torch.float32 else 0x7f
    small = torch.randint(1, most + 1, (rows, 44), generator=g, device=DEV)
    small[:, :4] = 0
    small = small.to(whole).view(dtype)
    small[:, 1::3] = -small[:, 1::3]
    x.scatter_(1, at, small)
    token = at[:, 9].tolist()
    t = np.where(np.arange(rows) % 2, 0.0, 1.0).astype(np.float32)
    check(x, run(x, token, t, 32), token, t, 32)
    check(x, run(x, token, t, 1), token, t, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(3000, 40), (150, 30000)])
def test_no_log_probability_above_zero(dtype, rows, vocab):
    # all the mass on one token: log p is 0 within its error, and not above
    g = torch.Generator(device=DEV).manual_seed(17)
    x = torch.full((rows, vocab), -float("inf"), device=DEV)
    token = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    x[torch.arange(rows), token] = torch.randn(
        rows, generator=g, device=DEV) * 10.0 ** torch.randint(
            -2, 6, (rows,), generator=g, device=DEV)
    x[::2] = torch.where(x[::2] == -float("inf"),
                         x[::2].amax(1, keepdim=True) - 30, x[::2])
    x = x.to(dtype)
    t = (0.2 + 2 * torch.rand(rows, generator=g, device=DEV)).cpu().numpy()
    out = run(x, token, t, 2)
    check(x, out, token.tolist(), t, 2)
    assert (out["logprob"] <= 0).all() and (out["top_logprobs"] <= 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab", [(9, 20000), (320, 3001)])
def test_temperatures_at_the_ends_of_their_range(rows, vocab):
    # logits as small or as large as the temperature, which counts as 2^-100
    # below that and as 2^100 above; subnormal ones are not zero
    x = logits(rows, vocab, torch.float32, seed=18)
    t = np.full(rows, 1.0)
    t[:9] = [1e-38, 1e-30, 1e-40, 1e-45, 3e38, 1e37, 1e30, 1e-31, -1e-45]
    scale = np.where((t == 1) | (t < 0), t, np.clip(t, 2.0 ** -100,
                                                    2.0 ** 100))
    x = x * torch.as_tensor(scale, dtype=torch.float32, device=DEV)[:, None]
    x[2, 5:9] = x[2].max()                  # equals share the mass
    x[3] = 0
    token = np.arange(rows) * 3 + 5
    out = run(x, token, t.astype(np.float32), 5)
    check(x, out, token, scale.astype(np.float32), 5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 3, 12, 30, 70, 153])
def test_parts_one_short_of_their_places(dtype, rows):
    # In each part that a row is cut into, top - 1 large logits and no other
    # that comes near: no part's last place is a bound for the join, which
    # then gets as many candidates as it can.
    top, vocab = 32, 248320
    size = 1                        # CTAs a row, by the rule of the launch
    while size < 16 and 2 * size * rows <= 2 * 152 and 2 * size * 4096 <= vocab:
        size *= 2
    x = logits(rows, vocab, dtype, seed=19, peaks=0)
    live = rows - 1
    part = vocab // size
    g = torch.Generator(device=DEV).manual_seed(20)
    for r in range(size):           # (off the parts' borders)
        at = r * part + 64 + torch.randperm(
            part - 128, generator=g, device=DEV)[:top - 1]
        x[live, at] = 100 + torch.randint(
            0, 64, (top - 1,), generator=g, device=DEV).to(dtype) / 2
    token = np.full(rows, -1)
    token[live] = 64
    check(x, run(x, token, None, top), token, None, top)


# ---------------------------------------------------------------- CPU tests

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: checks come first


def _raw(lib, **kw):
    d = _native.LogprobDesc(4, 1000, 0, 5, 1000)
    ptr = dict(logits=FAKE, token=FAKE, temperature=None, logprob=FAKE,
               entropy=FAKE, top_ids=FAKE, top_logprobs=FAKE)
    for name, val in kw.items():
        if name in ptr:
            ptr[name] = val
        else:
            setattr(d, name, val)
    return lib.spec_logprobs(ctypes.byref(d), *ptr.values(), None)


ODD = ctypes.c_void_p(0x100002)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), _native.SPEC_ERR_ARG),
    (dict(rows=(1 << 24) + 1), _native.SPEC_ERR_ARG),
    (dict(vocab=0), _native.SPEC_ERR_ARG),
    (dict(vocab=524289, row_stride=524289), _native.SPEC_ERR_UNSUPPORTED),
    (dict(dtype=2), _native.SPEC_ERR_ARG),
    (dict(row_stride=999), _native.SPEC_ERR_ARG),
    (dict(top=-1), _native.SPEC_ERR_ARG),
    (dict(top=33), _native.SPEC_ERR_ARG),
    (dict(top=0), _native.SPEC_ERR_ARG),
    (dict(top_ids=None), _native.SPEC_ERR_ARG),
    (dict(logits=None), _native.SPEC_ERR_ARG),
    (dict(token=None), _native.SPEC_ERR_ARG),
    (dict(top=0, top_ids=None, top_logprobs=None, logprob=None, entropy=None),
     _native.SPEC_ERR_ARG),
    (dict(logits=ODD), _native.SPEC_ERR_ALIGN),
    (dict(dtype=1, logits=ctypes.c_void_p(0x100001)), _native.SPEC_ERR_ALIGN),
    (dict(token=ODD), _native.SPEC_ERR_ALIGN),
    (dict(top_logprobs=ODD), _native.SPEC_ERR_ALIGN),
])
def test_refusals(kw, code):
    build.build()
    lib = _native.load()
    assert _raw(lib, **kw) == code
    assert lib.spec_last_error()


def test_no_rows_is_a_noop():
    build.build()
    assert _raw(_native.load(), rows=0, logits=None) == _native.SPEC_OK


def test_row_strides():
    stride = lambda x: _native._row_stride(x, x.shape[:-1].numel())
    x = torch.zeros((4, 6, 100))
    assert stride(x) == stride(x[0]) == 100
    assert stride(x[..., :90]) == stride(x[0, :, 5:95]) == 100
    assert stride(x[:, ::2, :90]) == 200 and stride(x[:, 3]) == 600
    assert stride(x[2:3, 3:4, 7:]) == 93
    for bad in (x[:, :4, :90], x[..., ::2], x.transpose(1, 2),
                x[0, :1].expand(3, 100), x[:, :1, :].expand(4, 2, 100)):
        with pytest.raises(sv.SpecError):
            stride(bad)


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 100))
    tok = torch.zeros(4, dtype=torch.int32)

    def refused(match, x=x, token=tok, **kw):
        with pytest.raises(sv.SpecError, match=match):
            sv.logprobs(x, token, **kw)
    refused("logits are", x=x.half())
    refused("token must be", token=tok.long())
    refused("token must be", token=tok[:3])
    refused("top", top=33)
    refused("top", top=10 ** 12)
    refused("top", top=-1)
    refused("temperature", temperature=torch.ones(3))
    refused("temperature", temperature=torch.ones(4, dtype=torch.float64))
    refused("CUDA device")                      # host tensors
