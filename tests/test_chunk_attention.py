"""Attention of a chunk of new tokens over the paged cache: the CUDA path
against the definition in 64 bits, and the calls that are refused.

Tolerances, from the roundings.  With w the softmax weights of a row,
A = sum_t w_t |v_t| per channel and X = max_t scale sum_c |q_c k_tc|:
  bf16 KV   the weights are rounded to bf16, 2^-8 each: 2^-8 A;
  FP8 KV    dequantised K and V and the weights are rounded to fp16, 2^-11
            each; K's moves a score by 2^-11 X, a weight (and their sum) by
            twice that: (2^-11 + 2^-11 + 2^-10 X) A;
  both      fp32 scores (256 terms, 2^-18 X for both sides of the softmax),
            exp2, sums and the merge, below 2^-13: (2^-13 + 2^-18 X) A;
            the output in bf16: 2^-8 of its value."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_target_gb300 as sv
from speculative_decoding_target_gb300 import _native, build

DEV = "cuda"
D = 256


class Case:
    """Requests of `widths` new tokens behind `prefixes` cached ones, in pages
    in random order; every slot that no token lies in holds NaN, and table
    entries behind a request's pages are no pages."""

    def __init__(self, widths, prefixes, *, q_len=None, page=16, kv="bf16",
                 hq=24, hkv=4, seed=0, seqs=None, lens=True, room=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv, self.page, self.hq, self.hkv = kv, page, hq, hkv
        self.widths = list(widths)
        self.q_len = q_len or max(widths)
        B = self.B = len(widths)
        self.seqs = seqs or [p + w for p, w in zip(prefixes, widths)]
        need = [-(-s // page) for s in self.seqs]
        cols = max(1, max(need)) + room
        pages = self.pages = sum(need) + 3
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(
            seed)).to(torch.int32)
        table = torch.full((B, cols), 1 << 28, dtype=torch.int32)
        used = torch.zeros((pages, page), dtype=torch.bool)
        at = 0
        for b, s in enumerate(self.seqs):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            t = torch.arange(s)
            used[table[b, t // page].long(), t % page] = True
        used = used.to(DEV)[:, None, :, None]
        self.table = table.to(DEV)
        self.seq = torch.tensor(self.seqs, dtype=torch.int32, device=DEV)
        self.q_lens = (torch.tensor(self.widths, dtype=torch.int32, device=DEV)
                       if lens else None)
        if not lens:
            assert self.widths == [self.q_len] * B
        self.q = torch.randn((B, self.q_len, hq, D), generator=g,
                             device=DEV).to(torch.bfloat16)
        shape = (pages, hkv, page, D)
        self.ks = self.vs = None
        if kv == "bf16":
            pool = lambda: torch.where(
                used, torch.randn(shape, generator=g, device=DEV),
                torch.full((), float("nan"), device=DEV)).to(torch.bfloat16)
            self.k, self.v = pool(), pool()
        else:
            codes = lambda: torch.where(
                used, torch.randn(shape, generator=g, device=DEV).mul(100)
                .clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8),
                torch.full((), 0x7F, dtype=torch.uint8, device=DEV))
            scl = lambda: torch.where(
                used, 0.005 + 0.01 * torch.rand(
                    shape[:3] + (4,), generator=g, device=DEV),
                torch.full((), float("nan"), device=DEV)).half()
            self.k, self.v, self.ks, self.vs = codes(), codes(), scl(), scl()
        self.scale = D ** -0.5

    def run(self, **kw):
        build.build()
        return sv.chunk_attention(
            self.q, self.k, self.v, self.table, self.seq, scale=self.scale,
            k_scales=self.ks, v_scales=self.vs, q_lens=self.q_lens, **kw)

    def dense(self, pages, scales, b, n):
        x = pages[self.table[b, :-(-n // self.page)].long()]
        if scales is not None:
            ids = self.table[b, :-(-n // self.page)].long()
            x = x.view(torch.float8_e4m3fn).double()
            x = x * scales[ids].double().repeat_interleave(64, -1)
        return x.double().transpose(0, 1).reshape(self.hkv, -1, D)[:, :n]

    def check(self, out, rows=64):
        """Every row, or of long chunks `rows` of them, the first, the last
        and those beside 256-row and 128-token borders among them."""
        assert torch.isfinite(out.float()).all()
        G = self.hq // self.hkv
        for b in range(self.B):
            w, n = min(self.widths[b], self.q_len), self.seqs[b]
            live = min(w, n)
            assert not out[b, :w - live].any() and not out[b, w:].any()
            if not live:
                continue
            k, v = (self.dense(p, s, b, n) for p, s in
                    ((self.k, self.ks), (self.v, self.vs)))
            i = torch.arange(w - live, w)
            if live > rows:
                step = max(1, live // rows)
                tile = 256 / G
                near = [round(m * tile) + d for m in range(int(live / tile) + 1)
                        for d in (-1, 0)]
                near += [t - (n - w) + d for t in range(0, n, 128)
                         for d in (-1, 0)]
                pick = set(range(w - live, w, step)) | {w - live, w - 1}
                pick |= set(x for x in near[::max(1, len(near) // rows)])
                i = torch.tensor(sorted(x for x in pick if w - live <= x < w))
            for part in i.split(64):
                part = part.to(DEV)
                hidden = (torch.arange(n, device=DEV)
                          > (n - w + part)[:, None])[:, None]     # [r, 1, n]
                q = self.q[b, part].double().view(-1, self.hkv, G, D)
                for h in range(self.hkv):
                    z = torch.einsum("rgd,td->rgt", q[:, h], k[h]) * self.scale
                    X = (torch.einsum("rgd,td->rgt", q[:, h].abs(), k[h].abs())
                         .masked_fill(hidden, 0).amax(-1) * self.scale)
                    p = torch.softmax(z.masked_fill(hidden, -np.inf), -1)
                    want = p @ v[h]
                    A = p @ v[h].abs()
                    e = 2.0 ** -13 + 2.0 ** -18 * X
                    if self.kv == "bf16":
                        e = e + 2.0 ** -8
                    else:
                        e = e + 2.0 ** -10 + 2.0 ** -10 * X
                    got = out[b, part].double().view(
                        len(part), self.hkv, G, D)[:, h]
                    tol = e[..., None] * A + 2.0 ** -8 * want.abs()
                    assert torch.all((got - want).abs() <= tol), (
                        b, h, ((got - want).abs() / tol).max())


# ---------------------------------------------------------------- GPU tests

@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("page,widths,prefixes", [
    (16, [17], [0]), (64, [128], [0]), (8, [43, 17, 1], [5, 0, 300]),
    (32, [127, 0, 129, 64], [1, 50, 127, 3000]), (128, [257], [1000]),
    (4096, [300, 20], [5000, 100]), (16, [1, 1, 200, 1], [7000, 0, 200, 129]),
    (64, [1500], [0]), (16, [700, 650], [20000, 3]),
])
def test_sizes(kv, page, widths, prefixes):
    c = Case(widths, prefixes, page=page, kv=kv, seed=len(widths) + page)
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (7, 1), (40, 2), (300, 1),
                                    (32, 4)])
def test_heads(kv, hq, hkv):
    c = Case([50, 33, 2], [300, 0, 1000], hq=hq, hkv=hkv, kv=kv, seed=hq)
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_rows_without_tokens(kv):
    # longer than the cache, an empty cache, padded blocks, idle requests,
    # lengths past the table, widths outside [0, q_len]
    c = Case([100, 60, 0, 20, 100, 40], None, q_len=100, kv=kv, seed=3,
             seqs=[30, 0, 70, 20, 99, 300])
    out = torch.full_like(c.q, float("nan"))
    assert c.run(out=out) is out
    c.check(out)
    c = Case([50, 50], None, kv=kv, seed=4, seqs=[64, 50], lens=False)
    c.seq[0] = 1000                       # past the table: its end
    c.q_lens = torch.tensor([50, 90], dtype=torch.int32, device=DEV)
    c.check(c.run())
    c.q_lens[1] = -4
    c.widths[1] = 0
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("widths,prefixes,page", [
    ([20], [30000], 64), ([300], [20000], 16), ([900, 30], [12000, 17000], 32),
    ([3000], [0], 64)])
def test_every_tile_counts_once(kv, widths, prefixes, page):
    # equal weights (q = 0), and V has a channel for each 128-token tile: a
    # row's channel c is the share of its tokens that lies in tiles c, c + 256
    c = Case(widths, prefixes, page=page, kv=kv, seed=7)
    c.q.zero_()
    c.v.zero_()
    one = 0x38 if kv == "fp8" else 1.0                        # E4M3 one
    for b, n in enumerate(c.seqs):
        t = torch.arange(n, device=DEV)
        c.v[c.table[b, t // page].long(), :, t % page, t // 128 % 256] = one
    if kv == "fp8":
        c.vs.fill_(1.0)
    out = c.run().double()
    for b, n in enumerate(c.seqs):
        w = c.widths[b]
        i = torch.arange(w, device=DEV)
        limit = n - w + i + 1
        tiles = torch.arange(-(-n // 128), device=DEV)
        seen = (limit[:, None] - tiles * 128).clamp(0, 128).double()
        want = torch.zeros(w, 256, device=DEV, dtype=torch.float64)
        want.index_add_(1, tiles % 256, seen)
        want = (want / limit[:, None])[:, None]
        # equal weights are exact; fp32 sums and divisions, a bf16 output
        assert torch.all((out[b, :w] - want).abs()
                         <= want * (2.0 ** -8 + 2.0 ** -13))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_maxima_that_grow(kv):
    # keys that grow along the cache and inside the chunk: O is rescaled again
    # and again, also where a row's first tiles hold almost nothing
    c = Case([200], [3000], kv=kv, seed=11)
    n = c.seqs[0]
    t = torch.arange(n, device=DEV)
    at = (c.table[0, t // 16].long(), slice(None), t % 16)
    size = 0.05 + 2.5 * (t / n) ** 2
    if kv == "bf16":
        c.k[at] = (c.k[at].float() * size[:, None, None]).to(torch.bfloat16)
    else:
        c.ks[at] = (c.ks[at].float() * size[:, None, None]).half()
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_short_chunks_are_blocks(kv):
    c = Case([5, 16, 0], [100, 3000, 40], q_len=16, kv=kv, hq=32, hkv=4)
    build.build()
    want = sv.verify_attention(c.q, c.k, c.v, c.table, c.seq, scale=c.scale,
                               k_scales=c.ks, v_scales=c.vs, q_lens=c.q_lens)
    assert torch.equal(c.run(), want)
    small = Case([5], [100], page=4, hq=8, hkv=4)     # pages of 4 tokens
    small.check(small.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_streams_graphs_and_repeats(kv):
    c = Case([90, 40], [2000, 500], kv=kv, seed=5, room=8)
    want = c.run()
    c.check(want)
    assert torch.equal(c.run(), want)                 # the same on every run
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)                             # not the current stream
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    # two graphs, a workspace each, replayed on two streams at once
    outs = [torch.empty_like(c.q) for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # lengths move between replays
    c.seq.copy_(torch.tensor([1500, 77]))
    c.q_lens.copy_(torch.tensor([33, 40]))
    c.seqs, c.widths = [1500, 77], [33, 40]
    graphs[0].replay()
    c.check(outs[0])


def shifted(t):
    """The same tensor 16 bytes behind a 512-byte border."""
    if t is None:
        return None
    n = 16 // t.element_size()
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    buf[n:].copy_(t.reshape(-1))
    return buf[n:].view(t.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_addresses_of_16_bytes(kv):
    c = Case([70, 300], [500, 64], kv=kv, seed=11)
    want = c.run()
    c.q, c.k, c.v = shifted(c.q), shifted(c.k), shifted(c.v)
    c.ks, c.vs = shifted(c.ks), shifted(c.vs)
    out = shifted(torch.full_like(c.q, 7))
    assert out.data_ptr() % 32 == 16
    assert torch.equal(c.run(out=out), want)


@pytest.mark.gpu
def test_status_of_bad_pages():
    c = Case([60, 40], [500, 100], seed=6)
    ws = sv.alloc_workspace(256 << 20, DEV)
    c.check(c.run(checked=True, workspace=ws))
    assert sv.verify_status(ws) == 0
    c.table[1, 3] = c.pages
    out = c.run(checked=True, workspace=ws)
    assert sv.verify_status(ws) == _native.SPEC_STATUS_BAD_PAGE
    c.B = 1                                # the other request is as it was
    c.check(out)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("page,hq,hkv", [(16, 24, 4), (64, 48, 1)])
def test_waits_that_run_out_are_reported(kv, page, hq, hkv):
    # several pieces a pair; queries by tensor copies and by threads
    c = Case([2500, 70], [1000, 5000], page=page, kv=kv, hq=hq, hkv=hkv,
             seed=12)
    ws = sv.alloc_workspace(256 << 20, DEV)
    sv.set_wait_limit(200)      # SM clock cycles: the first waits run out
    try:
        c.run(checked=True, workspace=ws)
        torch.cuda.synchronize()
    finally:
        sv.set_wait_limit(0)
    assert sv.verify_status(ws) & _native.SPEC_STATUS_TIMEOUT
    out = c.run(checked=True, workspace=ws)
    assert sv.verify_status(ws) == 0
    c.check(out, rows=8)


@pytest.mark.gpu
def test_pool_of_more_than_2_31_elements():
    page, pages = 64, 140000
    c = Case([40], [1000], page=page, hq=6, hkv=1, seed=9)
    big = [torch.empty((pages, 1, page, D), dtype=torch.bfloat16, device=DEV)
           for _ in range(2)]
    n = c.table.shape[1]
    ids = pages - 1 - torch.arange(n, device=DEV)
    for x, y in zip(big, (c.k, c.v)):
        x[ids] = y[c.table[0].long()]
    c.k, c.v = big
    c.table = ids.to(torch.int32)[None].contiguous()
    c.pages = pages
    c.check(c.run())


@pytest.mark.gpu
def test_many_requests():
    r = np.random.default_rng(3)
    widths = r.integers(0, 30, 300).tolist()
    widths[7] = 30
    c = Case(widths, r.integers(0, 400, 300).tolist(), hq=8, hkv=2, seed=13)
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("widths", [[5, 1], [40, 17], [300, 2]])
def test_scales_below_the_normal_numbers(kv, widths):
    # every score is as good as zero: equal weights over what a row sees
    c = Case(widths, [200, 0], kv=kv, seed=21)
    for c.scale in (1e-38, 1e-40, 1e-45):
        c.check(c.run())


def check_rows(c, out, b, i):
    """The rows of block rows i of request b against the definition."""
    G, n = c.hq // c.hkv, c.seqs[b]
    i = torch.tensor(sorted(i), device=DEV)
    q = c.q[b, i].double().view(-1, c.hkv, G, D)
    got = out[b, i].double().view(-1, c.hkv, G, D)
    hidden = (torch.arange(n, device=DEV)
              > (n - c.widths[b] + i)[:, None])[:, None]
    k, v = (c.dense(p, s, b, n) for p, s in ((c.k, c.ks), (c.v, c.vs)))
    for h in range(c.hkv):
        z = torch.einsum("rgd,td->rgt", q[:, h], k[h]) * c.scale
        X = (torch.einsum("rgd,td->rgt", q[:, h].abs(), k[h].abs())
             .masked_fill(hidden, 0).amax(-1) * c.scale)
        p = torch.softmax(z.masked_fill(hidden, -np.inf), -1)
        want, A = p @ v[h], p @ v[h].abs()
        e = 2.0 ** -13 + 2.0 ** -18 * X + (
            2.0 ** -8 if c.kv == "bf16" else 2.0 ** -10 + 2.0 ** -10 * X)
        tol = e[..., None] * A + 2.0 ** -8 * want.abs()
        assert torch.all((got[:, h] - want).abs() <= tol), (b, h)


def rows_beside_borders(c, b, most=40):
    """Block rows on both sides of the borders of the CTAs' rows (every other
    one a row tile's), of 128 or of whole tokens, and of the 128-token tiles
    of the cache."""
    G, w, n = c.hq // c.hkv, c.widths[b], c.seqs[b]
    cta = [[((R - 1) // G, R // G) for R in range(rows, w * G, rows)]
           for rows in {128, 128 // G * G or 128}]
    tile = [(t - (n - w) - 1, t - (n - w))
            for t in range(-(-(n - w + 1) // 128) * 128, n, 128)]
    pick = {0, w - 1}
    for borders in (*cta, tile):
        for pair in borders[::-(-len(borders) // most) or 1]:
            pick |= set(pair)
    assert all(0 <= x < w for x in pick)
    return pick


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,widths,prefixes", [
    (24, 4, [1500], [0]), (24, 4, [700, 650], [20000, 3]),
    (24, 4, [300], [5000]), (4, 4, [1100], [77]), (38, 2, [400], [900]),
    (26, 2, [400], [900]), (150, 1, [90, 70], [0, 1000])])
def test_rows_beside_borders(kv, hq, hkv, widths, prefixes):
    c = Case(widths, prefixes, hq=hq, hkv=hkv, kv=kv, seed=22)
    out = c.run()
    for b in range(c.B):
        check_rows(c, out, b, rows_beside_borders(c, b))


# new tokens, cached ones, heads; 4,248, 4,416 and 4,108 pieces of 1,062, 138 and
# 1,027 row tiles.  Dealt to 76 pairs, four long pieces of the last are left
# behind 54 rounds, and those are cut.
LARGE = [([30000, 14500, 1], [0, 300, 2000], 24, 4),
         ([20000, 15000], [0, 0], 32, 32),
         ([168] * 256 + [126], [8000] * 257, 24, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("widths,prefixes,hq,hkv", LARGE)
def test_plans_of_many_pieces(kv, widths, prefixes, hq, hkv):
    # more pieces than the plan holds in shared memory, more row tiles than it
    # has threads: sampled rows, the first and the last of requests
    c = Case(widths, prefixes, page=64, kv=kv, hq=hq, hkv=hkv, seed=23)
    out = c.run()
    assert torch.isfinite(out.float()).all()
    r = np.random.default_rng(24)
    for b in sorted({0, 1, c.B - 1, *r.integers(0, c.B, 6).tolist()}):
        w = c.widths[b]
        check_rows(c, out, b, {0, w - 1, w // 2, *r.integers(0, w, 12)})
    assert torch.equal(c.run(), out)
    # every token of every row counts once: equal weights, and V that is a
    # number of the token's tile
    c.q.zero_()
    c.v.zero_()
    one = 0x38 if kv == "fp8" else 1.0                        # E4M3 one
    for b, n in enumerate(c.seqs):
        t = torch.arange(n, device=DEV)
        c.v[c.table[b, t // 64].long(), :, t % 64, t // 128 % 256] = one
    if kv == "fp8":
        c.vs.fill_(1.0)
    out = c.run()
    for b, n in enumerate(c.seqs):
        w = c.widths[b]
        limit = n - w + torch.arange(w, device=DEV) + 1
        tiles = torch.arange(-(-n // 128), device=DEV)
        want = torch.zeros(w, 256, device=DEV, dtype=torch.float64)
        want.index_add_(1, tiles % 256, (limit[:, None] - tiles * 128)
                        .clamp(0, 128).double())
        want = (want / limit[:, None])[:, None]
        # equal weights are exact; fp32 sums and divisions, a bf16 output
        assert torch.all((out[b, :w].double() - want).abs()
                         <= want * (2.0 ** -8 + 2.0 ** -13))


# ---------------------------------------------------------------- CPU tests

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: checks come first


def _raw(lib, **kw):
    d = _native.make_desc(batch=2, q_len=100, num_q_heads=24, num_kv_heads=4,
                          head_dim=256, page_size=16, num_pages=64,
                          max_pages_per_seq=8)
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, table=FAKE, seq=FAKE,
             scale=0.0625, out=FAKE, ws=None, ws_bytes=0)
    for name, val in kw.items():
        if name in a:
            a[name] = val
        else:
            setattr(d, name, val)
    return lib.spec_chunk_attention(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), _native.SPEC_ERR_ARG),
    (dict(batch=1025), _native.SPEC_ERR_ARG),
    (dict(q_len=0), _native.SPEC_ERR_ARG),
    (dict(q_len=1 << 27), _native.SPEC_ERR_ARG),
    (dict(batch=4, q_len=2 ** 31 - 1, num_q_heads=2 ** 31 - 1,
          num_kv_heads=1), _native.SPEC_ERR_ARG),   # 2^64 and more
    (dict(num_kv_heads=5), _native.SPEC_ERR_ARG),
    (dict(head_dim=128), _native.SPEC_ERR_UNSUPPORTED),
    (dict(page_size=24), _native.SPEC_ERR_ARG),
    (dict(page_size=4), _native.SPEC_ERR_UNSUPPORTED),
    (dict(num_pages=0), _native.SPEC_ERR_ARG),
    (dict(kv_dtype=2), _native.SPEC_ERR_ARG),
    (dict(flags=2), _native.SPEC_ERR_ARG),
    (dict(num_pages=1 << 26), _native.SPEC_ERR_UNSUPPORTED),
    (dict(q=None), _native.SPEC_ERR_ARG),
    (dict(out=None), _native.SPEC_ERR_ARG),
    (dict(table=None), _native.SPEC_ERR_ARG),
    (dict(scale=0.0), _native.SPEC_ERR_ARG),
    (dict(scale=float("nan")), _native.SPEC_ERR_ARG),
    (dict(scale=float("inf")), _native.SPEC_ERR_ARG),
    (dict(q=ctypes.c_void_p(0x100008)), _native.SPEC_ERR_ALIGN),
    (dict(seq=ctypes.c_void_p(0x100002)), _native.SPEC_ERR_ALIGN),
    (dict(kv_dtype=1), _native.SPEC_ERR_ARG),
    (dict(kv_dtype=1, ks=FAKE, vs=ctypes.c_void_p(0x100008)),
     _native.SPEC_ERR_ALIGN),
])
def test_refusals(kw, code):
    build.build()
    lib = _native.load()
    assert _raw(lib, **kw) == code
    assert lib.spec_last_error()


def test_empty_batch_is_a_noop():
    build.build()
    assert _raw(_native.load(), batch=0, q=None) == _native.SPEC_OK


@pytest.mark.gpu
def test_small_workspace_is_refused():
    c = Case([50], [100])
    build.build()
    for ws in (torch.empty(1024, dtype=torch.uint8, device=DEV),
               torch.empty(256 << 20, dtype=torch.uint8, device=DEV)[8:]):
        with pytest.raises(sv.SpecError):
            c.run(workspace=ws)
    desc = sv.desc_for(c.q, c.k, c.table)
    n = sv.chunk_workspace_size(desc)
    c.check(c.run(workspace=sv.alloc_workspace(n, DEV)))


def test_binding_refuses_wrong_tensors():
    q = torch.zeros((2, 50, 8, 256), dtype=torch.bfloat16)
    pool = torch.zeros((4, 4, 16, 256), dtype=torch.bfloat16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    seq = torch.zeros(2, dtype=torch.int32)

    def refused(match="", q=q, kp=pool, vp=pool, t=table, s=seq, **kw):
        with pytest.raises(sv.SpecError, match=match):
            sv.chunk_attention(q, kp, vp, t, s, scale=0.1, **kw)
    refused("q must be", q=q.float())
    refused("contiguous", q=q.transpose(1, 2).contiguous().transpose(1, 2))
    refused("v_pages", vp=pool[:, :2])
    refused("k_pages", kp=pool.half())
    refused("rows", t=table[:1])
    refused("seq_lens", s=seq.long())
    refused("q_lens", q_lens=seq.long())
    refused("out", out=q[:, :20])
    refused("CUDA device")                      # host tensors
