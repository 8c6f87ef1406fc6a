"""Verify attention with shared prefixes where most of a row's weights are
small: each shared token has to count with its own share.

Tolerances are those of test_shared_prefix.py.  FP8 KV adds what fp16 does to
the smallest weights: they carry a factor of 2^11, so one below 2^-25 of the
largest is off by half of fp16's last step, 2^-25 2^-11 = 2^-36 of the largest
weight: 2^-36 max(w) sum_t |v_t|."""
import pytest
import torch

import speculative_decoding_target_gb300 as sv
import test_shared_prefix as base
from test_shared_prefix import D, DEV, Case

gpu = pytest.mark.gpu


def compare(c, out):
    """Case.check, with the term of the smallest weights."""
    assert torch.isfinite(out.float()).all()
    G = c.hq // c.hkv
    for b in range(c.B):
        w, n = c.widths[b], c.seqs[b]
        if w:
            k, v = (c.dense(p, s, b, n) for p, s in ((c.k, c.ks), (c.v, c.vs)))
        for i in range(w):
            got = out[b, i].double().view(c.hkv, G, D)
            m = n - w + i + 1
            q = c.q[b, i].double().view(c.hkv, G, D)
            p = torch.softmax(torch.einsum(
                "hgd,htd->hgt", q, k[:, :m]) * c.scale, -1)
            o = torch.einsum("hgt,htd->hgd", p, v[:, :m])
            A = torch.einsum("hgt,htd->hgd", p, v[:, :m].abs())
            X = (torch.einsum("hgd,htd->hgt", q.abs(), k[:, :m].abs())
                 * c.scale).amax(-1, keepdim=True)
            per, small = 2.0 ** -8, 0.0
            if c.kv == "fp8":
                per = 2.0 ** -10 + 2.0 ** -10 * X
                small = (2.0 ** -36 * p.amax(-1, keepdim=True)
                         * v[:, :m].abs().sum(1)[:, None])
            tol = ((per + 2.0 ** -13 + 2.0 ** -18 * X) * A
                   + 2.0 ** -8 * o.abs() + small)
            err = (got - o).abs()
            assert bool((err <= tol).all()), (
                b, i, float((err / tol.clamp_min(1e-30)).max()))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bits", [18, 26, 30])
def test_small_weights_beside_dominating_tokens(kv, bits):
    # One token in 512, so that each run of tiles has some, takes nearly all
    # of the weight and has no value; the output is what the 131,072 tokens
    # `bits` below them hold together.
    N = 131072
    c = Case([2], [N], [40, 9], q_len=1, page=64, kv=kv, hq=6, hkv=1, seed=21)
    c.q[..., :64] = 4.0
    first = c.table[0, :N // 64:8].long()
    nan = c.k == 0x7F if kv == "fp8" else c.k.isnan()
    c.k[..., :64] = torch.where(nan[..., :64], c.k[..., :64], 0)
    # 64 channels of 4 key / 16 make a score of 16 key; key, a multiple of
    # 1/8, is exact in bf16, and 128 key in E4M3
    key = round(bits * 0.6931 / 16 * 8) / 8
    if kv == "bf16":
        c.k *= 0.3
        c.k[first, :, 0, :64] = key
        c.v = c.v.abs()
    else:
        c.ks *= 0.3
        c.ks[first, :, 0, 0] = 2.0 ** -7
        c.k[first, :, 0, :64] = torch.tensor(key * 128, device=DEV).to(
            torch.float8_e4m3fn).view(torch.uint8)
        c.v &= 0x7F
    c.v[first, :, 0] = 0
    compare(c, c.run())


# ---- every tile of a shared prefix counts ------------------------------------

def mark_tiles(c):
    """The shared tokens of 128-token tile n keep their value, made positive,
    in channel n % 256 alone: that channel of the output is the weight of the
    tile, whatever the length of the prefix, and its tolerance a fraction of
    it."""
    starts = c.starts.tolist()
    for n, shared in enumerate(c.shared.tolist()):
        ids = c.table[starts[n], :shared // c.page].long()
        if not len(ids):
            continue
        tile = torch.arange(shared, device=c.v.device).view(
            len(ids), 1, c.page, 1) // 128
        own = tile % D == torch.arange(D, device=c.v.device)
        x = c.v[ids]
        x = x & 0x7F if c.kv == "fp8" else x.abs()
        c.v[ids] = torch.where(own, x, torch.zeros_like(x))
    return c


def evaluate(c, wrong=None):
    """The attention of c in 64 bits, rounded to bf16, with a mistake in the
    shared tokens of tile 7: (what, ...)."""
    out = torch.zeros_like(c.q)
    G = c.hq // c.hkv
    for b in range(c.B):
        w, n = c.widths[b], c.seqs[b]
        k, v = (c.dense(p, s, b, n) for p, s in ((c.k, c.ks), (c.v, c.vs)))
        a, z = slice(7 * 128, 8 * 128), slice(12 * 128, 13 * 128)
        count = torch.ones(n, dtype=torch.float64)
        if wrong == "dropped":
            count[a] = 0
        elif wrong == "twice":
            count[a] = 2
        elif wrong == "other V":
            v[:, a] = v[:, z].clone()
        elif wrong == "other K":
            k[:, a] = k[:, z].clone()
        elif wrong == "halves of V":
            v[:, a] = v[:, a].roll(64, 1)
        for i in range(w):
            m = n - w + i + 1
            q = c.q[b, i].double().view(c.hkv, G, D)
            s = torch.einsum("hgd,htd->hgt", q, k[:, :m]) * c.scale
            p = torch.softmax(s, -1) * count[:m]
            p = p / p.sum(-1, keepdim=True)
            out[b, i] = torch.einsum("hgt,htd->hgd", p, v[:, :m]).reshape(
                c.hq, D).to(torch.bfloat16)
    return out


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_mistake_in_one_tile_shows(kv, monkeypatch):
    # on the CPU: the tolerance holds the exact result, and none with one tile
    # of a long prefix dropped, counted twice or with another tile's K or V
    monkeypatch.setattr(base, "DEV", "cpu")
    c = mark_tiles(Case([2], [30000], [100, 31], q_len=2, page=64, kv=kv,
                        hq=6, hkv=1, seed=11))
    c.check(evaluate(c))
    for wrong in ("dropped", "twice", "other V", "other K", "halves of V"):
        with pytest.raises(AssertionError):
            c.check(evaluate(c, wrong))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("shape", ["long", "one row", "small pages",
                                   "many groups"])
def test_every_tile_counts(kv, shape):
    if shape == "long":            # several runs and pieces a CTA pair
        c = Case([9, 2], [30000, 9000], [100] * 11, q_len=6, page=64, kv=kv,
                 seed=11)
    elif shape == "one row":
        c = Case([40], [20000], [100 + b for b in range(40)], q_len=1,
                 page=64, kv=kv, seed=13)
    elif shape == "small pages":
        c = Case([3, 4], [12000, 7000], [9 * b for b in range(7)], q_len=8,
                 page=8, kv=kv, seed=14)
    else:                          # 240 segments of ten tiles
        c = Case([3] * 60, [1280] * 60, [20] * 180, q_len=2, page=64, kv=kv,
                 seed=15)
    mark_tiles(c)
    ws = sv.alloc_workspace(256 << 20, DEV)
    out = c.run(checked=True, workspace=ws)
    assert sv.verify_status(ws) == 0
    c.check(out)


# ---- maxima that grow along the prefix ---------------------------------------

def plant(c, b, row, tok, beta):
    """Make shared token `tok` of request b's group beta times the queries of
    block row `row` of request b, one head of each KV head: their scores grow
    by about 23 beta (base 2), other rows' hardly."""
    pg, at = c.table[b, tok // c.page].item(), tok % c.page
    G = c.hq // c.hkv
    for g in range(c.hkv):
        x = c.q[b, row, g * G + (b + g) % G].float() * beta
        if c.kv == "bf16":
            c.k[pg, g, at] = x.to(torch.bfloat16)
            continue
        s = (x.view(4, 64).abs().amax(1) / 448).half()
        c.ks[pg, g, at] = s
        c.k[pg, g, at] = (x / s.float().repeat_interleave(64)).clamp(
            -448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_maxima_of_single_rows_grow(kv):
    # one row of a warp at a time: in the second tile, in the middle twice in
    # a row, in the last; with 240 pieces on 76 CTA pairs also behind another
    # piece, in either of a pair's score buffers
    c = Case([3] * 60, [1280] * 60, [20] * 180, q_len=2, page=64, kv=kv,
             seed=31)
    mark_tiles(c)
    for n in range(60):
        b = 3 * n
        plant(c, b, 0, 128 + 5 + n, 0.6)
        plant(c, b + 1, 1, 4 * 128 + 2 * n, 0.5)
        plant(c, b + 1, 1, 5 * 128 + 127 - n, 1.0)
        plant(c, b + 2, 0, 9 * 128 + n, 0.8)
        plant(c, b, 0, 9 * 128 + 64 + n, 1.2)
    ws = sv.alloc_workspace(256 << 20, DEV)
    out = c.run(checked=True, workspace=ws)
    assert sv.verify_status(ws) == 0
    compare(c, out)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("pre", [2048, 30016])
def test_maxima_of_all_rows_grow_tile_by_tile(kv, pre):
    # keys that grow from page to page; 30,016 tokens are cut into runs that
    # each begin with a maximum of their own
    c = Case([5], [pre], [20] * 5, seed=10, page=64, kv=kv)
    n = pre // 64
    grow = (6.2 / n) * torch.arange(n, device=DEV)
    ids = c.table[0, :n].long()
    x = c.k if kv == "bf16" else c.ks
    x[ids] = (x[ids].float() * grow[:, None, None, None]).to(x.dtype)
    compare(c, c.run())
