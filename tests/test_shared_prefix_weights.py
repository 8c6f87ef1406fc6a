"""Verify attention with shared prefixes where most of a row's weights are
small: each shared token has to count with its own share.

Tolerances are those of test_shared_prefix.py.  FP8 KV adds what fp16 does to
the smallest weights: they carry a factor of 2^11, so one below 2^-25 of the
largest is off by half of fp16's last step, 2^-25 2^-11 = 2^-36 of the largest
weight: 2^-36 max(w) sum_t |v_t|."""
import pytest
import torch

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
