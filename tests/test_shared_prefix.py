"""Verify attention of requests that share cached prefixes: the CUDA path
against the definition in 64 bits, and the calls that are refused.

Tolerances, from the roundings.  With w the softmax weights of a row,
A = sum_t w_t |v_t| per channel and X = max_t scale sum_c |q_c k_tc|:
  bf16 KV   the weights of shared tokens are rounded to bf16, 2^-8 each: 2^-8 A;
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
    """Groups of requests over one pool.  `sizes` requests per group, `pre`
    shared tokens (whole pages of them are shared, the rest of the prefix is
    copied), `tails` own tokens and `widths` block rows per request."""

    def __init__(self, sizes, pre, tails, *, q_len=8, widths=None, page=16,
                 kv="bf16", hq=24, hkv=4, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv, self.page, self.q_len = kv, page, q_len
        self.hq, self.hkv = hq, hkv
        B = self.B = sum(sizes)
        self.widths = widths or [q_len] * B
        owner = [n for n, s in enumerate(sizes) for _ in range(s)]
        self.seqs = [pre[o] + t + w
                     for o, t, w in zip(owner, tails, self.widths)]
        cols = max(1, max(-(-s // page) for s in self.seqs))
        whole = [p // page for p in pre]
        need = [max(0, -(-s // page) - whole[o])
                for s, o in zip(self.seqs, owner)]
        pages = self.pages = sum(whole) + sum(need) + 3
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(
            seed)).to(torch.int32)
        table = torch.full((B, cols), 1 << 28, dtype=torch.int32)
        at, front = 0, []
        for w in whole:
            front.append(perm[at:at + w])
            at += w
        for b, o in enumerate(owner):
            table[b, :whole[o]] = front[o]
            table[b, whole[o]:whole[o] + need[b]] = perm[at:at + need[b]]
            at += need[b]
        self.table = table.to(DEV)
        self.seq = torch.tensor(self.seqs, dtype=torch.int32, device=DEV)
        self.q_lens = (None if widths is None else torch.tensor(
            widths, dtype=torch.int32, device=DEV))
        starts = [0]
        for s in sizes:
            starts.append(starts[-1] + s)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.shared = torch.tensor([w * page for w in whole],
                                   dtype=torch.int32, device=DEV)
        self.q = torch.randn((B, q_len, hq, D), generator=g,
                             device=DEV).to(torch.bfloat16)
        # every cached slot holds data, every other one NaN
        used = torch.zeros((pages, page), dtype=torch.bool)
        for b, s in enumerate(self.seqs):
            t = torch.arange(s)
            used[table[b, t // page].long(), t % page] = True
        used = used.to(DEV)[:, None, :, None]
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
        a = dict(starts=self.starts, shared=self.shared)
        a.update({k: kw.pop(k) for k in list(kw) if k in a})
        return sv.verify_attention_shared(
            self.q, self.k, self.v, self.table, self.seq, a["starts"],
            a["shared"], scale=self.scale, k_scales=self.ks,
            v_scales=self.vs, q_lens=self.q_lens, **kw)

    def dense(self, pages, scales, b, n):
        ids = self.table[b, :-(-n // self.page)].long()
        x = pages[ids]
        if scales is not None:
            x = x.view(torch.float8_e4m3fn).double()
            x = x * scales[ids].double().repeat_interleave(64, -1)
        return x.double().transpose(0, 1).reshape(self.hkv, -1, D)[:, :n]

    def check(self, out):
        assert torch.isfinite(out.float()).all()
        G = self.hq // self.hkv
        for b in range(self.B):
            w, n = self.widths[b], self.seqs[b]
            if w:
                k, v = (self.dense(p, s, b, n) for p, s in
                        ((self.k, self.ks), (self.v, self.vs)))
            for i in range(self.q_len):
                got = out[b, i].double().view(self.hkv, G, D)
                m = n - w + i + 1
                if i >= w or m <= 0:
                    assert not got.any()
                    continue
                q = self.q[b, i].double().view(self.hkv, G, D)
                p = torch.softmax(torch.einsum(
                    "hgd,htd->hgt", q, k[:, :m]) * self.scale, -1)
                o = torch.einsum("hgt,htd->hgd", p, v[:, :m])
                A = torch.einsum("hgt,htd->hgd", p, v[:, :m].abs())
                X = (torch.einsum("hgd,htd->hgt", q.abs(), k[:, :m].abs())
                     * self.scale).amax(-1, keepdim=True)
                per = (2.0 ** -8 if self.kv == "bf16"
                       else 2.0 ** -10 + 2.0 ** -10 * X)
                tol = (per + 2.0 ** -13 + 2.0 ** -18 * X) * A \
                    + 2.0 ** -8 * o.abs()
                err = (got - o).abs()
                assert bool((err <= tol).all()), (
                    b, i, float((err / tol).max()))


gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("page", [8, 16, 64, 128])
def test_one_group(kv, page):
    c = Case([3], [1000], [5, 300, 64], page=page, kv=kv, seed=page)
    c.check(c.run())


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("q_len", [1, 5, 16])
def test_row_counts(kv, q_len):
    # rows of a KV head: 2 .. 13 requests x q_len x 6, over and under one,
    # two and several tiles of 256 rows; FP8 blocks on either side of 64 rows
    c = Case([13, 2], [700, 300], [40 + 3 * b for b in range(15)],
             q_len=q_len, kv=kv, seed=q_len)
    c.check(c.run())


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_groups_widths_and_idle_requests(kv):
    sizes = [1, 4, 2, 3, 2]
    pre = [500, 1111, 127, 2000, 640]
    widths = [8, 3, 0, 8, 1, 8, 8, 0, 0, 5, 2, 7]
    tails = [0, 30, 5, 0, 700, 64, 2, 9, 9, 400, 1, 0]
    c = Case(sizes, pre, tails, widths=widths, kv=kv, seed=3)
    ws = sv.alloc_workspace(64 << 20, DEV)
    c.check(c.run(checked=True, workspace=ws))
    assert sv.verify_status(ws) == 0


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_long_prefix_many_pieces(kv):
    # several pieces per CTA pair and several partials per segment
    c = Case([9, 2], [30000, 9000], [100] * 11, q_len=6, page=64, kv=kv,
             seed=11)
    c.check(c.run())


@gpu
def test_other_head_counts():
    for hq, hkv, q_len in ((8, 8, 4), (16, 1, 8), (40, 8, 3)):
        c = Case([4], [777], [3, 9, 27, 81], q_len=q_len, hq=hq, hkv=hkv,
                 page=32, seed=hq)
        c.check(c.run())


@gpu
def test_shared_lengths_are_cut_to_what_all_rows_see():
    c = Case([3], [640], [0, 3, 200], q_len=8, seed=5)
    want = c.run()
    c.check(want)
    # the shortest request's first row sees 640 committed tokens; a longer
    # statement holds for what its table row has in common with the others
    c.table[:2, 40] = c.table[2, 40]            # one more page alike
    for n in (656, 640, 639, 127, 0, -5):
        c.check(c.run(shared=torch.tensor([n], dtype=torch.int32,
                                          device=DEV)))


@gpu
def test_groups_outside_and_bad_borders():
    c = Case([2, 3, 2], [400, 900, 300], [10] * 7, seed=6)
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    # only the middle group is named
    c.check(c.run(starts=t(2, 5), shared=t(896)))
    # empty groups between
    c.check(c.run(starts=t(0, 2, 2, 2, 5, 7), shared=t(400, 9, 9, 896, 288)))
    ws = sv.alloc_workspace(64 << 20, DEV)
    for bad in (t(0, 5, 2, 7), t(-1, 2, 5, 7), t(0, 2, 5, 8)):
        c.check(c.run(starts=bad, checked=True, workspace=ws))
        assert sv.verify_status(ws) == _native.SPEC_STATUS_BAD_GROUPS


@gpu
def test_bad_page_is_reported_and_not_read():
    c = Case([2, 2], [512, 512], [10] * 4, seed=7)
    c.table[0, 3] = c.pages
    c.table[1, 3] = c.pages
    ws = sv.alloc_workspace(64 << 20, DEV)
    out = c.run(checked=True, workspace=ws)
    assert sv.verify_status(ws) & _native.SPEC_STATUS_BAD_PAGE
    good = Case([2, 2], [512, 512], [10] * 4, seed=7)
    ref = good.run()
    assert torch.equal(out[2:], ref[2:])


@gpu
def test_equal_to_verify_attention_without_sharing():
    # groups of one: the tails hold everything, on the ordinary kernels
    c = Case([1, 1, 1], [900, 40, 3000], [10, 20, 30], page=64, seed=8)
    out = c.run()
    ref = sv.verify_attention(c.q, c.k, c.v, c.table, c.seq, scale=c.scale)
    err = (out.double() - ref.double()).abs()
    assert bool((err <= 2.0 ** -7 * ref.double().abs() + 1e-6).all())
    c.check(out)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_captured_graph_streams_and_repeats(kv):
    c = Case([4, 3], [2000, 1000], [50] * 7, kv=kv, page=64, seed=9)
    first = c.run()
    c.check(first)
    # the same inputs give the same bits: no atomics in the sums
    for _ in range(3):
        assert torch.equal(c.run(), first)
    desc = _native.make_desc(batch=c.B, q_len=c.q_len, num_q_heads=24,
                             num_kv_heads=4, head_dim=256, page_size=64,
                             num_pages=c.pages,
                             max_pages_per_seq=c.table.shape[1], kv_dtype=(
                                 "bf16" if kv == "bf16" else "fp8"))
    ws = sv.alloc_workspace(sv.shared_workspace_size(desc, 2), DEV)
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    shared = c.shared.clone()
    with torch.cuda.graph(g):
        c.run(out=out, workspace=ws, shared=shared)
    g.replay()
    assert torch.equal(out, first)
    shared.copy_(torch.tensor([0, 500]))       # read at replay
    g.replay()
    c.check(out)
    # two streams at once, a workspace each
    ws2 = torch.empty_like(ws)
    o1, o2 = torch.empty_like(first), torch.empty_like(first)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        c.run(out=o1, workspace=ws, stream=s1)
        c.run(out=o2, workspace=ws2, stream=s2)
    for s in (s1, s2):
        torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o1, first) and torch.equal(o2, first)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_many_calls_in_a_row(kv):
    # the pipelines of both CTAs of a pair under load: no wait runs out, and
    # every call gives the same bits
    c = Case([40], [20000], [100 + b for b in range(40)], q_len=1, page=64,
             kv=kv, seed=13)
    ws = sv.alloc_workspace(160 << 20, DEV)
    first = c.run(checked=True, workspace=ws)
    outs = [torch.empty_like(first) for _ in range(150)]
    for o in outs:
        c.run(out=o, workspace=ws)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    for _ in range(20):
        c.run(checked=True, workspace=ws)
        assert sv.verify_status(ws) == 0
    c.check(first)


@gpu
def test_own_buffers_belong_to_the_call_s_stream(monkeypatch):
    # a workspace dropped while its stream is still busy must not come back
    # from the allocator of the current stream
    build.build()
    B, ps = 4, 64
    q = torch.randn((B, 1, 24, 256), device=DEV).to(torch.bfloat16)
    pool = torch.randn((24, 4, ps, 256), device=DEV).to(torch.bfloat16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).repeat(B, 1)
    args = (q, pool, pool, table, i(500, 480, 512, 490), i(0, B), i(448))
    want = sv.verify_attention_shared(*args, scale=0.06)
    sizes, plain = [], _native.alloc_workspace

    def recorded(n, device):
        w = plain(n, device)
        sizes.append((n, w.data_ptr()))
        return w
    monkeypatch.setattr(_native, "alloc_workspace", recorded)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    out = sv.verify_attention_shared(*args, scale=0.06, stream=s)
    (n, at), = sizes
    again = [plain(n, DEV) for _ in range(3)]
    assert all(w.data_ptr() != at for w in again)
    s.synchronize()
    assert torch.equal(out, want)


@gpu
def test_large_scores_rescale():
    # keys that grow along the prefix, so the running maximum moves by far
    # more than the threshold, and one that dominates late
    c = Case([5], [2048], [20] * 5, seed=10, page=64)
    k = c.k.float()
    ids = c.table[0, :32].long()
    for n, pg in enumerate(ids.tolist()):
        k[pg] *= 0.2 * n
    c.k = k.to(torch.bfloat16)
    c.check(c.run())


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_short_wait_bound_reports_timeout_and_the_next_call_is_right(kv):
    c = Case([6, 3], [9000, 4000], [100] * 9, kv=kv, page=64, seed=12)
    ws = sv.alloc_workspace(128 << 20, DEV)
    build.build()
    sv.set_wait_limit(200)  # SM clock cycles: the first waits run out
    try:
        c.run(checked=True, workspace=ws)
        torch.cuda.synchronize()
    finally:
        sv.set_wait_limit(0)
    assert sv.verify_status(ws) & _native.SPEC_STATUS_TIMEOUT
    c.check(c.run(checked=True, workspace=ws))
    assert sv.verify_status(ws) == 0


# ---------------------------------------------------------------- CPU tests

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: checks come first
ODD = ctypes.c_void_p(0x100002)


def _raw(desc=None, groups=1, starts=FAKE, shared=FAKE, q=FAKE, ws=FAKE,
         ws_bytes=1 << 40, scale=0.0625, **kw):
    build.build()
    lib = _native.load()
    base = dict(batch=2, q_len=8, num_q_heads=24, num_kv_heads=4,
                head_dim=256, page_size=16, num_pages=64,
                max_pages_per_seq=8)
    base.update(kw)
    d = desc or _native.make_desc(**base)
    return lib.spec_verify_attention_shared(
        ctypes.byref(d), q, FAKE, FAKE, None, None, FAKE, FAKE, groups,
        starts, shared, scale, FAKE, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(groups=0), _native.SPEC_ERR_ARG),
    (dict(groups=1025), _native.SPEC_ERR_ARG),
    (dict(page_size=4), _native.SPEC_ERR_UNSUPPORTED),
    (dict(head_dim=128), _native.SPEC_ERR_UNSUPPORTED),
    (dict(q_len=17), _native.SPEC_ERR_ARG),
    (dict(q=None), _native.SPEC_ERR_ARG),
    (dict(starts=None), _native.SPEC_ERR_ARG),
    (dict(shared=None), _native.SPEC_ERR_ARG),
    (dict(starts=ODD), _native.SPEC_ERR_ALIGN),
    (dict(shared=ODD), _native.SPEC_ERR_ALIGN),
    (dict(scale=0.0), _native.SPEC_ERR_ARG),
    (dict(kv_dtype="fp8"), _native.SPEC_ERR_ARG),
])
def test_refusals(kw, code):
    assert _raw(**kw) == code
    assert _native.load().spec_last_error()


def test_empty_batch_is_a_noop():
    assert _raw(batch=0, q=None) == _native.SPEC_OK


def test_binding_refuses_wrong_tensors():
    q = torch.zeros((2, 8, 24, 256), dtype=torch.bfloat16)
    pool = torch.zeros((4, 4, 16, 256), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(q=q, k=pool, v=pool, t=i(2, 2), s=i(2), st=i(2), sh=i(1))

    def refused(**kw):
        a = {**good, **kw}
        with pytest.raises(sv.SpecError):
            sv.verify_attention_shared(a["q"], a["k"], a["v"], a["t"], a["s"],
                                       a["st"], a["sh"], scale=0.1)
    refused(q=q.float())
    refused(q=q.transpose(0, 1))
    refused(k=pool[:, ::2])
    refused(v=pool[:2])
    refused(t=i(3, 2))
    refused(s=i(3))
    refused(st=i(3))
    refused(sh=torch.zeros(1, dtype=torch.int64))
    refused()                                   # host tensors
