"""Rotary positions with the paged append: the CUDA path against the formula
in 64 bits, the calls that are refused, and the frequency tables.

Tolerances.  A rotated value m (x cos a - y sin a) is computed in fp32.  The
angle is off by its conversion to fp32, pi 2^-24, and by t (f / 2 pi) 2^-52
turns, 2.4e-7 radians at t = 2^30; sincospi by 2 ulp, 1.2e-7; m and the two
products round four times, 2.4e-7: together below 1e-6 m (|x| + |y|).  A bf16 result adds half
a step, 2^-8 of its value; an E4M3 code half a step of the code, 2^-4 of its
value or 2^-10 below the smallest normal; a scale half an fp16 step, 2^-11 of
its value or 2^-25."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_target_gb300 as sv
from speculative_decoding_target_gb300 import _native, build
from speculative_decoding_target_gb300 import workloads as wl

DEV = "cuda"
ARITH = 1e-6


# ------------------------------------------------------------ plain formula

def rotate64(x, pos, freq, interleaved, m):
    """[.., H, 256] float64, pos [..]: every head's leading pairs turned."""
    x = x.astype(np.float64).copy()
    n = 2 * len(freq)
    # the exact fraction of a turn first, so that sin and cos see small angles
    turns = np.asarray(freq, np.longdouble) / (2 * np.longdouble(math.pi)
                                               + np.longdouble(1.2246467991473531772e-16) * 2)
    frac = pos[..., None].astype(np.longdouble) * turns
    a = (2 * np.pi * (frac - np.floor(frac))).astype(np.float64)[..., None, :]
    c, s = np.cos(a) * m, np.sin(a) * m
    r = x[..., :n]
    if interleaved:
        u, v = r[..., 0::2].copy(), r[..., 1::2].copy()
        r[..., 0::2], r[..., 1::2] = u * c - v * s, v * c + u * s
        size = np.repeat(np.abs(u) + np.abs(v), 2, -1)
    else:
        u, v = r[..., :n // 2].copy(), r[..., n // 2:].copy()
        r[..., :n // 2], r[..., n // 2:] = u * c - v * s, v * c + u * s
        size = np.concatenate([np.abs(u) + np.abs(v)] * 2, -1)
    err = np.zeros_like(x)
    err[..., :n] = ARITH * abs(m) * size
    return x, err


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make_case(kv, page, widths, seqs, q_len, *, hq=24, hkv=4, seed=0,
              fused=False, pages_extra=3, cols=None):
    g = torch.Generator(device="cpu").manual_seed(seed)
    B = len(seqs)
    if fused:
        qkv = torch.randn((B, q_len, (hq + 2 * hkv) * 256 + 64),
                          generator=g).to(torch.bfloat16).to(DEV)
        q = qkv[..., :hq * 256].view(B, q_len, hq, 256)
        k = qkv[..., hq * 256:(hq + hkv) * 256].view(B, q_len, hkv, 256)
        v = qkv[..., (hq + hkv) * 256:(hq + 2 * hkv) * 256].view(
            B, q_len, hkv, 256)
    else:
        q, k, v = (torch.randn((B, q_len, h, 256), generator=g).to(
            torch.bfloat16).to(DEV) for h in (hq, hkv, hkv))
    cols = cols or max(1, -(-max(seqs) // page))
    used = sum(-(-max(s, 0) // page) for s in seqs)
    pages = used + pages_extra
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, cols), 1 << 28, dtype=torch.int32)  # no page
    at = 0
    for b, s in enumerate(seqs):
        n = min(cols, -(-max(s, 0) // page))
        table[b, :n] = perm[at:at + n]
        at += n
    if kv == "fp8":
        pool = lambda: torch.full((pages, hkv, page, 256), 0x7F,
                                  dtype=torch.uint8, device=DEV)
        scl = lambda: torch.full((pages, hkv, page, 4), float("nan"),
                                 dtype=torch.float16, device=DEV)
        kp, vp, ks, vs = pool(), pool(), scl(), scl()
    else:
        pool = lambda: torch.full((pages, hkv, page, 256), float("nan"),
                                  dtype=torch.bfloat16, device=DEV)
        kp, vp, ks, vs = pool(), pool(), None, None
    return dict(q=q, k=k, v=v, kp=kp, vp=vp, ks=ks, vs=vs,
                table=table.to(DEV), pages=pages,
                seq=torch.tensor(seqs, dtype=torch.int32, device=DEV),
                q_lens=(None if widths is None else
                        torch.tensor(widths, dtype=torch.int32, device=DEV)),
                page=page, q_len=q_len, kv=kv)


def call(c, freq, interleaved, m, **kw):
    B = c["k"].shape[0]
    c["pos"] = torch.full((B, c["q_len"]), -7, dtype=torch.int32, device=DEV)
    c["loc"] = torch.full((B, c["q_len"]), -7, dtype=torch.int64, device=DEV)
    kw.setdefault("positions", c["pos"])
    kw.setdefault("cache_loc", c["loc"])
    return sv.rope_append(
        c["q"], c["k"], c["v"], torch.as_tensor(freq, dtype=torch.float64,
                                                device=DEV),
        c["kp"], c["vp"], c["table"], c["seq"], interleaved=interleaved,
        attn_factor=m, k_scales=c["ks"], v_scales=c["vs"],
        q_lens=c["q_lens"], **kw)


def check(c, q_out, freq, interleaved, m):
    B, q_len, page = c["k"].shape[0], c["q_len"], c["page"]
    seq = c["seq"].cpu().numpy()
    table = c["table"].cpu().numpy()
    widths = (np.full(B, q_len) if c["q_lens"] is None
              else np.clip(c["q_lens"].cpu().numpy(), 0, q_len))
    pos = seq[:, None] - widths[:, None] + np.arange(q_len)[None]
    live = (np.arange(q_len)[None] < widths[:, None]) & (pos >= 0)
    kq, kqe = rotate64(f64(c["q"]), pos, freq, interleaved, m)
    kk, kke = rotate64(f64(c["k"]), pos, freq, interleaved, m)
    got = f64(q_out)
    want = np.where(live[..., None, None], kq, 0.0)
    tol = np.where(live[..., None, None],
                   np.abs(kq) * 2.0 ** -8 + kqe, 0.0)
    assert np.all(np.abs(got - want) <= tol)
    assert np.array_equal(c["pos"].cpu().numpy(), np.where(live, pos, -1))
    loc = np.full((B, q_len), -1, np.int64)
    written = np.zeros((c["pages"], page), bool)
    kp, vp = c["kp"].cpu(), c["vp"].cpu()
    v_in = f64(c["v"])
    for b in range(B):
        for i in range(q_len):
            t = pos[b, i]
            if not live[b, i] or t >= table.shape[1] * page:
                continue
            pg = table[b, t // page]
            if not 0 <= pg < c["pages"]:
                continue
            loc[b, i] = int(pg) * page + t % page
            written[pg, t % page] = True
            at = (int(pg), slice(None), int(t % page))
            if c["kv"] == "bf16":
                assert np.all(np.abs(f64(kp[at]) - kk[b, i])
                              <= np.abs(kk[b, i]) * 2.0 ** -8 + kke[b, i])
                assert np.array_equal(f64(vp[at]), v_in[b, i])
                continue
            for pool, scl, x, e in ((kp, c["ks"], kk[b, i], kke[b, i]),
                                    (vp, c["vs"], v_in[b, i],
                                     np.zeros_like(v_in[b, i]))):
                sc = f64(scl[at])                             # [H, 4]
                xb = x.reshape(x.shape[0], 4, 64)
                eb = e.reshape(xb.shape)
                true = np.abs(xb).max(-1) / 448
                one = (sc == 1) & (true <= 2.0 ** -25 * 1.01)
                assert np.all(one | (np.abs(sc - true) <= true * 2.0 ** -11
                                     + eb.max(-1) / 448 + 2.0 ** -25))
                codes = f64(pool[at].view(torch.float8_e4m3fn)).reshape(
                    xb.shape)
                y = np.clip(xb / sc[..., None], -448, 448)
                assert np.all(np.abs(codes - y) <= np.maximum(
                    np.abs(y) * 2.0 ** -4, 2.0 ** -10)
                    + eb / sc[..., None] + 448 * 2.0 ** -23)
    assert np.array_equal(c["loc"].cpu().numpy(), loc)
    # every slot that no row went to is as it was (NaN)
    w = torch.from_numpy(written)
    for pool in (kp, vp):
        rest = pool.transpose(1, 2)[~w]
        if c["kv"] == "bf16":
            assert torch.isnan(rest.float()).all()
        else:
            assert (rest == 0x7F).all()


# ---------------------------------------------------------------- GPU tests

@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("rotary,page", [(8, 1), (64, 16), (96, 8), (200, 64),
                                         (256, 128)])
def test_layouts_and_sizes(interleaved, kv, rotary, page):
    build.build()
    freq, m = sv.rope_frequencies(rotary, base=1e6, scaling="yarn",
                                  factor=4.0, original_context=4096)
    c = make_case(kv, page, [8, 0, 3, 8], [8, 40, 1000, 77], 8, seed=rotary)
    check(c, call(c, freq, interleaved, m), freq.numpy(), interleaved, m)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("q_len,widths,seqs", [
    (1, None, [1, 2, 65]), (33, [33, 1, 20], [33, 4, 5000]),
    (300, [300, 299, 0], [300, 811, 64])])
def test_lengths_and_strided_inputs(kv, q_len, widths, seqs):
    build.build()
    freq, m = sv.rope_frequencies(128)
    c = make_case(kv, 16, widths, seqs, q_len, seed=q_len, fused=True)
    check(c, call(c, freq, False, m), freq.numpy(), False, m)


@pytest.mark.gpu
def test_many_tokens_and_other_head_counts():
    build.build()
    freq, m = sv.rope_frequencies(64, scaling="linear", factor=8.0)
    # more tokens than resident CTAs; one KV head; query heads beyond one
    # round of the warps; rows left after a whole round
    c = make_case("bf16", 64, None, [2500, 700], 700, hq=41, hkv=1, seed=4)
    check(c, call(c, freq, True, m), freq.numpy(), True, m)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    build.build()
    freq, m = sv.rope_frequencies(256, base=10000.0)
    page, cols = 4096, 1 << 18
    for t in (1 << 20, (1 << 30) - 8):
        c = make_case("bf16", page, None, [8], 8, hq=2, hkv=1, cols=cols)
        c["seq"].fill_(t + 8)
        c["table"][0, t // page] = 1
        c["table"][0, (t + 7) // page] = 2
        check(c, call(c, freq, interleaved, m), freq.numpy(), interleaved, m)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_no_rotation_equals_plain_append(kv):
    build.build()
    c = make_case(kv, 16, [5, 2, 8], [100, 3, 64], 8, seed=9)
    freq = np.zeros(32)
    got = call(c, freq, False, 1.0)
    bits = wl.to_numpy_bits
    fp8 = kv == "fp8"
    fresh = make_case(kv, 16, [5, 2, 8], [100, 3, 64], 8, seed=9)
    want = oracle.kv_append(
        bits(c["k"]), bits(c["v"]), bits(fresh["kp"]), bits(fresh["vp"]),
        c["table"].cpu().numpy(), c["seq"].cpu().numpy(),
        k_scales=bits(fresh["ks"]) if fp8 else None,
        v_scales=bits(fresh["vs"]) if fp8 else None,
        q_lens=c["q_lens"].cpu().numpy())
    assert np.array_equal(bits(c["kp"]), want[0])
    assert np.array_equal(bits(c["vp"]), want[1])
    if fp8:
        assert np.array_equal(bits(c["ks"]), want[2])
        assert np.array_equal(bits(c["vs"]), want[3])
    assert np.array_equal(c["pos"].cpu().numpy(), want[4])
    assert np.array_equal(c["loc"].cpu().numpy(), want[5])
    w = c["q_lens"].cpu().numpy()
    for b in range(3):
        assert torch.equal(got[b, :w[b]], c["q"][b, :w[b]])
        assert not got[b, w[b]:].any()


@pytest.mark.gpu
def test_rows_without_a_slot_and_bad_pages():
    build.build()
    freq, m = sv.rope_frequencies(64)
    # a block longer than the cache, a table that ends inside the block, a
    # page id outside the pool
    c = make_case("bf16", 16, None, [5, 40, 64], 8, cols=4)
    c["seq"][1] = 68
    c["table"][1, 3] = 0
    c["table"][2, 3] = c["pages"]
    free = [p for p in range(c["pages"]) if p not in c["table"].cpu()]
    c["table"][1, 3] = free[0]
    ws = sv.alloc_workspace(256, DEV)
    check(c, call(c, freq, False, m, checked=True, workspace=ws),
          freq.numpy(), False, m)
    assert sv.verify_status(ws) == _native.SPEC_STATUS_BAD_PAGE


@pytest.mark.gpu
def test_in_place_keys_only_stream_and_graph():
    build.build()
    freq, m = sv.rope_frequencies(64)
    fd = freq.to(DEV)
    c = make_case("fp8", 16, [8, 3], [30, 19], 8, seed=2)
    want = call(c, freq, False, m)
    codes = c["kp"].clone()
    kept = c["q"].clone()
    c["q"] = kept.clone()
    got = call(c, freq, False, m, q_out=c["q"])        # in place
    assert got.data_ptr() == c["q"].data_ptr() and torch.equal(got, want)
    # keys and values alone, on another stream
    c["kp"].fill_(0x7F)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert sv.rope_append(None, c["k"], c["v"], fd, c["kp"], c["vp"],
                              c["table"], c["seq"], k_scales=c["ks"],
                              v_scales=c["vs"], q_lens=c["q_lens"]) is None
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(c["kp"], codes)
    # captured: the lengths move between replays
    c["q"] = kept.clone()
    out = torch.empty_like(kept)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call_kw = dict(q_out=out, positions=None, cache_loc=None)
        sv.rope_append(c["q"], c["k"], c["v"], fd, c["kp"], c["vp"],
                       c["table"], c["seq"], k_scales=c["ks"],
                       v_scales=c["vs"], q_lens=c["q_lens"], **call_kw)
    g.replay()
    assert torch.equal(out, want)
    c["seq"].copy_(torch.tensor([31, 12]))
    g.replay()
    again = call(c, freq, False, m)
    assert torch.equal(out, again) and not torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 3])
def test_as_many_rows_as_a_call_allows(batch):
    # keys and values of a block padded to the largest batch * q_len, through
    # strides of 0; the rows behind each width hold no token
    build.build()
    q_len = (2 ** 31 - 1) // batch
    g = torch.Generator(device=DEV).manual_seed(4)
    k, v = (torch.randn((1, 1, 1, 256), generator=g, device=DEV).to(
        torch.bfloat16) for _ in range(2))
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    widths, seqs = [5, 0, 3][:batch], [5, 7, 20][:batch]
    table = torch.arange(2 * batch, dtype=torch.int32, device=DEV).view(
        batch, 2)
    freq = sv.rope_frequencies(64, device=DEV)[0]
    pools = []
    for n in (8, q_len):
        kp, vp = (torch.zeros((2 * batch, 1, 16, 256), dtype=torch.bfloat16,
                              device=DEV) for _ in range(2))
        assert sv.rope_append(
            None, k.expand(batch, n, 1, 256), v.expand(batch, n, 1, 256), freq,
            kp, vp, table, i32(*seqs), q_lens=i32(*widths)) is None
        torch.cuda.synchronize()
        pools.append((kp, vp))
    assert torch.equal(pools[0][0], pools[1][0])
    assert torch.equal(pools[0][1], pools[1][1])
    assert int(pools[0][1].abs().amax(-1).count_nonzero()) == sum(widths)


# ---------------------------------------------------------------- CPU tests

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: checks come first


def _raw(lib, **kw):
    d = _native.RopeDesc(2, 8, 24, 4, 256, 16, 64, 8, 0, 0, None, 64, 0, 1.0)
    ptr = dict(q=FAKE, k=FAKE, v=FAKE, freq=FAKE, out=FAKE, kp=FAKE, vp=FAKE,
               ks=None, vs=None, table=FAKE, seq=FAKE, pos=None, loc=None,
               ws=None)
    for name, val in kw.items():
        if name in ptr:
            ptr[name] = val
        elif name.endswith("_strides"):
            setattr(d, name, (ctypes.c_int64 * 2)(*val))
        else:
            setattr(d, name, val)
    return lib.spec_rope_append(ctypes.byref(d), *ptr.values(), None)


ODD = ctypes.c_void_p(0x100008)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), _native.SPEC_ERR_ARG),
    (dict(q_len=0), _native.SPEC_ERR_ARG),
    (dict(batch=1 << 16, q_len=1 << 15), _native.SPEC_ERR_ARG),
    (dict(num_kv_heads=0), _native.SPEC_ERR_ARG),
    (dict(head_dim=128), _native.SPEC_ERR_UNSUPPORTED),
    (dict(page_size=24), _native.SPEC_ERR_ARG),
    (dict(page_size=4096, max_pages_per_seq=(1 << 18) + 1),
     _native.SPEC_ERR_ARG),
    (dict(num_pages=0), _native.SPEC_ERR_ARG),
    (dict(kv_dtype=2), _native.SPEC_ERR_ARG),
    (dict(flags=2), _native.SPEC_ERR_ARG),
    (dict(rotary_dim=0), _native.SPEC_ERR_ARG),
    (dict(rotary_dim=12), _native.SPEC_ERR_ARG),
    (dict(rotary_dim=264), _native.SPEC_ERR_ARG),
    (dict(interleaved=2), _native.SPEC_ERR_ARG),
    (dict(attn_factor=float("nan")), _native.SPEC_ERR_ARG),
    (dict(q_strides=(0, 4)), _native.SPEC_ERR_ARG),
    (dict(v_strides=(-8, 8)), _native.SPEC_ERR_ARG),
    (dict(k=None), _native.SPEC_ERR_ARG),
    (dict(freq=None), _native.SPEC_ERR_ARG),
    (dict(q=None), _native.SPEC_ERR_ARG),
    (dict(num_q_heads=0), _native.SPEC_ERR_ARG),
    (dict(q=ODD), _native.SPEC_ERR_ALIGN),
    (dict(out=ODD), _native.SPEC_ERR_ALIGN),
    (dict(freq=ctypes.c_void_p(0x100004)), _native.SPEC_ERR_ALIGN),
    (dict(loc=ctypes.c_void_p(0x100004)), _native.SPEC_ERR_ALIGN),
    (dict(kv_dtype=1), _native.SPEC_ERR_ARG),
    (dict(kv_dtype=1, ks=FAKE, vs=ODD), _native.SPEC_ERR_ALIGN),
    (dict(flags=1), _native.SPEC_ERR_WORKSPACE),
])
def test_refusals(kw, code):
    build.build()
    lib = _native.load()
    assert _raw(lib, **kw) == code
    assert lib.spec_last_error()


def test_empty_batch_is_a_noop():
    build.build()
    assert _raw(_native.load(), batch=0, k=None) == _native.SPEC_OK


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((2, 8, 4, 256), dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    pool = torch.zeros((4, 4, 16, 256), dtype=torch.bfloat16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    seq = torch.zeros(2, dtype=torch.int32)
    good = dict(q=x, k=x, v=x, f=f, kp=pool, vp=pool, t=table, s=seq)

    def refused(**kw):
        a = {**good, **kw}
        with pytest.raises(sv.SpecError):
            sv.rope_append(a["q"], a["k"], a["v"], a["f"], a["kp"], a["vp"],
                           a["t"], a["s"])
    refused(k=x.float())
    refused(v=x[:, :, :2])
    refused(q=x.transpose(1, 2))
    refused(f=f.float())
    refused(f=torch.zeros(64, dtype=torch.float64)[::2])
    refused(t=table.t())
    refused(s=seq.long())
    refused(kp=pool[:, :2])
    refused(vp=pool.half())
    refused()                                   # host tensors
    for kw, what in ((dict(t=table[:1]), "rows"), (dict(t=table[0]), "rows"),
                     (dict(f=f.view(4, 8)), "freq")):
        a = {**good, **kw}
        with pytest.raises(sv.SpecError, match=what):
            sv.rope_append(x, x, x, a["f"], pool, pool, a["t"], seq)
    with pytest.raises(sv.SpecError, match="4 bytes"):
        sv.rope_append(x, x, x, f, pool, pool, table, seq, checked=True,
                       workspace=torch.zeros(3, dtype=torch.uint8))


def test_frequencies():
    f, m = sv.rope_frequencies(64, base=1e6)
    j = np.arange(32)
    assert m == 1.0 and f.dtype == torch.float64
    assert np.allclose(f.numpy(), 1e6 ** (-2 * j / 64), rtol=1e-15)
    lin, _ = sv.rope_frequencies(64, base=1e6, scaling="linear", factor=4.0)
    assert np.allclose(lin.numpy() * 4, f.numpy(), rtol=1e-15)
    ntk, _ = sv.rope_frequencies(64, base=1e6, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / 4, rel_tol=1e-12)
    y, m = sv.rope_frequencies(64, base=1e6, scaling="yarn", factor=4.0,
                               original_context=4096)
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    turns = 4096 * f.numpy() / (2 * np.pi)
    assert np.allclose(y.numpy()[turns > 33], f.numpy()[turns > 33])
    assert np.allclose(y.numpy()[turns < 0.6], f.numpy()[turns < 0.6] / 4)
    assert np.all(np.diff(y.numpy()) < 0)
    w, m = sv.rope_frequencies(128, base=5e5, scaling="wavelength",
                               factor=8.0, original_context=8192)
    f = sv.rope_frequencies(128, base=5e5)[0].numpy()
    wave = 2 * np.pi / f
    assert m == 1.0
    assert np.allclose(w.numpy()[wave < 2048], f[wave < 2048])
    assert np.allclose(w.numpy()[wave > 8192], f[wave > 8192] / 8)
    mid = (wave > 2048) & (wave < 8192)
    assert mid.any() and np.all(w.numpy()[mid] < f[mid])
    assert np.all(w.numpy()[mid] > f[mid] / 8)
    for bad in (dict(scaling="other"), dict(rotary_dim=12), dict(factor=0.5),
                dict(base=1.0), dict(original_context=0)):
        kw = {"rotary_dim": 64, **bad}
        with pytest.raises(ValueError):
            sv.rope_frequencies(kw.pop("rotary_dim"), **kw)
    assert sv.rope_frequencies(64, attn_factor=2.5)[1] == 2.5
