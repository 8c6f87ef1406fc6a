"""Head norms with rotary positions and the paged append: the CUDA path against
the formula in 64 bits, and the calls that are refused.

Tolerances.  A normed channel is x rsqrt(ss / 256 + eps) w in fp32.  The sum of
squares of 256 bf16 values (exact squares) takes 8 fused steps and 5 sums, 13
roundings of 2^-24, halved by the root; with the step for eps, the division,
rsqrt's 2 ulp (2^-22), w's sum with its offset and two products: below
(6.5 + 1 + 1 + 4 + 3) 2^-24 = 9.3e-7 of the value, taken as 1e-6.  The rotation adds
1e-6 m (|x| + |y|) (tests/test_rope_append.py) of the normed pair, so a rotated
channel is off by 2e-6 m (|x| + |y|).  Then the store: bf16 2^-8 of the value,
an E4M3 code 2^-4 of its value or 2^-10, a scale 2^-11 of its value or 2^-25."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_target_gb300 as sv
from speculative_decoding_target_gb300 import _native, build
from test_rope_append import FAKE, ODD, f64, make_case, rotate64

DEV = "cuda"
NORM = 1e-6


def normed64(x, w, eps, offset):
    x = x.astype(np.float64)
    return (x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
            * (w.astype(np.float64) + offset))


def expected(x, w, eps, offset, pos, freq, interleaved, m):
    y = normed64(x, w, eps, offset)
    z, e = rotate64(y, pos, freq, interleaved, m)
    n = 2 * len(freq)
    e[..., :n] *= 2                    # the norm's share beside the rotation's
    e[..., n:] = NORM * np.abs(y[..., n:])
    return z, e


def weights(seed, dtype, offset):
    g = torch.Generator().manual_seed(seed)
    w = 1.0 - offset + 0.3 * torch.randn((2, 256), generator=g)
    return w.to(dtype).to(DEV)


def call(c, w, freq, interleaved, m, **kw):
    B = c["k"].shape[0]
    c["pos"] = torch.full((B, c["q_len"]), -7, dtype=torch.int32, device=DEV)
    c["loc"] = torch.full((B, c["q_len"]), -7, dtype=torch.int64, device=DEV)
    kw.setdefault("positions", c["pos"])
    kw.setdefault("cache_loc", c["loc"])
    return sv.norm_rope_append(
        c["q"], c["k"], c["v"], w[0], w[1],
        torch.as_tensor(freq, dtype=torch.float64, device=DEV), c["kp"],
        c["vp"], c["table"], c["seq"], interleaved=interleaved, attn_factor=m,
        k_scales=c["ks"], v_scales=c["vs"], q_lens=c["q_lens"], **kw)


def check(c, q_out, w, freq, interleaved, m, eps=1e-6, offset=0.0):
    B, q_len, page = c["k"].shape[0], c["q_len"], c["page"]
    seq = c["seq"].cpu().numpy()
    table = c["table"].cpu().numpy()
    widths = (np.full(B, q_len) if c["q_lens"] is None
              else np.clip(c["q_lens"].cpu().numpy(), 0, q_len))
    pos = seq[:, None] - widths[:, None] + np.arange(q_len)[None]
    live = (np.arange(q_len)[None] < widths[:, None]) & (pos >= 0)
    wq, wk = f64(w[0]), f64(w[1])
    if q_out is not None:
        want, err = expected(f64(c["q"]), wq, eps, offset, pos, freq,
                             interleaved, m)
        on = live[..., None, None]
        assert np.all(np.abs(f64(q_out) - np.where(on, want, 0.0))
                      <= np.where(on, np.abs(want) * 2.0 ** -8 + err, 0.0))
    kk, kke = expected(f64(c["k"]), wk, eps, offset, pos, freq, interleaved, m)
    v_in = f64(c["v"])
    assert np.array_equal(c["pos"].cpu().numpy(), np.where(live, pos, -1))
    loc = np.full((B, q_len), -1, np.int64)
    written = np.zeros((c["pages"], page), bool)
    kp, vp = c["kp"].cpu(), c["vp"].cpu()
    for b, i in np.argwhere(live):
        t = pos[b, i]
        if t >= table.shape[1] * page:
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
            sc = f64(scl[at])                                 # [H, 4]
            xb = x.reshape(x.shape[0], 4, 64)
            eb = e.reshape(xb.shape)
            true = np.abs(xb).max(-1) / 448
            one = (sc == 1) & (true <= 2.0 ** -25 * 1.01)
            assert np.all(one | (np.abs(sc - true) <= true * 2.0 ** -11
                                 + eb.max(-1) / 448 + 2.0 ** -25))
            codes = f64(pool[at].view(torch.float8_e4m3fn)).reshape(xb.shape)
            y = np.clip(xb / sc[..., None], -448, 448)
            assert np.all(np.abs(codes - y) <= np.maximum(
                np.abs(y) * 2.0 ** -4, 2.0 ** -10)
                + eb / sc[..., None] + 448 * 2.0 ** -23)
    assert np.array_equal(c["loc"].cpu().numpy(), loc)
    on = torch.from_numpy(written)     # every other slot is as it was
    for pool in (kp, vp):
        rest = pool.transpose(1, 2)[~on]
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
    w = weights(rotary, torch.bfloat16, 0.0)
    check(c, call(c, w, freq, interleaved, m), w, freq.numpy(), interleaved, m)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("q_len,widths,seqs", [
    (1, None, [1, 2, 65]), (33, [33, 1, 20], [33, 4, 5000]),
    (300, [300, 299, 0], [300, 811, 64])])
@pytest.mark.parametrize("interleaved", [False, True])
def test_lengths_strides_and_weights(kv, q_len, widths, seqs, interleaved):
    build.build()
    freq, m = sv.rope_frequencies(128)
    c = make_case(kv, 16, widths, seqs, q_len, seed=q_len, fused=True)
    w = weights(3, torch.float32, 1.0)
    check(c, call(c, w, freq, interleaved, m, eps=1e-3, weight_offset=1.0), w,
          freq.numpy(), interleaved, m, 1e-3, 1.0)


@pytest.mark.gpu
def test_many_tokens_and_other_head_counts():
    build.build()
    freq, m = sv.rope_frequencies(64, scaling="linear", factor=8.0)
    w = weights(5, torch.bfloat16, 1.0)
    for hq, hkv, inter in ((41, 1, True), (3, 5, False)):
        c = make_case("bf16", 64, None, [2500, 700], 700, hq=hq, hkv=hkv,
                      seed=4)
        check(c, call(c, w, freq, inter, m, weight_offset=1.0), w,
              freq.numpy(), inter, m, offset=1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv", [(64, 8), (96, 1), (6, 21)])
def test_more_heads_than_a_round_of_warps(kv, hq, hkv):
    build.build()
    freq, m = sv.rope_frequencies(128)
    w = weights(9, torch.float32, 0.0)
    c = make_case(kv, 16, [5, 33, 0], [40, 33, 9], 33, hq=hq, hkv=hkv, seed=8)
    for inter in (False, True):
        check(c, call(c, w, freq, inter, m), w, freq.numpy(), inter, m)


@pytest.mark.gpu
def test_quantised_values_are_rope_append_s():
    # byte for byte: all sizes, borders between codes, zeros of both signs, NaN,
    # infinities, rows whose scale is infinite, one or a subnormal
    build.build()
    freq, m = sv.rope_frequencies(64)
    w = weights(11, torch.bfloat16, 0.0)
    c = make_case("fp8", 16, None, [700, 700], 700, seed=30)
    g = torch.Generator(device=DEV).manual_seed(31)
    v = torch.randn(c["v"].shape, generator=g, device=DEV)
    at = torch.arange(700, device=DEV)[:, None, None]
    v = torch.where(at < 300, v * 2.0 ** (at - 150) / 4, v)
    steps = torch.randint(-448 * 16, 448 * 16, v.shape, generator=g,
                          device=DEV) / 16.0     # on and between codes
    v = torch.where((at >= 300) & (at < 450), steps, v)
    v[:, 450:500] *= 2.0 ** torch.randint(
        -40, 1, v[:, 450:500].shape, generator=g, device=DEV)
    v[:, 500:520, :, ::3] = 0.0
    v[:, 510:530, :, ::5] = -0.0
    v[:, 540, :, 7] = float("nan")
    v[:, 541, :, 9] = float("inf")
    v[:, 542, :, 70] = -float("inf")
    v[:, 543] = 0.0
    v[:, 544:546] = 1e30
    v[:, 546] = -1e-39
    c["v"].copy_(v)
    want = [torch.full_like(c[x], 0) for x in ("kp", "vp", "ks", "vs")]
    got = [t.clone() for t in want]
    sv.rope_append(None, c["k"], c["v"], freq.to(DEV), want[0], want[1],
                   c["table"], c["seq"], k_scales=want[2], v_scales=want[3])
    c["kp"], c["vp"], c["ks"], c["vs"] = got
    for inter in (False, True):
        call(c, w, freq, inter, m)
        assert torch.equal(got[3].view(torch.int16), want[3].view(torch.int16))
        assert torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_addresses_of_16_bytes_and_two_calls_at_once(kv):
    def shifted(t):
        if t is None:
            return None
        n = 16 // t.element_size()
        buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
        buf[n:].copy_(t.reshape(-1))
        return buf[n:].view(t.shape)
    build.build()
    freq, m = sv.rope_frequencies(64)
    w = weights(10, torch.bfloat16, 0.0)
    cases = [make_case(kv, 16, None, [100, 70], 50, seed=20 + k)
             for k in range(2)]
    for c in cases:
        for x in ("q", "k", "v", "kp", "vp", "ks", "vs"):
            c[x] = shifted(c[x])
        c["out"] = shifted(torch.zeros_like(c["q"]))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            call(c, w, freq, False, m, q_out=c["out"], stream=s,
                 positions=None, cache_loc=None)
    torch.cuda.synchronize()
    for c in cases:
        n = c["kp"].clone()
        check(c, call(c, w, freq, False, m, q_out=c["out"]), w, freq.numpy(),
              False, m)
        assert torch.equal(n.view(torch.uint8), c["kp"].view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_small_large_and_zero_heads(kv):
    # rows whose size eps decides, rows of 2^40, rows of zeros; a block longer
    # than its cache, a table that ends inside the block
    build.build()
    freq, m = sv.rope_frequencies(256)
    c = make_case(kv, 16, None, [40, 5, 64], 8, cols=4, seed=6)
    c["seq"][0] = 68
    size = 2.0 ** torch.tensor([-60, -20, -10, 0, 40, 10, 3, -3.],
                               device=DEV)
    for x in ("q", "k"):
        c[x] = (c[x].float() * size[:, None, None]).to(torch.bfloat16)
        c[x][1, 6] = 0
    w = weights(7, torch.bfloat16, 0.0)
    check(c, call(c, w, freq, False, m), w, freq.numpy(), False, m)


@pytest.mark.gpu
def test_bad_page_in_place_keys_only_streams_and_graph():
    build.build()
    freq, m = sv.rope_frequencies(64)
    fd = freq.to(DEV)
    w = weights(8, torch.bfloat16, 0.0)
    c = make_case("fp8", 16, [8, 3], [30, 19], 8, seed=2)
    want = call(c, w, freq, False, m)
    check(c, want, w, freq.numpy(), False, m)
    codes = c["kp"].clone()
    kept = c["q"].clone()
    got = call(c, w, freq, False, m, q_out=c["q"])            # in place
    assert got.data_ptr() == c["q"].data_ptr() and torch.equal(got, want)
    # keys and values alone, on another stream than the current one
    c["kp"].fill_(0x7F)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert sv.norm_rope_append(
        None, c["k"], c["v"], None, w[1], fd, c["kp"], c["vp"], c["table"],
        c["seq"], k_scales=c["ks"], v_scales=c["vs"], q_lens=c["q_lens"],
        stream=s) is None
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(c["kp"], codes)
    # captured: lengths and weights move between replays
    c["q"] = kept.clone()
    out = torch.empty_like(kept)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, w, fd, False, m, q_out=out, positions=None, cache_loc=None)
    g.replay()
    assert torch.equal(out, want)
    c["seq"].copy_(torch.tensor([31, 12]))
    w *= 2
    g.replay()
    again = call(c, w, freq, False, m)
    assert torch.equal(out, again) and not torch.equal(out, want)
    # a page id outside the pool
    c["table"][1, 0] = c["pages"]
    ws = sv.alloc_workspace(256, DEV)
    call(c, w, freq, False, m, checked=True, workspace=ws)
    assert sv.verify_status(ws) == _native.SPEC_STATUS_BAD_PAGE


# ---------------------------------------------------------------- CPU tests

def _raw(lib, norm=True, **kw):
    d = _native.RopeDesc(2, 8, 24, 4, 256, 16, 64, 8, 0, 0, None, 64, 0, 1.0)
    n = _native.NormDesc(1, 1e-6, 0.0, 0x100000, 0x100000)
    ptr = dict(q=FAKE, k=FAKE, v=FAKE, freq=FAKE, out=FAKE, kp=FAKE, vp=FAKE,
               ks=None, vs=None, table=FAKE, seq=FAKE, pos=None, loc=None,
               ws=None)
    for name, val in kw.items():
        if name in ptr:
            ptr[name] = val
        elif name in ("weight_dtype", "eps", "weight_offset", "q_weight",
                      "k_weight"):
            setattr(n, name, val)
        else:
            setattr(d, name, val)
    return lib.spec_norm_rope_append(ctypes.byref(d), ctypes.byref(n)
                                     if norm else None, *ptr.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(norm=False), _native.SPEC_ERR_ARG),
    (dict(weight_dtype=2), _native.SPEC_ERR_ARG),
    (dict(eps=0.0), _native.SPEC_ERR_ARG),
    (dict(eps=1e-40), _native.SPEC_ERR_ARG),
    (dict(eps=float("nan")), _native.SPEC_ERR_ARG),
    (dict(eps=float("inf")), _native.SPEC_ERR_ARG),
    (dict(weight_offset=float("inf")), _native.SPEC_ERR_ARG),
    (dict(k_weight=None), _native.SPEC_ERR_ARG),
    (dict(q_weight=None), _native.SPEC_ERR_ARG),
    (dict(num_q_heads=0, q=None, out=None), _native.SPEC_ERR_ARG),
    (dict(q_weight=0x100002), _native.SPEC_ERR_ALIGN),
    (dict(k_weight=0x100002), _native.SPEC_ERR_ALIGN),
    (dict(batch=-1), _native.SPEC_ERR_ARG),
    (dict(head_dim=128), _native.SPEC_ERR_UNSUPPORTED),
    (dict(rotary_dim=12), _native.SPEC_ERR_ARG),
    (dict(q=ODD), _native.SPEC_ERR_ALIGN),
    (dict(kv_dtype=1), _native.SPEC_ERR_ARG),
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
    w = torch.ones(256)
    pool = torch.zeros((4, 4, 16, 256), dtype=torch.bfloat16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    seq = torch.zeros(2, dtype=torch.int32)

    def refused(q=x, wq=w, wk=w, match="", **kw):
        with pytest.raises(sv.SpecError, match=match):
            sv.norm_rope_append(q, x, x, wq, wk, f, pool, pool, table, seq,
                                **kw)
    refused(wq=None, match="q_weight")
    refused(q=None, match="q_weight")
    refused(wk=None, match="q_weight")
    refused(wk=w.half(), match="bf16 or fp32")
    refused(wq=w.bfloat16(), match="q_weight must be")
    refused(wq=w[:128], match="q_weight must be")
    refused(wk=torch.ones(512)[::2], match="k_weight must be contiguous")
    refused(wk=torch.ones(24, 256), match="k_weight must be")
    refused(match="CUDA device")                # host tensors
