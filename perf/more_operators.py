"""The operators of a prompt's way through the cache, as they are measured.

Three operators that a server calls one after the other for a prompt's pieces
and for the tokens it is asked about:

  norm    RMS norms of every query and key head, their rotary positions, and
          the append of keys and values to the paged cache, in one pass;
  chunk   attention of a piece of new tokens over the paged cache, causal
          within the piece (bf16 cache, or FP8 with scales);
  logp    log probabilities of given tokens, the entropy of their
          distributions and the most likely alternatives.

`own` chooses between the plain forms below (elementary torch operations in
32 bits, 64 where 32 lose what matters) and the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
HQ, HKV, D = 24, 4, 256         # the attention geometry of the benchmark
GROUP = HQ // HKV
VOCAB = 248320


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request's verify block at a short context: launch latency
        dict(name="norm_b1_q8", op="norm", kv="bf16", batch=1, q_len=8,
             prefix=4096, page=16, rotary=64, layout="half", offset=0.0,
             ragged=False),
        # a batch of verify blocks into an FP8 cache, contexts up to 128K
        dict(name="norm_b32_q8_fp8", op="norm", kv="fp8", batch=32, q_len=8,
             prefix=131072, page=64, rotary=64, layout="half", offset=1.0,
             ragged=True),
        # a long prompt in one call, the whole head rotated
        dict(name="norm_prompt_8k", op="norm", kv="bf16", batch=1, q_len=8192,
             prefix=32768, page=64, rotary=256, layout="half", offset=0.0,
             ragged=False),
        # prompt pieces of several requests, padded, quantised on write
        dict(name="norm_prompts_fp8", op="norm", kv="fp8", batch=5,
             q_len=1531, prefix=20000, page=16, rotary=128,
             layout="interleaved", offset=1.0, ragged=True),
        # a user's next message, a few tokens behind a short conversation
        dict(name="chunk_q50_p4k", op="chunk", kv="bf16", batch=1, q_len=50,
             prefix=4096, page=16, ragged=False),
        # a prompt from its start
        dict(name="chunk_q4096_p0", op="chunk", kv="bf16", batch=1,
             q_len=4096, prefix=0, page=64, ragged=False),
        # a piece of a long document
        dict(name="chunk_q2048_p32k", op="chunk", kv="bf16", batch=1,
             q_len=2048, prefix=32768, page=64, ragged=False),
        # pieces of several requests' prompts, different lengths and
        # contexts, some idle, FP8 cache
        dict(name="chunk_b6_ragged_fp8", op="chunk", kv="fp8", batch=6,
             q_len=701, prefix=12000, page=16, ragged=True),
        # the tokens of one request's verify block
        dict(name="logp_r8", op="logp", dtype="fp32", rows=8, vocab=VOCAB,
             top=0, tempered=False, peaks=24, idle=False),
        # a batch's verify blocks with alternatives, temperatures
        dict(name="logp_r256_top5", op="logp", dtype="fp32", rows=256,
             vocab=VOCAB, top=5, tempered=True, peaks=24, idle=True),
        # a prompt's tokens, scored with alternatives
        dict(name="logp_prompt_1k_top20", op="logp", dtype="bf16", rows=1024,
             vocab=VOCAB, top=20, tempered=False, peaks=8, idle=False),
        # an odd vocabulary, few rows, flat distributions
        dict(name="logp_r17_v50001", op="logp", dtype="bf16", rows=17,
             vocab=50001, top=8, tempered=True, peaks=0, idle=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "chunk", "logp"])
    if op == "norm":
        q_len = _log_int(rng, 1, 4096)
        batch = _log_int(rng, 1, max(1, min(64, 8192 // q_len)))
        return dict(op="norm", kv=rng.choice(["bf16", "fp8"]), batch=batch,
                    q_len=q_len, prefix=_log_int(rng, 16, 500000),
                    page=rng.choice([8, 16, 32, 64, 128]),
                    rotary=rng.choice([32, 64, 96, 128, 192, 256]),
                    layout=rng.choice(["half", "interleaved"]),
                    offset=rng.choice([0.0, 1.0]),
                    ragged=rng.random() < 0.5)
    if op == "chunk":
        q_len = _log_int(rng, 1, 4096)
        # no more scores and no longer caches than the listed pieces have
        most = 68000000 // q_len - q_len
        prefix = _log_int(rng, 1, min(100000, most))
        total = q_len + prefix
        batch = _log_int(rng, 1, max(1, min(24, 68000000 // (q_len * total),
                                            400000 // total)))
        return dict(op="chunk", kv=rng.choice(["bf16", "fp8"]), batch=batch,
                    q_len=q_len, prefix=prefix,
                    page=rng.choice([8, 16, 32, 64, 128]),
                    ragged=rng.random() < 0.5)
    return dict(op="logp", dtype=rng.choice(["fp32", "bf16"]),
                rows=_log_int(rng, 1, 480), vocab=_log_int(rng, 900, 260000),
                top=rng.choice([0, 1, 5, 20, 32]),
                tempered=rng.random() < 0.5, peaks=rng.choice([0, 8, 64]),
                idle=rng.random() < 0.3)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV)


def _quantise(x):
    """E4M3 codes and fp16 scales of 64-channel blocks: scale = amax / 448
    (1 where that is zero), code = x / scale."""
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    s = (blocks.abs().amax(-1) / 448.0).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    c = (blocks / s.float()[..., None]).clamp(-448.0, 448.0)
    return c.to(torch.float8_e4m3fn).reshape(x.shape), s


def _pool(g, pages, page, kv):
    """A page pool with cached values in every slot: bf16, or E4M3 bytes and
    their scales."""
    def one():
        x = torch.empty((pages, HKV, page, D), dtype=torch.bfloat16,
                        device=DEV).normal_(generator=g)
        if kv == "bf16":
            return x, None
        codes = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
        scales = torch.empty((pages, HKV, page, D // 64),
                             dtype=torch.float16, device=DEV)
        step = max(1, (1 << 26) // (HKV * page * D))
        for i in range(0, pages, step):
            c, s = _quantise(x[i:i + step].float())
            codes[i:i + step] = c.view(torch.uint8)
            scales[i:i + step] = s
        return codes, scales
    k, ks = one()
    v, vs = one()
    return k, v, ks, vs


def prepare(case, seed):
    g = _gen(seed)
    return {"norm": _prepare_norm, "chunk": _prepare_chunk,
            "logp": _prepare_logp}[case["op"]](case, g)


def _prepare_norm(case, g):
    B, q_len, page = case["batch"], case["q_len"], case["page"]
    # the projections' output, one row per token: queries, keys, values, of
    # different sizes from head to head
    qkv = _randn(g, B, q_len, HQ + 2 * HKV, D)
    size = torch.exp(_randn(g, HQ + 2 * HKV))
    qkv = (qkv * size[:, None]).to(torch.bfloat16).view(B, q_len, -1)
    q = qkv[..., :HQ * D].view(B, q_len, HQ, D)
    k = qkv[..., HQ * D:(HQ + HKV) * D].view(B, q_len, HKV, D)
    v = qkv[..., (HQ + HKV) * D:].view(B, q_len, HKV, D)
    # weights near one, kept as such or as their distance from one
    w = (1.0 - case["offset"] + 0.2 * _randn(g, 2, D)).to(torch.bfloat16)
    q_lens = None
    widths = torch.full((B,), q_len, device=DEV, dtype=torch.int64)
    if case["ragged"]:
        widths = _ints(g, (q_len + 1) // 2, q_len, B)
        q_lens = widths.to(torch.int32)
    prefix = _ints(g, max(1, case["prefix"] // 8), case["prefix"], B)
    prefix[0] = case["prefix"]
    seq = prefix + widths
    # the pages that the block touches, in random order; every entry before
    # them belongs to the prefix and lies in pages that are not looked at
    cols = -(-(case["prefix"] + q_len) // page)
    per = -(-q_len // page) + 1
    pages = B * per + 1
    perm = (torch.randperm(pages - 1, generator=g, device=DEV) + 1).to(torch.int32)
    table = torch.zeros((B, cols), dtype=torch.int32, device=DEV)
    first = prefix // page
    at = torch.arange(per, device=DEV)[None, :] + first[:, None]
    ok = at < cols
    rows = torch.arange(B, device=DEV)[:, None].expand(B, per)
    table[rows[ok], at[ok]] = perm.view(B, per)[ok]
    k_pages, v_pages, ks, vs = _pool(g, pages, page, case["kv"])
    j = torch.arange(0, case["rotary"], 2, dtype=torch.float64, device=DEV)
    return dict(op="norm", q=q, k=k, v=v, wq=w[0].contiguous(),
                wk=w[1].contiguous(), offset=case["offset"], eps=1e-6,
                q_lens=q_lens, table=table, seq=seq.to(torch.int32),
                k_pages=k_pages, v_pages=v_pages, ks=ks, vs=vs,
                freq=1.0e6 ** (-j / case["rotary"]),
                interleaved=case["layout"] == "interleaved",
                positions=torch.empty((B, q_len), dtype=torch.int32,
                                      device=DEV),
                cache_loc=torch.empty((B, q_len), dtype=torch.int64,
                                      device=DEV))


def _prepare_chunk(case, g):
    B, q_len, page = case["batch"], case["q_len"], case["page"]
    widths = torch.full((B,), q_len, device=DEV, dtype=torch.int64)
    prefix = torch.full((B,), case["prefix"], device=DEV, dtype=torch.int64)
    q_lens = None
    if case["ragged"]:
        widths = _ints(g, 0, q_len, B)
        widths[0] = q_len
        if B > 2:
            widths[B // 2] = 0          # an idle request
            widths[B - 1] = 1           # one that decodes
        prefix = _ints(g, 0, case["prefix"], B)
        prefix[-1] = case["prefix"]
        q_lens = widths.to(torch.int32)
    seq = prefix + widths
    cols = -(-(case["prefix"] + q_len) // page)
    pages = B * cols
    table = torch.randperm(pages, generator=g, device=DEV).to(
        torch.int32).view(B, cols)
    k_pages, v_pages, ks, vs = _pool(g, pages, page, case["kv"])
    return dict(op="chunk", q=_randn(g, B, q_len, HQ, D).to(torch.bfloat16),
                q_lens=q_lens, table=table, seq=seq.to(torch.int32),
                k_pages=k_pages, v_pages=v_pages, ks=ks, vs=vs,
                scale=1.0 / math.sqrt(D))


def _prepare_logp(case, g):
    rows, vocab = case["rows"], case["vocab"]
    # a bulk of scores and, where the model is sure, a few tokens above it
    x = _randn(g, rows, vocab) * 2.0
    token = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    if case["peaks"]:
        # one in each part of the vocabulary, so that no two are the same
        part = vocab // case["peaks"]
        at = torch.randint(0, part, (rows, case["peaks"]), generator=g,
                           device=DEV)
        at = at + part * torch.arange(case["peaks"], device=DEV)
        up = 6.0 + 10.0 * torch.rand((rows, case["peaks"]), generator=g,
                                     device=DEV)
        x.scatter_(1, at, up)
        # most of the given tokens are likely ones
        likely = torch.rand(rows, generator=g, device=DEV) < 0.8
        pick = torch.randint(0, case["peaks"], (rows, 1), generator=g,
                             device=DEV)
        token = torch.where(likely, at.gather(1, pick)[:, 0], token)
    if case["dtype"] == "bf16":
        x = x.to(torch.bfloat16)
    if case["idle"]:                    # padding behind the accepted tokens
        off = torch.rand(rows, generator=g, device=DEV) < 0.4
        token = torch.where(off, torch.full_like(token, -1), token)
    t = None
    if case["tempered"]:
        t = 0.6 + 0.7 * torch.rand(rows, generator=g, device=DEV)
    return dict(op="logp", x=x, token=token.to(torch.int32), t=t,
                top=case["top"])


# ---------------------------------------------------------------- one pass

def run(s):
    return {"norm": _run_norm, "chunk": _run_chunk,
            "logp": _run_logp}[s["op"]](s)


def _run_norm(s):
    if own:
        import speculative_decoding_target_gb300 as sv
        q_out = sv.norm_rope_append(
            s["q"], s["k"], s["v"], s["wq"], s["wk"], s["freq"],
            s["k_pages"], s["v_pages"], s["table"], s["seq"], eps=s["eps"],
            weight_offset=s["offset"], interleaved=s["interleaved"],
            k_scales=s["ks"], v_scales=s["vs"], q_lens=s["q_lens"],
            positions=s["positions"], cache_loc=s["cache_loc"])
        pos, loc = s["positions"], s["cache_loc"]
    else:
        q_out, pos, loc = _plain_norm(s)
    out = dict(q=q_out, positions=pos, cache_loc=loc, k=s["k_pages"],
               v=s["v_pages"])
    if s["ks"] is not None:
        out.update(k=s["k_pages"].view(torch.float8_e4m3fn),
                   v=s["v_pages"].view(torch.float8_e4m3fn), ks=s["ks"],
                   vs=s["vs"])
    return out


def _widths(s, B, q_len):
    if s["q_lens"] is None:
        return torch.full((B,), q_len, device=DEV, dtype=torch.int64)
    return s["q_lens"].long().clamp(0, q_len)


def _normed(x, w, s):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    return x * r * (w.float() + s["offset"])


def _turn(x, cos, sin, n, interleaved):
    """The first n channels of every head rotated in pairs."""
    r, rest = x[..., :n], x[..., n:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned.flatten(-2), rest), -1)
    a, b = r[..., :n // 2], r[..., n // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)


def _plain_norm(s):
    B, q_len = s["q"].shape[:2]
    page = s["k_pages"].shape[2]
    w = _widths(s, B, q_len)
    i = torch.arange(q_len, device=DEV)
    pos = s["seq"].long()[:, None] - w[:, None] + i
    live = (i < w[:, None]) & (pos >= 0)
    n = 2 * s["freq"].shape[0]
    angle = pos.double()[..., None, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _turn(_normed(s["q"], s["wq"], s), cos, sin, n, s["interleaved"])
    q = torch.where(live[..., None, None], q, torch.zeros_like(q))
    k = _turn(_normed(s["k"], s["wk"], s), cos, sin, n, s["interleaved"])
    cols = s["table"].shape[1]
    slot_ok = live & (pos < cols * page)
    at = torch.where(slot_ok, pos, torch.zeros_like(pos))
    ids = s["table"].gather(1, at // page).long()
    loc = torch.where(slot_ok, ids * page + at % page,
                      torch.full_like(at, -1))
    where = (ids[slot_ok], slice(None), (at % page)[slot_ok])
    for new, pages, scales in ((k, s["k_pages"], s["ks"]),
                               (s["v"].float(), s["v_pages"], s["vs"])):
        rows = new[slot_ok]
        if scales is None:
            pages[where] = rows.to(pages.dtype)
        else:
            codes, sc = _quantise(rows)
            pages[where] = codes.view(torch.uint8)
            scales[where] = sc
    pos = torch.where(live, pos, torch.full_like(pos, -1)).to(torch.int32)
    return q.to(torch.bfloat16), pos, loc


def _run_chunk(s):
    if own:
        import speculative_decoding_target_gb300 as sv
        return sv.chunk_attention(
            s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq"],
            scale=s["scale"], k_scales=s["ks"], v_scales=s["vs"],
            q_lens=s["q_lens"])
    return _plain_chunk(s)


def _dense(pages, scales, table, valid):
    """[B, Hkv, T, D] in 32 bits from the pages of every request."""
    x = pages[table.long()]                       # [B, n, Hkv, page, D]
    if scales is not None:
        sc = scales[table.long()].float()
        x = x.view(torch.float8_e4m3fn).float()
        x = (x.view(*x.shape[:-1], D // 64, 64) * sc[..., None]).view(x.shape)
    x = x.float().transpose(1, 2)
    x = x.reshape(x.shape[0], HKV, -1, D)
    return torch.where(valid[:, None, :, None], x, torch.zeros_like(x))


def _plain_chunk(s):
    B, q_len = s["q"].shape[:2]
    T = s["table"].shape[1] * s["k_pages"].shape[2]
    t = torch.arange(T, device=DEV)
    w = _widths(s, B, q_len)
    i = torch.arange(q_len, device=DEV)
    limit = torch.where(i < w[:, None], s["seq"].long()[:, None] - w[:, None]
                        + i + 1, torch.zeros_like(i))
    valid = t < s["seq"].long()[:, None]
    k = _dense(s["k_pages"], s["ks"], s["table"], valid)
    q = s["q"].float().view(B, q_len, HKV, GROUP, D).transpose(1, 2)
    score = q.reshape(B, HKV, q_len * GROUP, D) @ k.transpose(2, 3)
    del k
    score = score.view(B, HKV, q_len, GROUP, T) * s["scale"]
    seen = t < limit[:, None, :, None, None]
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top > -math.inf, top,
                                      torch.zeros_like(top)))
    del score
    total = e.sum(-1, keepdim=True)
    v = _dense(s["v_pages"], s["vs"], s["table"], valid)
    o = (e.view(B, HKV, q_len * GROUP, T) @ v).view(B, HKV, q_len, GROUP, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.transpose(1, 2).reshape(B, q_len, HQ, D).to(torch.bfloat16)


def _run_logp(s):
    if own:
        import speculative_decoding_target_gb300 as sv
        return sv.logprobs(s["x"], s["token"], temperature=s["t"],
                           top=s["top"])
    return _plain_logp(s)


def _plain_logp(s):
    rows, vocab = s["x"].shape
    live = s["token"] >= 0
    x = s["x"].float()
    top = x.amax(-1, keepdim=True)
    z = x - top
    if s["t"] is not None:
        z = z / s["t"][:, None]
    e = torch.exp(z)
    total = e.sum(-1, dtype=torch.float64)
    mean = (e * z).sum(-1, dtype=torch.float64) / total
    lse = total.log()
    at = s["token"].long().clamp(min=0)[:, None]
    given = z.gather(1, at)[:, 0].double() - lse
    zero = torch.zeros_like(lse)
    out = dict(logprob=torch.where(live, given, zero).float(),
               entropy=torch.where(live, lse - mean, zero).float())
    if s["top"]:
        order = x.sort(dim=-1, descending=True, stable=True)[1]
        ids = order[:, :s["top"]]
        best = z.gather(1, ids).double() - lse[:, None]
        out.update(
            top_ids=torch.where(live[:, None], ids, torch.full_like(ids, -1)
                                ).to(torch.int32),
            top_logprobs=torch.where(live[:, None], best, torch.full_like(
                best, -math.inf)).float())
    return out


# ------------------------------------------------------------ work, exactly

def work(case):
    if case["op"] == "norm":
        n = case["batch"] * case["q_len"] * (0.75 if case["ragged"] else 1.0)
        row = HQ * D * 4 + 2 * HKV * D * 2
        kv = 2 * HKV * D * (2 if case["kv"] == "bf16" else 1 + 2 / 64)
        return dict(bytes=n * (row + kv + 12),
                    flops=n * (HQ + HKV) * (case["rotary"] * 3 + 4 * D))
    if case["op"] == "chunk":
        # the mean width of a piece and length of a prefix
        part = 0.5 if case["ragged"] and case["batch"] > 1 else 1.0
        w = max(1.0, part * case["q_len"])
        p = part * case["prefix"]
        tok = 2 * HKV * D * (2 if case["kv"] == "bf16" else 1 + 2 / 64)
        return dict(bytes=case["batch"] * ((p + w) * tok + w * HQ * D * 4),
                    flops=case["batch"] * w * (p + (w + 1) / 2) * HQ * D * 4)
    n = case["rows"] * case["vocab"] * (0.6 if case["idle"] else 1.0)
    return dict(bytes=n * (4 if case["dtype"] == "fp32" else 2)
                + case["rows"] * (12 + 8 * case["top"]), flops=6 * n)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "chunk": _exact_chunk,
            "logp": _exact_logp}[case["op"]](s)


def _exact_norm(s):
    """By complex numbers: a pair is x + iy, turned by exp(i angle)."""
    B, q_len = s["q"].shape[:2]
    page = s["k_pages"].shape[2]
    half = s["freq"].shape[0]
    fp8 = s["ks"] is not None
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)

    def pools(pages, scales):
        x = pages.view(torch.float8_e4m3fn) if fp8 else pages
        return x.double(), None if scales is None else scales.double()
    kp, ks = pools(s["k_pages"], s["ks"])
    vp, vs = pools(s["v_pages"], s["vs"])

    def spin(x, weight, z):
        x = x.double()
        length = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        x = x / torch.sqrt(length * length / D + s["eps"])
        x = x * (weight.double() + s["offset"])
        r = x[..., :2 * half].clone()
        if s["interleaved"]:
            c = torch.view_as_complex(r.view(*r.shape[:-1], half, 2)) * z
            r = torch.view_as_real(c).flatten(-2)
        else:
            c = torch.complex(r[..., :half].contiguous(),
                              r[..., half:].contiguous()) * z
            r = torch.cat((c.real, c.imag), -1)
        return torch.cat((r, x[..., 2 * half:]), -1)

    def put(pages, scales, ids, slots, rows):
        if not fp8:
            pages[ids, :, slots] = rows
            return
        b = rows.view(*rows.shape[:-1], D // 64, 64)
        sc = (b.abs().amax(-1) / 448.0)
        sc = torch.where(sc.half() == 0, torch.ones_like(sc), sc)
        pages[ids, :, slots] = (b / sc[..., None]).view(rows.shape)
        scales[ids, :, slots] = sc
    for b in range(B):
        n = q_len if s["q_lens"] is None else min(q_len, max(0, int(s["q_lens"][b])))
        first = int(s["seq"][b]) - n
        for i0 in range(0, n, 2048):
            i1 = min(n, i0 + 2048)
            at = torch.arange(first + i0, first + i1, device=DEV)
            z = torch.polar(torch.ones((i1 - i0, 1, half), dtype=torch.float64,
                                       device=DEV),
                            at.double()[:, None, None] * s["freq"])
            q_out[b, i0:i1] = spin(s["q"][b, i0:i1], s["wq"], z)
            ids = s["table"][b, at // page].long()
            put(kp, ks, ids, at % page, spin(s["k"][b, i0:i1], s["wk"], z))
            put(vp, vs, ids, at % page, s["v"][b, i0:i1].double())
    out = dict(q=q_out, positions=None, cache_loc=None, k=kp, v=vp)
    if fp8:
        out.update(ks=ks, vs=vs)
    return out


def _exact_chunk(s):
    """Request by request and head by head, some rows at a time."""
    B, q_len = s["q"].shape[:2]
    page = s["k_pages"].shape[2]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)

    def rows(pages, scales, b, n):
        ids = s["table"][b, :-(-n // page)].long()
        x = pages[ids]
        if scales is not None:
            sc = scales[ids].double().repeat_interleave(64, -1)
            x = x.view(torch.float8_e4m3fn).double() * sc
        return x.double().transpose(0, 1).reshape(HKV, -1, D)[:, :n]
    for b in range(B):
        w = q_len if s["q_lens"] is None else int(s["q_lens"][b])
        n = int(s["seq"][b])
        if w == 0:
            continue
        k, v = rows(s["k_pages"], s["ks"], b, n), rows(s["v_pages"], s["vs"], b, n)
        for i0 in range(0, w, 512):
            i1 = min(w, i0 + 512)
            m = n - w + i1
            hidden = (torch.arange(m, device=DEV)[None, :]
                      > torch.arange(n - w + i0, m, device=DEV)[:, None])
            for h in range(HQ):
                z = s["q"][b, i0:i1, h].double() @ k[h // GROUP, :m].T
                p = torch.softmax((z * s["scale"]).masked_fill(
                    hidden, -math.inf), -1)
                out[b, i0:i1, h] = p @ v[h // GROUP, :m]
    return out


def _exact_logp(s):
    """Row by row with the library's log softmax."""
    rows = s["x"].shape[0]
    given, spread, best = [], [], []
    for r in range(rows):
        tok = int(s["token"][r])
        if tok < 0:
            given.append(0.0)
            spread.append(0.0)
            best.append(torch.full((s["top"],), -math.inf,
                                   dtype=torch.float64, device=DEV))
            continue
        x = s["x"][r].double()
        if s["t"] is not None:
            x = x / s["t"][r].double()
        lp = torch.log_softmax(x, 0)
        given.append(float(lp[tok]))
        spread.append(float(-(lp.exp() * lp).sum()))
        best.append(lp.topk(s["top"])[0] if s["top"] else lp[:0])
    f64 = dict(dtype=torch.float64, device=DEV)
    out = dict(logprob=torch.tensor(given, **f64),
               entropy=torch.tensor(spread, **f64))
    if s["top"]:
        out.update(top_ids=None, top_logprobs=torch.stack(best))
    return out
