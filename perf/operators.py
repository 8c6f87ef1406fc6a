"""The serving operators next to verify attention, as they are measured.

Three operators of a decode or verify step:

  rope    rotary positions on the block's queries and keys, and the append of
          its keys and values to the paged cache (bf16, or FP8 with scales);
  shared  verify attention of requests that share cached prefixes, each shared
          part computed once for its whole group;
  sample  the next token from logits with temperature, top-k, top-p and min-p
          and given uniforms, and the distribution that was drawn from.

`own` chooses between the plain forms below (elementary torch operations in
32 bits, 64 where 32 lose what matters) and the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
HQ, HKV, D = 24, 4, 256         # the attention geometry of the benchmark
VOCAB = 248320
GROUP = HQ // HKV


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request's verify block at a short context: launch latency
        dict(name="rope_b1_q8", op="rope", kv="bf16", batch=1, q_len=8,
             prefix=4096, page=16, rotary=64, layout="half", scaling="none",
             ragged=False),
        # a batch of verify blocks into an FP8 cache, contexts up to 128K
        dict(name="rope_b32_q8_fp8", op="rope", kv="fp8", batch=32, q_len=8,
             prefix=131072, page=64, rotary=64, layout="half",
             scaling="linear", ragged=True),
        # a long prompt in one call, the whole head rotated
        dict(name="rope_prompt_8k", op="rope", kv="bf16", batch=1,
             q_len=8192, prefix=32768, page=64, rotary=256,
             layout="interleaved", scaling="yarn", ragged=False),
        # prompt pieces of several requests, padded, quantised on write
        dict(name="rope_prompts_fp8", op="rope", kv="fp8", batch=5,
             q_len=1531, prefix=20000, page=16, rotary=128,
             layout="interleaved", scaling="wavelength", ragged=True),
        # four samples of one short prompt, one token each: latency
        dict(name="shared_b4_q1_p4k", op="shared", kv="bf16", q_len=1,
             groups="4", prefixes="4096", tail=200, page=64, ragged=False),
        # a batch of verify blocks behind one long system prompt
        dict(name="shared_b32_q8_p32k", op="shared", kv="bf16", q_len=8,
             groups="32", prefixes="32768", tail=2048, page=64,
             ragged=False),
        # plain decoding of many samples of one document, FP8 cache
        dict(name="shared_b64_q1_p64k_fp8", op="shared", kv="fp8", q_len=1,
             groups="64", prefixes="65536", tail=1500, page=64,
             ragged=False),
        # several groups of different sizes, a request of its own, odd
        # lengths, blocks of different widths
        dict(name="shared_groups_ragged", op="shared", kv="bf16", q_len=5,
             groups="1,5,11,7", prefixes="0,3001,20011,9000", tail=1777,
             page=16, ragged=True),
        # one request's next token
        dict(name="sample_r1", op="sample", dtype="fp32", rows=1,
             vocab=VOCAB, kind="kp", peaks=24, probs=False),
        # a batch with a setting of its own for every request
        dict(name="sample_r64_mixed", op="sample", dtype="fp32", rows=64,
             vocab=VOCAB, kind="mixed", peaks=24, probs=False),
        # drafts of 32 requests at 7 positions with their distributions, as
        # the stochastic verify reads them; flat rows, wide nuclei
        dict(name="sample_r224_probs", op="sample", dtype="bf16", rows=224,
             vocab=VOCAB, kind="p", peaks=0, probs=True),
        # an odd vocabulary, few rows
        dict(name="sample_r17_v50001", op="sample", dtype="bf16", rows=17,
             vocab=50001, kind="mixed", peaks=8, probs=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "shared", "sample"])
    if op == "rope":
        q_len = _log_int(rng, 1, 4096)
        batch = _log_int(rng, 1, max(1, min(64, 8192 // q_len)))
        return dict(op="rope", kv=rng.choice(["bf16", "fp8"]), batch=batch,
                    q_len=q_len, prefix=_log_int(rng, 16, 500000),
                    page=rng.choice([8, 16, 32, 64, 128]),
                    rotary=rng.choice([32, 64, 96, 128, 192, 256]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn",
                                        "wavelength"]),
                    ragged=rng.random() < 0.5)
    if op == "shared":
        q_len = rng.randint(1, 16)
        n = rng.randint(1, 4)
        sizes = [_log_int(rng, 1, 24) for _ in range(n)]
        pre = [_log_int(rng, 30, min(40000, 2000000 // (x * q_len)))
               for x in sizes]
        return dict(op="shared", kv=rng.choice(["bf16", "fp8"]), q_len=q_len,
                    groups=",".join(map(str, sizes)),
                    prefixes=",".join(map(str, pre)),
                    tail=_log_int(rng, 20, 2000),
                    page=rng.choice([8, 16, 32, 64, 128]),
                    ragged=rng.random() < 0.5)
    return dict(op="sample", dtype=rng.choice(["fp32", "bf16"]),
                rows=_log_int(rng, 1, 128), vocab=_log_int(rng, 900, 260000),
                kind=rng.choice(["kp", "p", "mixed", "free"]),
                peaks=rng.choice([0, 8, 64]), probs=rng.random() < 0.5)


# ------------------------------------------------------------------- inputs

def _frequencies(rotary, scaling):
    """Inverse frequencies in radians per position (64 bits) and the factor
    on the rotated channels, for the usual ways to reach long contexts."""
    j = torch.arange(0, rotary, 2, dtype=torch.float64)
    base = 1.0e6
    if scaling == "ntk":         # a larger base for 4 times the context
        base = base * 4.0 ** (rotary / max(rotary - 2, 1))
    f = base ** (-j / rotary)
    factor = 1.0
    if scaling == "linear":
        f = f / 4.0
    elif scaling == "yarn":      # 4 times an original context of 32,768
        def at(turns):
            return rotary * math.log(32768 / (turns * 2 * math.pi)) / (
                2 * math.log(base))
        lo = max(math.floor(at(32.0)), 0)
        hi = min(math.ceil(at(1.0)), rotary - 1)
        ramp = ((torch.arange(rotary // 2, dtype=torch.float64) - lo)
                / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / 4.0 * ramp + f * (1 - ramp)
        factor = 0.1 * math.log(4.0) + 1.0
    elif scaling == "wavelength":  # 8 times an original context of 8,192,
        # long wavelengths stretched, short ones kept, a blend between
        wave = 2 * math.pi / f
        mix = ((8192 / wave - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = (1 - mix) * f / 8.0 + mix * f
    return f, factor


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
    return {"rope": _prepare_rope, "shared": _prepare_shared,
            "sample": _prepare_sample}[case["op"]](case, g)


def _prepare_rope(case, g):
    B, q_len, page = case["batch"], case["q_len"], case["page"]
    # the projections' output, one row per token: queries, keys, values
    qkv = _randn(g, B, q_len, (HQ + 2 * HKV) * D).to(torch.bfloat16)
    q = qkv[..., :HQ * D].view(B, q_len, HQ, D)
    k = qkv[..., HQ * D:(HQ + HKV) * D].view(B, q_len, HKV, D)
    v = qkv[..., (HQ + HKV) * D:].view(B, q_len, HKV, D)
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
    freq, factor = _frequencies(case["rotary"], case["scaling"])
    return dict(op="rope", q=q, k=k, v=v, q_lens=q_lens, table=table,
                seq=seq.to(torch.int32), k_pages=k_pages, v_pages=v_pages,
                ks=ks, vs=vs, freq=freq.to(DEV), factor=factor,
                interleaved=case["layout"] == "interleaved",
                positions=torch.empty((B, q_len), dtype=torch.int32,
                                      device=DEV),
                cache_loc=torch.empty((B, q_len), dtype=torch.int64,
                                      device=DEV))


def _split(case):
    return ([int(x) for x in case["groups"].split(",")],
            [int(x) for x in case["prefixes"].split(",")])


def _prepare_shared(case, g):
    sizes, shared = _split(case)
    B, q_len, page = sum(sizes), case["q_len"], case["page"]
    widths = torch.full((B,), q_len, device=DEV, dtype=torch.int64)
    q_lens = None
    if case["ragged"]:
        widths = _ints(g, 1, q_len, B)
        q_lens = widths.to(torch.int32)
    tails = _ints(g, max(1, case["tail"] // 4), case["tail"], B)
    tails[-1] = case["tail"]
    owner = torch.repeat_interleave(torch.arange(len(sizes)),
                                    torch.tensor(sizes)).tolist()
    pre = torch.tensor([shared[o] for o in owner], device=DEV)
    seq = pre + tails + widths
    cols = -(-(max(shared) + case["tail"] + q_len) // page)
    # whole pages are shared: a group's first shared // page pages are the
    # same for all, every later page is a request's own
    whole = [s // page for s in shared]
    own_pages = [cols - whole[o] for o in owner]
    pages = sum(whole) + sum(own_pages)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.empty((B, cols), dtype=torch.int32, device=DEV)
    at, front = 0, []
    for w in whole:
        front.append(perm[at:at + w])
        at += w
    for b, o in enumerate(owner):
        table[b, :whole[o]] = front[o]
        table[b, whole[o]:] = perm[at:at + own_pages[b]]
        at += own_pages[b]
    k_pages, v_pages, ks, vs = _pool(g, pages, page, case["kv"])
    starts = [0]
    for s in sizes:
        starts.append(starts[-1] + s)
    return dict(op="shared",
                q=_randn(g, B, q_len, HQ, D).to(torch.bfloat16),
                q_lens=q_lens, table=table, seq=seq.to(torch.int32),
                k_pages=k_pages, v_pages=v_pages, ks=ks, vs=vs,
                starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                shared=torch.tensor([w * page for w in whole],
                                    dtype=torch.int32, device=DEV),
                scale=1.0 / math.sqrt(D))


def _prepare_sample(case, g):
    rows, vocab = case["rows"], case["vocab"]
    # a bulk of scores and, where the model is sure, a few tokens above it
    x = _randn(g, rows, vocab) * 2.0
    if case["peaks"]:
        at = torch.randint(0, vocab, (rows, case["peaks"]), generator=g,
                           device=DEV)
        up = 6.0 + 10.0 * torch.rand((rows, case["peaks"]), generator=g,
                                     device=DEV)
        x.scatter_(1, at, up)
    if case["dtype"] == "bf16":
        x = x.to(torch.bfloat16)

    def pick(*values):
        i = torch.randint(0, len(values), (rows,), generator=g, device=DEV)
        return torch.tensor(values, device=DEV)[i]
    kind = case["kind"]
    t = 0.6 + 0.7 * torch.rand(rows, generator=g, device=DEV)
    k = p = m = None
    if kind == "kp":
        k = pick(20, 50, 200).to(torch.int32)
        p = pick(0.8, 0.9, 0.95)
    elif kind == "p":
        p = pick(0.9, 0.95, 0.99)
    elif kind == "mixed":
        t = torch.where(pick(0, 1, 1, 1, 1) == 0, torch.zeros_like(t), t)
        k = pick(0, 0, 1, 50, 1000).to(torch.int32)
        p = pick(1.0, 0.5, 0.9, 0.95)
        m = pick(0.0, 0.0, 0.02, 0.1)
    u = torch.rand(rows, generator=g, device=DEV).clamp_(min=2.0 ** -25)
    return dict(op="sample", x=x, t=t, k=k, p=p, m=m, u=u,
                probs=case["probs"])


# ---------------------------------------------------------------- one pass

def run(s):
    return {"rope": _run_rope, "shared": _run_shared,
            "sample": _run_sample}[s["op"]](s)


def _run_rope(s):
    if own:
        import speculative_decoding_target_gb300 as sv
        q_out = sv.rope_append(
            s["q"], s["k"], s["v"], s["freq"], s["k_pages"], s["v_pages"],
            s["table"], s["seq"], interleaved=s["interleaved"],
            attn_factor=s["factor"], k_scales=s["ks"], v_scales=s["vs"],
            q_lens=s["q_lens"], positions=s["positions"],
            cache_loc=s["cache_loc"])
        pos, loc = s["positions"], s["cache_loc"]
    else:
        q_out, pos, loc = _plain_rope(s)
    out = dict(q=q_out, positions=pos, cache_loc=loc, k=s["k_pages"],
               v=s["v_pages"])
    if s["ks"] is not None:
        out.update(k=s["k_pages"].view(torch.float8_e4m3fn),
                   v=s["v_pages"].view(torch.float8_e4m3fn), ks=s["ks"],
                   vs=s["vs"])
    return out


def _turn(x, cos, sin, n, interleaved, dtype):
    """The first n channels of every head rotated in pairs."""
    x = x.to(dtype)
    r, rest = x[..., :n], x[..., n:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned.flatten(-2), rest), -1)
    a, b = r[..., :n // 2], r[..., n // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)


def _widths(s, B, q_len):
    if s["q_lens"] is None:
        return torch.full((B,), q_len, device=DEV, dtype=torch.int64)
    return s["q_lens"].long().clamp(0, q_len)


def _plain_rope(s):
    B, q_len = s["q"].shape[:2]
    page = s["k_pages"].shape[2]
    w = _widths(s, B, q_len)
    i = torch.arange(q_len, device=DEV)
    pos = s["seq"].long()[:, None] - w[:, None] + i
    live = (i < w[:, None]) & (pos >= 0)
    n = 2 * s["freq"].shape[0]
    angle = pos.double()[..., None, None] * s["freq"]
    cos = (angle.cos() * s["factor"]).float()
    sin = (angle.sin() * s["factor"]).float()
    q = _turn(s["q"], cos, sin, n, s["interleaved"], torch.float32)
    q = torch.where(live[..., None, None], q, torch.zeros_like(q))
    k = _turn(s["k"], cos, sin, n, s["interleaved"], torch.float32)
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


def _run_shared(s):
    if own:
        import speculative_decoding_target_gb300 as sv
        return sv.verify_attention_shared(
            s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq"],
            s["starts"], s["shared"], scale=s["scale"], k_scales=s["ks"],
            v_scales=s["vs"], q_lens=s["q_lens"])
    return _plain_shared(s)


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


def _plain_shared(s):
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


def _run_sample(s):
    if own:
        import speculative_decoding_target_gb300 as sv
        probs = (torch.empty(s["x"].shape, device=DEV) if s["probs"]
                 else None)
        tok = sv.sample(s["x"], s["u"], temperature=s["t"], top_k=s["k"],
                        top_p=s["p"], min_p=s["m"], probs=probs)
        return dict(token=tok, probs=probs)
    return _plain_sample(s)


def _plain_sample(s):
    x = s["x"].float()
    rows, vocab = x.shape
    dev = x.device
    value, order = x.sort(dim=-1, descending=True, stable=True)
    greedy = s["t"] == 0
    t = torch.where(greedy, torch.ones_like(s["t"]), s["t"]).double()
    # weights next to a cumulative border decide a token: 64 bits
    w = torch.exp((value.double() - value[:, :1].double()) / t[:, None])
    rank = torch.arange(vocab, device=dev)
    keep = torch.ones(rows, vocab, dtype=torch.bool, device=dev)
    if s["k"] is not None:
        k = torch.where(s["k"] > 0, s["k"].long(), torch.full_like(
            s["k"], vocab, dtype=torch.int64))
        keep &= rank < k[:, None]
    keep &= ~greedy[:, None] | (rank == 0)
    w = torch.where(keep, w, torch.zeros_like(w))
    if s["p"] is not None:
        run = w.cumsum(-1)
        before = run - w
        on = s["p"].double() < 1.0
        keep &= ~on[:, None] | (before < s["p"].double()[:, None]
                                * run[:, -1:]) | (rank == 0)
    if s["m"] is not None:
        keep &= (w >= s["m"].double()[:, None]) | (rank == 0)
    w = torch.where(keep, w, torch.zeros_like(w))
    by_id = torch.zeros_like(w).scatter_(1, order, w)
    run = by_id.cumsum(-1)
    total = run[:, -1:]
    target = s["u"].double()[:, None] * total
    token = torch.searchsorted(run, target, right=True)[:, 0]
    last = (by_id > 0).long().mul_(rank).amax(-1)
    token = torch.minimum(token, last).to(torch.int32)
    probs = (by_id / total).float() if s["probs"] else None
    return dict(token=token, probs=probs)


# ------------------------------------------------------------ work, exactly

def work(case):
    if case["op"] == "rope":
        n = case["batch"] * case["q_len"] * (0.75 if case["ragged"] else 1.0)
        row = HQ * D * 4 + 2 * HKV * D * 2
        kv = 2 * HKV * D * (2 if case["kv"] == "bf16" else 1 + 2 / 64)
        return dict(bytes=n * (row + kv + 12),
                    flops=n * (HQ + HKV) * case["rotary"] * 3)
    if case["op"] == "shared":
        sizes, shared = _split(case)
        q_len = case["q_len"]
        # the mean width of a block, and of a tail
        width = (q_len + 1) / 2 if case["ragged"] else q_len
        tail = 0.625 * case["tail"]
        tok = 2 * HKV * D * (2 if case["kv"] == "bf16" else 1 + 2 / 64)
        b = f = 0.0
        for n, p in zip(sizes, shared):
            b += (p + n * (tail + width)) * tok + n * width * HQ * D * 4
            f += n * width * (p + tail + width / 2) * HQ * D * 4
        return dict(bytes=b, flops=f)
    n = case["rows"] * case["vocab"]
    return dict(bytes=n * ((4 if case["dtype"] == "fp32" else 2)
                           + (4 if case["probs"] else 0)), flops=8 * n)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "shared": _exact_shared,
            "sample": _exact_sample}[case["op"]](s)


def _exact_rope(s):
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

    def spin(x, z):
        x = x.double().clone()
        r = x[..., :2 * half]
        if s["interleaved"]:
            c = torch.complex(r[..., 0::2].contiguous(),
                              r[..., 1::2].contiguous()) * z
            r[..., 0::2], r[..., 1::2] = c.real, c.imag
        else:
            c = torch.complex(r[..., :half].contiguous(),
                              r[..., half:].contiguous()) * z
            r[..., :half], r[..., half:] = c.real, c.imag
        return x

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
            z = torch.polar(torch.full((i1 - i0, 1, half), float(s["factor"]),
                                       dtype=torch.float64, device=DEV),
                            at.double()[:, None, None] * s["freq"])
            q_out[b, i0:i1] = spin(s["q"][b, i0:i1], z)
            ids = s["table"][b, at // page].long()
            put(kp, ks, ids, at % page, spin(s["k"][b, i0:i1], z))
            put(vp, vs, ids, at % page, s["v"][b, i0:i1].double())
    out = dict(q=q_out, positions=None, cache_loc=None, k=kp, v=vp)
    if fp8:
        out.update(ks=ks, vs=vs)
    return out


def _exact_shared(s):
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
        k, v = rows(s["k_pages"], s["ks"], b, n), rows(s["v_pages"], s["vs"], b, n)
        for i in range(w):
            m = n - w + i + 1
            q = s["q"][b, i].double().view(HKV, GROUP, D)
            p = torch.softmax(torch.einsum("hgd,htd->hgt", q, k[:, :m])
                              * s["scale"], -1)
            out[b, i] = torch.einsum("hgt,htd->hgd", p, v[:, :m]).reshape(HQ, D)
    return out


def _exact_sample(s):
    """Row by row, by a search for the border in the sorted weights."""
    rows, vocab = s["x"].shape
    tokens, dist = [], []
    for r in range(rows):
        x = s["x"][r].double()
        t = float(s["t"][r])
        ids = torch.argsort(-x, stable=True)
        n = vocab
        if t == 0:
            n, t = 1, 1.0
        if s["k"] is not None and int(s["k"][r]) > 0:
            n = min(n, int(s["k"][r]))
        w = torch.exp((x[ids[:n]] - x[ids[0]]) / t)
        if s["p"] is not None and float(s["p"][r]) < 1.0:
            c = torch.cumsum(w, 0)
            n = int(torch.searchsorted(c, c[-1] * float(s["p"][r]))) + 1
            w = w[:n]
        if s["m"] is not None:
            n = max(1, int((w >= float(s["m"][r])).sum()))
            w = w[:n]
        full = torch.zeros(vocab, dtype=torch.float64, device=DEV)
        full[ids[:w.shape[0]]] = w
        p = full / full.sum()
        c = torch.cumsum(full, 0)
        tok = torch.searchsorted(c, c[-1] * float(s["u"][r]), right=True)
        tokens.append(tok.to(torch.int32))
        if s["probs"]:
            dist.append(p)
    return dict(token=torch.stack(tokens),
                probs=torch.stack(dist) if s["probs"] else None)
