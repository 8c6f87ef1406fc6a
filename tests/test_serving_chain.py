"""A decode step as a server runs it: rotary append of the block, attention
with the shared prompt, the next token drawn from the head's logits; eager and
as one captured graph that is replayed step after step."""
import numpy as np
import pytest
import torch

import speculative_decoding_target_gb300 as sv
from speculative_decoding_target_gb300 import build
from test_rope_append import f64, rotate64
from test_sample import reference
from test_shared_prefix import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Step:
    """Requests that share a prompt, one token each a step.  The projection's
    output is the step's input; everything else is kept by the server."""

    def __init__(self, kv, q_len=1):
        build.build()
        self.c = c = Case([3, 2], [600, 300], [20, 33, 5, 64, 1],
                          q_len=q_len, page=16, kv=kv, seed=21)
        B = c.B
        # the tables hold room for 8 more tokens in pages of their own
        room = 8
        cols = -(-(max(c.seqs) + room) // 16)
        extra = torch.arange(B * 2, dtype=torch.int32, device=DEV).view(B, 2)
        pad = torch.zeros((2 * B,) + c.k.shape[1:], dtype=c.k.dtype,
                          device=DEV)
        table = torch.zeros((B, cols + 1), dtype=torch.int32, device=DEV)
        table[:, :c.table.shape[1]] = c.table
        for b in range(B):
            have = -(-c.seqs[b] // 16)
            table[b, have:have + 2] = extra[b] + c.pages
        c.table = table.contiguous()
        c.k, c.v = torch.cat([c.k, pad]), torch.cat([c.v, pad])
        if kv == "fp8":
            one = torch.ones((2 * B,) + c.ks.shape[1:], dtype=c.ks.dtype,
                             device=DEV)
            c.ks, c.vs = torch.cat([c.ks, one]), torch.cat([c.vs, one])
        g = torch.Generator(device=DEV).manual_seed(5)
        freq, self.m = sv.rope_frequencies(64, base=1e6, scaling="yarn",
                                           factor=2.0, original_context=512)
        self.freq = freq.to(DEV)
        self.head = torch.randn((24 * 256, 5000), generator=g,
                                device=DEV) * 0.3
        f = lambda *v: torch.tensor(v, device=DEV)
        self.t = f(1.0, 0.7, 1.2, 0.0, 0.9)
        self.k = f(0, 50, 1000, 0, 5).to(torch.int32)
        self.p = f(0.9, 0.95, 1.0, 1.0, 0.8)
        self.ws = sv.alloc_workspace(64 << 20, DEV)
        self.qkv = torch.empty((B, q_len, 32 * 256), dtype=torch.bfloat16,
                               device=DEV)
        self.u = torch.empty(B, device=DEV)
        self.q_rot = torch.empty((B, q_len, 24, 256), dtype=torch.bfloat16,
                                 device=DEV)
        self.out = torch.empty_like(self.q_rot)
        self.token = torch.empty(B, dtype=torch.int32, device=DEV)
        self.probs = torch.empty((B, 5000), device=DEV)

    def run(self):
        c, x = self.c, self.qkv
        B, q_len = x.shape[:2]
        c.seq += q_len                      # the block joins the cache
        sv.rope_append(x[..., :24 * 256].view(B, q_len, 24, 256),
                       x[..., 24 * 256:28 * 256].view(B, q_len, 4, 256),
                       x[..., 28 * 256:].view(B, q_len, 4, 256), self.freq,
                       c.k, c.v, c.table, c.seq, attn_factor=self.m,
                       q_out=self.q_rot, k_scales=c.ks, v_scales=c.vs)
        sv.verify_attention_shared(
            self.q_rot, c.k, c.v, c.table, c.seq, c.starts, c.shared,
            scale=c.scale, k_scales=c.ks, v_scales=c.vs, out=self.out,
            workspace=self.ws)
        self.logits = self.out[:, -1].reshape(B, -1).float() @ self.head
        sv.sample(self.logits, self.u, temperature=self.t, top_k=self.k,
                  top_p=self.p, token=self.token, probs=self.probs)

    def fill(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g, device=DEV))
        self.u.copy_(torch.rand(self.u.shape, generator=g, device=DEV))

    def check(self):
        """The step just run, each part against its definition."""
        c = self.c
        B, q_len = self.qkv.shape[:2]
        x = f64(self.qkv)
        pos = c.seq.cpu().numpy()[:, None] - q_len + np.arange(q_len)
        freq = self.freq.cpu().numpy()
        q, qe = rotate64(x[..., :24 * 256].reshape(B, q_len, 24, 256), pos,
                         freq, False, self.m)
        assert np.all(np.abs(f64(self.q_rot) - q)
                      <= np.abs(q) * 2.0 ** -8 + qe)
        k, ke = rotate64(x[..., 24 * 256:28 * 256].reshape(B, q_len, 4, 256),
                         pos, freq, False, self.m)
        for b in range(B):
            n = int(c.seq[b])
            got = c.dense(c.k, c.ks, b, n)[:, n - q_len:].cpu().numpy()
            want = k[b].transpose(1, 0, 2)
            e = ke[b].transpose(1, 0, 2)
            # FP8: half a code's step, and half an fp16 step of its scale
            step = 2.0 ** -8 if c.kv == "bf16" else 2.0 ** -4 + 2.0 ** -10
            low = 0.0 if c.kv == "bf16" else \
                np.abs(want).max(-1, keepdims=True) / 448 * 2.0 ** -9
            assert np.all(np.abs(got - want) <= np.abs(want) * step + e + low)
        # attention over the cache as it is now, and the draw from its logits
        c.seqs = c.seq.tolist()
        c.widths = [q_len] * B
        keep, c.q = c.q, self.q_rot
        c.check(self.out)
        c.q = keep
        x = self.logits.cpu().numpy()
        for b in range(B):
            tok, ids, pr, margin = reference(
                x[b], float(self.t[b]), int(self.k[b]), float(self.p[b]), 0.0,
                np.float32(self.u[b].item()))
            if margin >= 5000 * 2.0 ** -43:
                assert int(self.token[b]) == tok
                assert np.array_equal(np.flatnonzero(
                    self.probs[b].cpu().numpy()), np.sort(ids[pr[ids] > 1e-37]))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("q_len", [1, 3])
def test_decode_steps_eager_and_captured(kv, q_len):
    s = Step(kv, q_len)
    s.fill(1)
    s.run()
    s.check()
    start = s.c.seq.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    s.c.seq.copy_(start)                     # capturing runs nothing
    for step in range(2):
        s.fill(10 + step)
        graph.replay()
        torch.cuda.synchronize()
        s.check()
    # the replayed steps' results are the eager ones
    token, probs, out = (t.clone() for t in (s.token, s.probs, s.out))
    s.c.seq -= q_len
    s.run()
    assert torch.equal(s.out, out) and torch.equal(s.token, token)
    assert torch.equal(s.probs, probs)
