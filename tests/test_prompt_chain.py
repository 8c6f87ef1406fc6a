"""A prompt as a server runs it: head norms with rotary append and attention over
the cache, piece by piece, log probabilities of the prompt's tokens, then tokens
drawn and scored one at a time; eager and as one captured graph."""
import numpy as np
import pytest
import torch

import speculative_decoding_target_gb300 as sv
from speculative_decoding_target_gb300 import build
from test_chunk_attention import Case
from test_logprobs import check as check_logprobs
from test_norm_rope import expected, f64, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, VOCAB = 8, 2, 6001


class Server:
    """Two requests' caches; a layer's projection and head are its input."""

    def __init__(self, kv, lengths, piece):
        build.build()
        self.kv, self.lengths, self.piece = kv, lengths, piece
        B = len(lengths)
        # a cache with room for the prompt and a few tokens, all of it unwritten
        self.c = c = Case([n + 8 for n in lengths], [0] * B, hq=HQ, hkv=HKV,
                          kv=kv, page=16, seed=3)
        if kv == "bf16":
            c.k.fill_(float("nan"))
            c.v.fill_(float("nan"))
        else:
            c.k.fill_(0x7F)
            c.v.fill_(0x7F)
            c.ks.fill_(float("nan"))
            c.vs.fill_(float("nan"))
        self.w = weights(4, torch.bfloat16, 1.0)
        freq, self.m = sv.rope_frequencies(64, base=1e6, scaling="linear",
                                           factor=2.0)
        self.freq = freq.to(DEV)
        g = torch.Generator(device=DEV).manual_seed(6)
        self.head = torch.randn((HQ * 256, VOCAB), generator=g,
                                device=DEV) * 0.1
        self.seq = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.width = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.qkv = torch.zeros((B, piece, HQ + 2 * HKV, 256),
                               dtype=torch.bfloat16, device=DEV)
        self.given = torch.zeros((B, piece), dtype=torch.int32, device=DEV)
        self.k_all = [[] for _ in lengths]     # what the cache should hold
        self.v_all = [[] for _ in lengths]

    def step(self):
        """A piece of every prompt: the lengths include it already."""
        c, x = self.c, self.qkv
        self.q = sv.norm_rope_append(
            x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], self.w[0],
            self.w[1], self.freq, c.k, c.v, c.table, self.seq,
            weight_offset=1.0, attn_factor=self.m, k_scales=c.ks,
            v_scales=c.vs, q_lens=self.width)
        self.out = sv.chunk_attention(
            self.q, c.k, c.v, c.table, self.seq, scale=c.scale,
            k_scales=c.ks, v_scales=c.vs, q_lens=self.width)
        self.logits = self.out.flatten(2).float() @ self.head
        self.scores = sv.logprobs(self.logits, self.given, top=4)

    def load(self, first, seed):
        """The next piece's inputs: tokens first .. of every prompt."""
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g, device=DEV))
        n = [max(0, min(self.piece, L - first)) for L in self.lengths]
        self.width.copy_(torch.tensor(n))
        self.seq.copy_(torch.tensor([min(first + self.piece, L)
                                     for L in self.lengths]))
        self.given.copy_(torch.randint(0, VOCAB, self.given.shape, generator=g,
                                       device=DEV))
        for b, k in enumerate(n):
            self.given[b, k:] = -1             # padding is not scored

    def check(self):
        c, x = self.c, f64(self.qkv)
        w, n = self.width.tolist(), self.seq.tolist()
        pos = np.array(n)[:, None] - np.array(w)[:, None] + np.arange(self.piece)
        freq = self.freq.cpu().numpy()
        q, qe = expected(x[:, :, :HQ], f64(self.w[0]), 1e-6, 1.0, pos, freq,
                         False, self.m)
        k, ke = expected(x[:, :, HQ:HQ + HKV], f64(self.w[1]), 1e-6, 1.0, pos,
                         freq, False, self.m)
        for b in range(len(w)):
            i = slice(0, w[b])
            assert np.all(np.abs(f64(self.q[b, i]) - q[b, i])
                          <= np.abs(q[b, i]) * 2.0 ** -8 + qe[b, i])
            assert not self.q[b, w[b]:].any()
            if not w[b]:
                continue
            self.k_all[b].append(k[b, i])
            self.v_all[b].append(x[b, i, HQ + HKV:])
            # every token of the cache so far is what was appended for it
            for pages, scales, rows, e in (
                    (c.k, c.ks, self.k_all[b], 2e-6),
                    (c.v, c.vs, self.v_all[b], 0.0)):
                want = np.concatenate(rows).transpose(1, 0, 2)
                got = c.dense(pages, scales, b, n[b]).cpu().numpy()
                big = np.abs(want).reshape(HKV, -1, 4, 64).max(-1).repeat(64, -1)
                # FP8: half a code's step of its block, half a scale's step
                tol = (np.abs(want) * 2.0 ** -8 if self.kv == "bf16" else
                       np.abs(want) * (2.0 ** -4 + 2.0 ** -10)
                       + big / 448 * 2.0 ** -9)
                assert np.all(np.abs(got - want) <= tol + 2 * e * big)
        c.q, c.seqs, c.widths, c.q_len = self.q, n, w, self.piece
        c.check(self.out)
        check_logprobs(self.logits.view(-1, VOCAB),
                       {k: v.flatten(0, 1) for k, v in self.scores.items()},
                       self.given.flatten().tolist(), None, 4)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("lengths,piece", [([300, 90], 128), ([70, 41], 16)])
def test_prompts_in_pieces(kv, lengths, piece):
    s = Server(kv, lengths, piece)
    for first in range(0, max(lengths), piece):
        s.load(first, 10 + first)
        s.step()
        s.check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_captured_pieces(kv):
    s = Server(kv, [200, 150], 64)
    s.load(0, 1)
    s.step()
    s.check()
    graph = torch.cuda.CUDAGraph()
    s.load(64, 2)
    with torch.cuda.graph(graph):
        s.step()
    for first in range(64, 200, 64):
        s.load(first, 3 + first)
        graph.replay()
        torch.cuda.synchronize()
        s.check()
    out, lp = s.out.clone(), s.scores["logprob"].clone()
    s.step()                                   # the same eagerly
    assert torch.equal(s.out, out)
    assert torch.equal(s.scores["logprob"], lp)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_drawn_tokens_are_scored(kv):
    s = Server(kv, [40, 25], 40)
    s.load(0, 1)
    s.step()
    s.check()
    # one token each: the draw from the last row's logits, and its score
    g = torch.Generator(device=DEV).manual_seed(8)
    s.piece = 1
    s.qkv = s.qkv[:, :1].contiguous()
    last = s.logits[torch.arange(2, device=DEV), s.width.long() - 1]
    s.lengths = [n + 1 for n in s.lengths]
    for _ in range(3):
        u = torch.rand(2, generator=g, device=DEV)
        probs = torch.empty((2, VOCAB), device=DEV)
        token = sv.sample(last, u, probs=probs)
        score = sv.logprobs(last, token, top=1)
        p = probs.gather(1, token.long()[:, None])[:, 0]
        assert torch.allclose(score["logprob"].exp(), p, rtol=1e-4)
        s.qkv.copy_(torch.randn(s.qkv.shape, generator=g, device=DEV))
        s.width.fill_(1)
        s.seq += 1
        s.given = token[:, None].contiguous()
        s.step()
        s.check()
        last = s.logits[:, 0]
