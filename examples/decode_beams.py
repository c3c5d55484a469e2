"""Beam search with a small mixture-of-experts decoder, every operator of a decode step together:

    prompt      its tokens go through the step one by one, into one sequence of the cache
    fork        every beam becomes a copy of the prompt's sequence: whole pages are shared
    step        extend -> per layer: qkv GEMV, write (the sequences that grew), attention over shared
                prefix and own pages, output GEMV, router, experts -> vocabulary GEMV
    fork        the best continuations' parents become the next beams
    compact     at the end, with the prompt's own sequence freed

Weights are random; embedding, norms and the choice of beams are plain torch.

    python examples/decode_beams.py [--beams 4] [--tokens 24]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from block_scaled_bit_gb300 import bsgemv, synth  # noqa: E402


class Linear:
    """Block-scaled weights [N, K] of roughly unit gain, and a plan for up to max_M rows."""

    def __init__(self, N: int, K: int, max_M: int, seed: int):
        s = 0.2 / math.sqrt(K)  # int4 codes about their zero points spread by some 5 steps
        case = synth.make_case("int4", "f16", 32, True, N, K, 1, seed, scale_range=(s, 1.2 * s))
        self.w = bsgemv.upload(case)
        self.N = N
        self.plan = bsgemv.Plan("int4", "f16", 32, True, N, K, max_M)

    def __call__(self, x):
        y = torch.empty(x.shape[0], self.N, dtype=torch.float16, device=x.device)
        self.plan.run(x, self.w.W, self.w.scales, self.w.zp, y)
        return y


class Experts:
    def __init__(self, H: int, I: int, E: int, top_k: int, max_T: int, seed: int):
        def stacked(N, K, seed):
            s = 0.2 / math.sqrt(K)
            return bsgemv.upload(synth.make_case("int4", "f16", 32, True, E * N, K, 1, seed,
                                                 scale_range=(s, 1.2 * s)))

        self.w13, self.w2 = stacked(2 * I, H, seed), stacked(H, I, seed + 1)
        g = torch.Generator().manual_seed(seed)
        self.router = (torch.randn(H, E, generator=g) / math.sqrt(H)).half().cuda()  # [K, N]
        self.route = bsgemv.DensePlan("f16", E, H, max_M=min(max_T, 8))  # eight rows a call at most
        self.plan = bsgemv.MoePlan("int4", "f16", 32, True, H, I, E, top_k, max_T)
        self.E = E

    def __call__(self, x):
        logits = torch.empty(x.shape[0], self.E, dtype=torch.float16, device=x.device)
        for i in range(0, x.shape[0], 8):
            self.route.run(x[i:i + 8], self.router, logits[i:i + 8])
        y = torch.empty_like(x)
        self.plan.run(x, logits, self.w13.W, self.w13.scales, self.w13.zp,
                      self.w2.W, self.w2.scales, self.w2.zp, y)
        return y


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()


class Decoder:
    def __init__(self, max_seqs: int = 9, layers: int = 2, H: int = 512, Hq: int = 8, Hkv: int = 2,
                 D: int = 64, I: int = 256, E: int = 16, top_k: int = 4, vocab: int = 1024,
                 page_size: int = 16, num_pages: int = 128, max_pages: int = 16, seed: int = 0):
        self.H, self.Hq, self.Hkv, self.D, self.ps = H, Hq, Hkv, D, page_size
        g = torch.Generator().manual_seed(seed)
        self.embed = torch.randn(vocab, H, generator=g).half().cuda()
        self.place = torch.randn(max_pages * page_size, H, generator=g).half().cuda()
        self.qkv = [Linear((Hq + 2 * Hkv) * D, H, max_seqs, seed + 10 * i + 1)
                    for i in range(layers)]
        self.o = [Linear(H, Hq * D, max_seqs, seed + 10 * i + 2) for i in range(layers)]
        self.experts = [Experts(H, I, E, top_k, max_seqs, seed + 10 * i + 3)
                        for i in range(layers)]
        self.head = Linear(vocab, H, max_seqs, seed + 9)
        self.attn = bsgemv.AttnPlan("f16", Hq, Hkv, D, page_size, max_seqs)

        # the cache: a plane each for K and V of a layer, pages [row][head][D]
        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device="cuda")

        self.pool = torch.zeros(2 * layers, num_pages, page_size, Hkv, D, dtype=torch.float16,
                                device="cuda")
        self.refs, self.tables = ints(num_pages), ints(max_seqs, max_pages, fill=-1)
        self.lens = ints(max_seqs)
        self.short = torch.zeros((), dtype=torch.bool, device="cuda")  # a page was wanted, none left
        self.cache = bsgemv.PageCache(2 * layers, num_pages, page_size * Hkv * D * 2, page_size,
                                      max_seqs, max_pages)

    def plane(self, i):  # as attention reads it: [page][head][row][D]
        return self.pool[i].permute(0, 2, 1, 3)

    def step(self, tokens, seqs, prefix_seq: int = 0, prefix_len: int = 0):
        """One token for each sequence of `seqs` (a run of slots: a first slot and one per token).
        The first prefix_len positions are those of sequence prefix_seq.  Returns log
        probabilities [n, vocab]."""
        n, Hq, Hkv, D = tokens.shape[0], self.Hq, self.Hkv, self.D
        slots = torch.arange(seqs, seqs + n, dtype=torch.int32, device="cuda")
        grown = torch.empty_like(slots)
        self.cache.extend(self.pool, self.refs, self.tables, self.lens, slots, grown)
        self.short |= (grown == 0).any()
        # a sequence that did not grow has its last token where a new one would be written
        write = torch.where(grown > 0, slots, -1)
        tables, lens = self.tables[seqs:seqs + n], self.lens[seqs:seqs + n]
        x = self.embed[tokens] + self.place[lens.long() - 1]
        for i, (qkv_of, o_of, experts) in enumerate(zip(self.qkv, self.o, self.experts)):
            qkv = qkv_of(norm(x)).view(n, Hq + 2 * Hkv, D)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            self.cache.write(self.pool, self.tables, self.lens, write, k, v, head_stride=D,
                             row_stride=Hkv * D, k_plane=2 * i, v_plane=2 * i + 1)
            out = torch.empty(n, Hq, D, dtype=torch.float16, device="cuda")
            self.attn.run(q, self.plane(2 * i), self.plane(2 * i + 1), self.tables[prefix_seq],
                          prefix_len, tables, lens, out)
            x = x + o_of(out.view(n, Hq * D))
            x = x + experts(norm(x))
        return torch.log_softmax(self.head(norm(x)).float(), -1)

    def fork(self, parents, children):
        new = torch.empty_like(children)
        self.cache.fork(self.pool, self.refs, self.tables, self.lens, parents.int(), children, new)
        self.short |= (new == -2).any()

    def check(self):
        """Raises if a sequence found no page or row to grow in, or a wait of a kernel ran out."""
        if self.short:
            raise RuntimeError("the cache's pages or a sequence's row ran out")
        for plan in [self.attn] + [e.plan for e in self.experts]:
            status = plan.device_status()
            if status != 0:
                raise RuntimeError(bsgemv.status_string(status))


def beam_search(model: Decoder, prompt, beams: int, tokens: int):
    """The `beams` best continuations found, [beams, tokens] with their log probabilities.  Slots
    0 .. beams-1 hold the beams, slot `beams` the prompt."""
    slots = torch.arange(beams, dtype=torch.int32, device="cuda")
    for t in prompt:
        logp = model.step(t[None], seqs=beams)
    score, last = logp[0].topk(beams)
    model.fork(torch.full_like(slots, beams), slots)
    out = last[:, None]
    for _ in range(tokens - 1):
        logp = model.step(last, seqs=0, prefix_seq=beams, prefix_len=len(prompt))
        score, flat = (score[:, None] + logp).flatten().topk(beams)
        parents, last = flat // logp.shape[1], flat % logp.shape[1]
        model.fork(parents, slots)
        out = torch.cat([out[parents], last[:, None]], 1)
    model.check()
    return out, score


def main() -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--prompt", type=int, default=37)
    a = ap.parse_args()
    if not 1 <= a.beams <= 31 or a.tokens < 1 or a.prompt < 1:
        ap.error("1 to 31 beams, a token and a prompt of one token at least")
    # every sequence's pages, and the copies of a fork beside the pages that it gives back
    ps = 16
    pages = -(-(a.prompt + a.tokens) // ps)
    model = Decoder(max_seqs=a.beams + 1, page_size=ps, max_pages=pages,
                    num_pages=(a.beams + 1) * pages + a.beams)
    g = torch.Generator().manual_seed(1)
    prompt = torch.randint(model.embed.shape[0], (a.prompt,), generator=g).cuda()
    out, score = beam_search(model, prompt, a.beams, a.tokens)
    for o, s in zip(out.tolist(), score.tolist()):
        print(f"{s:9.4f}  {o}")
    pages = int((model.refs > 0).sum())
    model.cache.free(model.refs, model.tables, model.lens,
                     torch.tensor([a.beams], dtype=torch.int32, device="cuda"))
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    model.cache.compact(model.pool, model.refs, model.tables, model.lens, model.refs, model.tables,
                        live)
    print(f"pages in use: {pages}, after the prompt's sequence is freed and the pool compacted: "
          f"{int(live)}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
