"""Several prompts served at once by a small mixture-of-experts decoder: every call takes up to 32 rows,
pieces of prompts beside sequences that decode one token each.

    call        grow -> per layer: qkv GEMV, append (head norms, rotation, keys and values into their
                pages), attention of the new tokens, output GEMV, router, experts -> vocabulary GEMV
                for each entry's last row
    schedule    sequences that decode first, then prompts in order, as far as the rows go
    end         a sequence that has all its tokens is freed, and its pages go to the next prompt

Weights are random; embedding, the layers' norms and the choice of tokens (the likeliest) are plain torch.

    python examples/serve_chunks.py [--prompts 6] [--tokens 12] [--rows 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from block_scaled_bit_gb300 import bsgemv  # noqa: E402
from decode_beams import Experts, Linear, norm  # noqa: E402


class Server:
    def __init__(self, slots: int = 4, rows: int = 32, layers: int = 2, H: int = 512, Hq: int = 8,
                 Hkv: int = 2, D: int = 64, I: int = 256, E: int = 16, top_k: int = 4,
                 vocab: int = 1024, page_size: int = 16, num_pages: int = 96, max_pages: int = 32,
                 seed: int = 0):
        self.H, self.Hq, self.Hkv, self.D, self.ps, self.rows = H, Hq, Hkv, D, page_size, rows
        g = torch.Generator().manual_seed(seed)
        self.embed = torch.randn(vocab, H, generator=g).half().cuda()
        self.qkv = [Linear((Hq + 2 * Hkv) * D, H, rows, seed + 10 * i + 1) for i in range(layers)]
        self.o = [Linear(H, Hq * D, rows, seed + 10 * i + 2) for i in range(layers)]
        self.experts = [Experts(H, I, E, top_k, rows, seed + 10 * i + 3) for i in range(layers)]
        self.norms = [[(1 + 0.1 * torch.randn(D, generator=g)).half().cuda() for _ in range(2)]
                      for _ in range(layers)]
        self.head = Linear(vocab, H, slots, seed + 9)
        self.rope = bsgemv.RopePlan("f16", Hq, Hkv, D, base=10000.0)
        # every other layer sees a window of its sequence only
        self.windows = [0 if i % 2 == 0 else 64 for i in range(layers)]
        self.attn = bsgemv.ChunkPlan("f16", Hq, Hkv, D, page_size, max_n=slots, max_T=rows)

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device="cuda")

        # the cache: a plane each for K and V of a layer, pages [row][head][D]
        self.pool = torch.zeros(2 * layers, num_pages, page_size, Hkv, D, dtype=torch.float16,
                                device="cuda")
        self.refs, self.tables = ints(num_pages), ints(slots, max_pages, fill=-1)
        self.lens = ints(slots)
        self.cache = bsgemv.PageCache(2 * layers, num_pages, page_size * Hkv * D * 2, page_size,
                                      slots, max_pages)

    def plane(self, i):  # as attention reads it: [page][head][row][D]
        return self.pool[i].permute(0, 2, 1, 3)

    def call(self, entries):
        """entries: (slot, tokens) each, at most `rows` tokens in all.  Returns log probabilities of
        each entry's next token [n, vocab], and which entries found room (a tensor)."""
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        counts = [len(tokens) for _, tokens in entries]
        starts = ints([0] + counts).cumsum(0, dtype=torch.int32)
        seqs, grown = ints([slot for slot, _ in entries]), ints([0] * len(entries))
        self.cache.grow(self.pool, self.refs, self.tables, self.lens, seqs, starts, grown)
        seqs = torch.where(grown > 0, seqs, -1)  # the others' rows are padding
        tokens = torch.tensor([t for _, ts in entries for t in ts], device="cuda")
        T = tokens.shape[0]
        x = self.embed[tokens]
        for i, (qkv_of, o_of, experts) in enumerate(zip(self.qkv, self.o, self.experts)):
            qkv = qkv_of(norm(x)).view(T, Hq + 2 * Hkv, D)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            self.cache.append(self.rope, self.pool, self.tables, self.lens, seqs, starts, q, k, v, q,
                              head_stride=D, row_stride=Hkv * D, k_plane=2 * i, v_plane=2 * i + 1,
                              q_weight=self.norms[i][0], k_weight=self.norms[i][1])
            out = torch.empty(T, Hq, D, dtype=torch.float16, device="cuda")
            self.attn.run(q, self.plane(2 * i), self.plane(2 * i + 1), self.tables, self.lens, seqs,
                          starts, out, window=self.windows[i])
            x = x + o_of(out.view(T, Hq * D))
            x = x + experts(norm(x))
        last = x[starts[1:].long() - 1]
        return torch.log_softmax(self.head(norm(last)).float(), -1), grown

    def free(self, slots):
        self.cache.free(self.refs, self.tables, self.lens,
                        torch.tensor(slots, dtype=torch.int32, device="cuda"))

    def check(self):
        """Raises if a wait of a kernel ran out."""
        for plan in [self.attn] + [e.plan for e in self.experts]:
            status = plan.device_status()
            if status != 0:
                raise RuntimeError(bsgemv.status_string(status))


def serve(server: Server, prompts, tokens: int, rows: int | None = None):
    """`tokens` tokens after each prompt (a list of token lists): the lists of tokens, and the calls'
    row counts."""
    rows = min(rows or server.rows, server.rows)
    slots = server.lens.shape[0]
    waiting = list(range(len(prompts)))
    state = [None] * slots        # (prompt's number, its tokens still to come) of each slot
    made = [[] for _ in prompts]
    sizes = []
    while waiting or any(state):
        for s in range(slots):
            if state[s] is None and waiting:
                n = waiting.pop(0)
                state[s] = (n, list(prompts[n]))
        # one token of every sequence that decodes, then pieces of prompts
        order = sorted((s for s in range(slots) if state[s]), key=lambda s: len(state[s][1]) > 1)
        entries, left = [], rows
        for s in order:
            piece = state[s][1][:left]
            if piece:
                entries.append((s, piece))
                left -= len(piece)
        logp, grown = server.call(entries)
        sizes.append(rows - left)
        if not grown.all():
            raise RuntimeError("the cache's pages or a sequence's row ran out")
        best = logp.argmax(-1).tolist()
        for (s, piece), token in zip(entries, best):
            n, rest = state[s]
            rest = rest[len(piece):]
            if not rest:
                made[n].append(token)
                rest = [token]
            state[s] = (n, rest)
            if len(made[n]) == tokens:
                server.free([s])
                state[s] = None
    server.check()
    return made, sizes


def main() -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompts", type=int, default=6)
    ap.add_argument("--tokens", type=int, default=12)
    ap.add_argument("--rows", type=int, default=32)
    a = ap.parse_args()
    if a.prompts < 1 or a.tokens < 1 or not 4 <= a.rows <= 32:
        ap.error("a prompt and a token at least, 4 to 32 rows")
    server = Server(rows=a.rows)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(1024, (int(n),), generator=g).tolist()
               for n in torch.randint(5, 150, (a.prompts,), generator=g)]
    made, sizes = serve(server, prompts, a.tokens)
    for p, m in zip(prompts, made):
        print(f"{len(p):4d} tokens -> {m}")
    print(f"{len(sizes)} calls, {sum(sizes)} rows")
    return 0


if __name__ == "__main__":
    sys.exit(main())
