"""The model of serve_tree.py with rotary positions, normalised queries and keys,
and greedy tokens under penalties: tree-speculative decoding through the
operators between a model's projections and the library's other calls.

    prompt   kv_append (norm and rotation on the way into the pages, queries and
             keys beside them), tree_attention, count_prompt
    rounds   index and qk_norm_rope (a node's position is its user's length and
             its depth), verify, tree_attention, adjust_logits, accept, path,
             commit, page_extend, kv_commit, count_commit
    replay   one user's tokens again, one at a time: step, page_extend,
             kv_append, tree_attention, adjust_logits, count_commit

Usage: python examples/serve_rotary.py     (needs the built library and a GPU)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_tree as base  # noqa: E402
from serve_tree import D, KVHEADS, PAGE, QHEADS, SEQS, VOCAB, g, ints  # noqa: E402

DEV = "cuda"
REPETITION, PRESENCE, FREQUENCY = 1.3, 0.5, 0.25


class RotaryServer(base.Server):
    def __init__(self, model, users, seed):
        super().__init__(model, users)
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        weight = lambda: 1 + 0.1 * torch.randn(D, generator=gen, device=DEV)
        self.q_weight, self.k_weight = weight(), weight()
        # half of each head is rotated, for four times the context of 64 tokens
        self.inv_freq, self.magnitude = g.rope_frequencies(D // 2, scaling="yarn", factor=4,
                                                           original=64, low=1, high=8)
        self.counts = torch.zeros(SEQS, VOCAB, dtype=torch.int16, device=DEV)

    def project(self, x):
        """queries, keys and values as views of one projection"""
        return (x @ self.m.a_qkv).bfloat16().unflatten(-1, (QHEADS + 2 * KVHEADS, D)).split(
            (QHEADS, KVHEADS, KVHEADS), dim=-2)

    def append_and_attend(self, x, row, parent, cu=None):
        """x [n][width]: n more tokens of a row, into its pages; their attention"""
        n = x.shape[0]
        q, k, v = self.project(x)
        begin = g.page_extend(self.table, self.length, self.ref, row, ints(n), PAGE)
        keys = torch.empty(k.shape, dtype=k.dtype, device=DEV)
        queries, _ = g.kv_append(self.cache[0], self.cache[1], self.table, row, begin, k, v, cu=cu,
                                 inv_freq=self.inv_freq, scale=self.magnitude, norm="rms",
                                 k_weight=self.k_weight, q=q, q_weight=self.q_weight, k_out=keys)
        pages = self.table[row.long()].contiguous()
        return g.tree_attention(queries[None], keys[None], v.contiguous()[None], parent,
                                self.cache[0], self.cache[1], pages, begin, D ** -0.5)

    def fork(self, src, dst):
        super().fork(src, dst)
        self.counts[dst.long()] = self.counts[src.long()]

    def pick(self, logits, rows, tokens, parent):
        """the greedy tokens under penalties, and the logits that they are from"""
        many = lambda x: torch.full((rows.numel(),), x, device=DEV)
        out = torch.empty_like(logits)
        best = g.adjust_logits(logits, counts=self.counts, slot=rows, tokens=tokens, parent=parent,
                               repetition=many(REPETITION), presence=many(PRESENCE),
                               frequency=many(FREQUENCY), out=out)
        return best, out

    def read_prompt(self, tokens):
        x = self.m.embed[tokens]
        row, n = ints(self.prompt), len(tokens)
        o = g.prefill(*self.m.delta_inputs(x), ints(0, n), self.S, ints(-1), row)
        x = self.m.delta_output(x, o)
        for t in range(0, n, base.CHAIN):
            part = x[t:t + base.CHAIN]
            m = part.shape[0]
            chain = torch.arange(-1, m - 1, dtype=torch.int32, device=DEV)[None].contiguous()
            o = self.append_and_attend(part, row, chain, ints(0, m))
        g.count_prompt(self.counts, row, ints(0, n), tokens.to(torch.int32))
        return self.m.logits(part[None], o)[0, -1]

    def round(self, tokens, parent, shared):
        rows = torch.arange(self.users, dtype=torch.int32, device=DEV)
        x = self.m.embed[tokens.long()]
        dq, dk, dv, alpha, beta = self.m.delta_inputs(x)
        S = self.S[:self.users]
        h = self.m.delta_output(x, g.verify(dq, dk, dv, alpha, beta, parent, S))
        q, k, v = self.project(h)
        length = self.length[:self.users].clone()
        depth, _ = g.index(parent)
        q, k = g.qk_norm_rope(q, k, self.q_weight, self.k_weight, depth, self.inv_freq,
                              scale=self.magnitude, base=length)
        v = v.contiguous()
        o = g.tree_attention(q, k, v, parent, self.cache[0], self.cache[1],
                             self.table[:self.users].contiguous(), length, D ** -0.5, shared=shared)
        best, logits = self.pick(self.m.logits(h, o), rows, tokens, parent)
        accepted, _, bonus = g.accept(parent, tokens, best)
        path, add = g.path(parent, accepted, parent.shape[1])
        g.commit(S, path, add, dk, dv, alpha, beta, parent)
        self.append(rows, k, v, path, add)
        g.count_commit(self.counts, rows, tokens, path, add)
        return logits, path, add, bonus

    def one_token(self, token, src, row):
        x = self.m.embed[token.long()]
        h = self.m.delta_output(x, g.step(*self.m.delta_inputs(x), self.S, src, row))
        root = torch.full((1, 1), -1, dtype=torch.int32, device=DEV)
        o = self.append_and_attend(h, row, root)
        best, logits = self.pick(self.m.logits(h[None], o), row, token[None], root)
        g.count_commit(self.counts, row, token[None], torch.zeros_like(root), ints(1))
        return best[0, 0], logits[0, 0]


def serve(users=4, rounds=6, prompt_len=150, seed=0):
    model = base.Model(seed)
    s = RotaryServer(model, users, seed + 2)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 1)
    prompt = torch.randint(VOCAB, (prompt_len,), generator=gen, device=DEV)
    root = s.read_prompt(prompt).topk(users).indices.to(torch.int32)
    rows = torch.arange(users, dtype=torch.int32, device=DEV)
    s.fork(torch.full_like(rows, s.prompt), rows)
    parent = ints(*base.PARENT).repeat(users, 1)
    shared = (ints(0, users), ints(prompt_len // PAGE * PAGE))
    emitted, seen, picked = [[] for _ in range(users)], [], []
    for _ in range(rounds):
        tokens = base.draft(model, root)
        logits, path, add, bonus = s.round(tokens, parent, shared)
        for u in range(users):
            nodes = path[u, : int(add[u])].long()
            emitted[u] += tokens[u, nodes].tolist()
            if u == 0:
                seen.append(logits[0, nodes])
                picked += tokens[0, nodes[1:]].tolist() + [int(bonus[0])]
        root = bonus
    # user 0's tokens once more, one at a time
    s.fork(ints(s.prompt), ints(s.replay))
    again = [s.one_token(ints(t), ints(s.replay), ints(s.replay)) for t in emitted[0]]
    return dict(emitted=emitted, logits=torch.cat(seen), again=torch.stack([x for _, x in again]),
                picked=picked, best=[int(b) for b, _ in again], model=model, server=s)


def main():
    r = serve()
    diff = (r["logits"] - r["again"]).abs().max()
    same = sum(a == b for a, b in zip(r["picked"], r["best"]))
    print(f"tokens per user {[len(e) for e in r['emitted']]}, tree against single tokens: "
          f"adjusted logits differ by {diff:.2g}, {same} of {len(r['best'])} greedy tokens alike")


if __name__ == "__main__":
    main()
