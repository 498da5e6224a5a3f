"""Tree-speculative decoding of a small hybrid model, every serving operator in
its place: one Gated DeltaNet layer and one softmax-attention layer with random
weights, several users who continue one shared prompt.

    prompt   prefill (DeltaNet state), chains through tree_attention, page_extend
             and kv_commit (paged keys and values)
    users    page_fork and page_copy, states forked by an empty prefill
    rounds   verify and tree_attention over a draft tree, accept, path, commit,
             page_extend and kv_commit of the accepted branch
    replay   the emitted tokens of one user again, one at a time, through step
             and single-token tree_attention
    end      page_free, page_compact, page_copy

Usage: python examples/serve_tree.py     (needs the built library and a GPU)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_tree_verify_amd as g  # noqa: E402

DEV = "cuda"
VOCAB, WIDTH = 96, 128
HEADS, DK = 4, 64                      # DeltaNet layer
QHEADS, KVHEADS, D = 4, 2, 64          # attention layer
PAGE, POOL, MAX_PAGES, SEQS = 16, 128, 32, 8
PARENT = [-1, 0, 0, 1, 1, 2, 3, 6]     # the shape of every draft tree
CHAIN = 64                             # prompt tokens per attention call


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    def __init__(self, seed):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        mat = lambda *s: torch.randn(*s, generator=gen, device=DEV) * s[0] ** -0.5
        self.embed = torch.randn(VOCAB, WIDTH, generator=gen, device=DEV)
        self.w_qkv, self.w_out = mat(WIDTH, 3 * HEADS * DK), mat(HEADS * DK, WIDTH)
        self.w_gate = mat(WIDTH, 2 * HEADS)
        self.a_qkv = mat(WIDTH, (QHEADS + 2 * KVHEADS) * D)
        self.a_out = mat(QHEADS * D, WIDTH)

    def delta_inputs(self, x):
        """q, k, v bf16 [..][HEADS][DK]; alpha, beta fp32 [..][HEADS]"""
        q, k, v = (x @ self.w_qkv).unflatten(-1, (3, HEADS, DK)).unbind(-3)
        unit = lambda y: (y / y.norm(dim=-1, keepdim=True)).bfloat16().contiguous()
        gate = x @ self.w_gate
        alpha = torch.exp(-torch.nn.functional.softplus(gate[..., :HEADS] - 2))
        beta = torch.sigmoid(gate[..., HEADS:]).contiguous()
        return unit(q), unit(k), v.bfloat16().contiguous(), alpha, beta

    def delta_output(self, x, o):
        return x + o.float().flatten(-2) @ self.w_out

    def attention_inputs(self, x):
        q, k, v = (x @ self.a_qkv).bfloat16().unflatten(-1, (QHEADS + 2 * KVHEADS, D)).split(
            (QHEADS, KVHEADS, KVHEADS), dim=-2)
        return q.contiguous(), k.contiguous(), v.contiguous()

    def logits(self, x, o):
        return (x + o.float().flatten(-2) @ self.a_out) @ self.embed.t()


class Server:
    def __init__(self, model, users):
        assert users % 4 == 0 and users + 2 <= SEQS     # rows are passed as aligned slices
        self.m, self.users, self.prompt, self.replay = model, users, users, users + 1
        self.S = torch.zeros(SEQS, HEADS, DK, DK, device=DEV)
        self.cache = torch.zeros(2, POOL, KVHEADS, PAGE, D, dtype=torch.bfloat16, device=DEV)
        self.table = torch.full((SEQS, MAX_PAGES), -1, dtype=torch.int32, device=DEV)
        self.length = torch.zeros(SEQS, dtype=torch.int32, device=DEV)
        self.ref = torch.zeros(POOL, dtype=torch.int32, device=DEV)

    def attend(self, x, parent, rows, shared=None):
        q, k, v = self.m.attention_inputs(x)
        pages, length = self.table[rows].contiguous(), self.length[rows].clone()
        o = g.tree_attention(q, k, v, parent, self.cache[0], self.cache[1], pages, length,
                             D ** -0.5, shared=shared)
        return o, k, v

    def append(self, rows, k, v, path, add):
        begin = g.page_extend(self.table, self.length, self.ref, rows, add, PAGE)
        g.kv_commit(self.cache[0], self.cache[1], self.table, rows, begin, k, v, path, add)

    def fork(self, src, dst):
        """rows and states dst continue src"""
        copies = g.page_fork(self.table, self.length, self.ref, src, dst, PAGE)
        g.page_copy(self.cache, copies)
        n = len(src)
        none = [torch.empty(0, HEADS, DK, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        gate = torch.empty(0, HEADS, device=DEV)
        g.prefill(*none, gate, gate, ints(*[0] * (n + 1)), self.S, src, dst)

    def read_prompt(self, tokens):
        """the prompt into row and state `prompt`; logits of its last token"""
        x = self.m.embed[tokens]
        row = ints(self.prompt)
        o = g.prefill(*self.m.delta_inputs(x), ints(0, len(tokens)), self.S, ints(-1), row)
        x = self.m.delta_output(x, o)[None]
        for t in range(0, len(tokens), CHAIN):
            part = x[:, t:t + CHAIN].contiguous()
            n = part.shape[1]
            chain = torch.arange(-1, n - 1, dtype=torch.int32, device=DEV)[None].contiguous()
            o, k, v = self.attend(part, chain, slice(self.prompt, self.prompt + 1))
            self.append(row, k, v, (chain + 1).contiguous(), ints(n))
        return self.m.logits(part, o)[0, -1]

    def round(self, tokens, parent, shared):
        """one draft tree per user: logits, accepted paths and the tokens after them"""
        users = slice(0, self.users)
        x = self.m.embed[tokens.long()]
        q, k, v, alpha, beta = self.m.delta_inputs(x)
        S = self.S[users]
        o = g.verify(q, k, v, alpha, beta, parent, S)
        h = self.m.delta_output(x, o)
        o, ak, av = self.attend(h, parent, users, shared)
        logits = self.m.logits(h, o)
        best = logits.argmax(-1).to(torch.int32)
        accepted, _, bonus = g.accept(parent, tokens, best)
        path, add = g.path(parent, accepted, parent.shape[1])
        g.commit(S, path, add, k, v, alpha, beta, parent)
        self.append(torch.arange(self.users, dtype=torch.int32, device=DEV), ak, av, path, add)
        return logits, path, add, bonus

    def one_token(self, token, src, row):
        """logits after one more token of a row, its state read from slot src"""
        x = self.m.embed[token.long()]
        o = g.step(*self.m.delta_inputs(x), self.S, src, row)
        h = self.m.delta_output(x, o)[:, None].contiguous()
        root = torch.full((1, 1), -1, dtype=torch.int32, device=DEV)
        o, k, v = self.attend(h, root, row.long())
        self.append(row, k, v, torch.zeros_like(root), ints(1))
        return self.m.logits(h, o)[0, 0]


def draft(model, root):
    """draft tokens of PARENT's tree: a node's children are the two tokens nearest to its own"""
    near = (model.embed @ model.embed.t()).topk(2, dim=-1).indices
    tokens = [root]
    for i, p in enumerate(PARENT[1:], 1):
        tokens.append(near[tokens[p].long(), PARENT[1:i].count(p) % 2].to(torch.int32))
    return torch.stack(tokens, dim=1).contiguous()


def serve(users=4, rounds=6, prompt_len=150, seed=0):
    model = Model(seed)
    s = Server(model, users)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 1)
    prompt = torch.randint(VOCAB, (prompt_len,), generator=gen, device=DEV)
    first = s.read_prompt(prompt).topk(users).indices.to(torch.int32)      # one start a user
    rows = torch.arange(users, dtype=torch.int32, device=DEV)
    s.fork(torch.full_like(rows, s.prompt), rows)
    parent = ints(*PARENT).repeat(users, 1)
    shared = (ints(0, users), ints(prompt_len // PAGE * PAGE))
    root, emitted, seen = first, [[] for _ in range(users)], []
    for _ in range(rounds):
        tokens = draft(model, root)
        logits, path, add, bonus = s.round(tokens, parent, shared)
        for u in range(users):
            nodes = path[u, : int(add[u])].long()
            emitted[u] += tokens[u, nodes].tolist()
            if u == 0:
                seen.append(logits[0, nodes])
        root = bonus
    # user 0's tokens once more, one at a time
    again = []
    s.fork(ints(s.prompt), ints(s.replay))
    for t in emitted[0]:
        again.append(s.one_token(ints(t), ints(s.replay), ints(s.replay)))
    held = s.table[0, : (int(s.length[0]) + PAGE - 1) // PAGE].long()
    before = s.cache[:, held].clone()
    g.page_free(s.table, s.length, s.ref, ints(s.replay, 1), PAGE)
    copies, count = g.page_compact(s.table, s.length, s.ref, PAGE)
    g.page_copy(s.cache, copies, count)
    held = s.table[0, : held.numel()].long()
    used = int((s.ref != 0).sum())
    return dict(emitted=emitted, logits=torch.cat(seen), again=torch.stack(again), model=model,
                server=s, moved=int(count), dense=bool((s.ref[:used] > 0).all()),
                kept=bool(torch.equal(before, s.cache[:, held])), used=used)


def main():
    r = serve()
    n = [len(e) for e in r["emitted"]]
    diff = (r["logits"] - r["again"]).abs().max()
    print(f"tokens per user {n}, tree against single tokens: logits differ by {diff:.2g}; "
          f"{r['used']} pages in use, {r['moved']} moved by compaction")


if __name__ == "__main__":
    main()
