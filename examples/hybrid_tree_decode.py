"""Speculative decoding of a small hybrid model (a Mamba2 layer and an attention layer) with drafted trees.

Every step runs a tree of drafted tokens per request through both layers in one pass, keeps the longest
path that greedy decoding would have taken, and goes on from there:

  kv_block_tables     blocks, slots and positions of the step's tokens, from lengths on the GPU
  ssm_decode_update   the Mamba2 layer, one tree level per call: a node reads its parent's state slot
                      and writes its own
  kv_qk_norm_rope     norms and rotation of the attention layer's queries and keys
  kv_tree_attention   a node attends to the cache and to its ancestors
  kv_commit_tokens    keys and values of the kept path to the cache

Weights and drafts are random; the drafts hold the right continuation often enough to be kept.

    python examples/hybrid_tree_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_mamba2_gb300 as ssd  # noqa: E402

VOCAB, WIDTH = 512, 256
SSM_HEADS, SSM_P, SSM_N = 4, 64, 128
HEADS, KV_HEADS, HEAD_DIM = 4, 2, 64
BLOCK = 16
# a node's parent: two chains of three from the root, the first forking once more
PARENTS = [-1, 0, 1, 2, 0, 4, 1]
NODES = len(PARENTS)


def _depth(i):
    return 0 if PARENTS[i] < 0 else 1 + _depth(PARENTS[i])


DEPTHS = [_depth(i) for i in range(NODES)]


class HybridModel:
    """Weights and caches of the two layers for ``requests`` requests."""

    def __init__(self, requests, max_len, dtype=torch.float32, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)

        self.dtype, self.device, self.requests = dtype, device, requests
        self.embed = rand(VOCAB, WIDTH)
        inner = SSM_HEADS * SSM_P
        self.ssm_in = rand(WIDTH, inner + 2 * SSM_N + SSM_HEADS, scale=WIDTH ** -0.5)
        self.ssm_out = rand(inner, WIDTH, scale=inner ** -0.5)
        self.A = -torch.exp(torch.rand(SSM_HEADS, generator=g, device=device))
        self.D = torch.randn(SSM_HEADS, generator=g, device=device)
        self.qkv = rand(WIDTH, (HEADS + 2 * KV_HEADS) * HEAD_DIM, scale=WIDTH ** -0.5)
        self.attn_out = rand(HEADS * HEAD_DIM, WIDTH, scale=(HEADS * HEAD_DIM) ** -0.5)
        self.q_weight = 1 + 0.1 * torch.randn(HEAD_DIM, generator=g, device=device)
        self.k_weight = 1 + 0.1 * torch.randn(HEAD_DIM, generator=g, device=device)
        angle = torch.arange(max_len + NODES, device=device)[:, None] * \
            (10000.0 ** (-torch.arange(0, HEAD_DIM, 2, device=device) / HEAD_DIM))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        # Mamba2 states: a slot per request and tree node, and one for where the request stands (slot 0 is null)
        self.states = torch.zeros(1 + requests * (NODES + 1), SSM_HEADS, SSM_P, SSM_N, device=device)
        self.first_slot = 1 + torch.arange(requests, device=device) * (NODES + 1)
        self.stand = self.first_slot.int()
        # attention cache: pages, block table, the ring of free blocks (block 0 is null)
        cols = -(-(max_len + NODES) // BLOCK)
        self.blocks = 1 + requests * cols
        self.k_cache = torch.zeros(self.blocks, BLOCK, KV_HEADS, HEAD_DIM, dtype=dtype, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = torch.zeros(requests, cols, dtype=torch.int32, device=device)
        self.ring = torch.arange(1, self.blocks, device=device).int()
        self.ring_state = torch.tensor([0, self.blocks - 1], device=device).int()
        self.context = torch.zeros(requests, device=device).int()
        self.reserved = torch.zeros(requests, device=device).int()
        self.error = torch.zeros(1, dtype=torch.int32, device=device)

    def ssm_layer(self, h, parents, node_slots):
        """h [R, n, WIDTH]: the tree's levels one after the other; node i reads its parent's state."""
        R, n, _ = h.shape
        inner = SSM_HEADS * SSM_P
        z = h @ self.ssm_in
        x, B, C, dt = z.split([inner, SSM_N, SSM_N, SSM_HEADS], -1)
        y = torch.empty(R, n, SSM_HEADS, SSM_P, dtype=self.dtype, device=self.device)
        depths = []
        for p in parents:
            depths.append(0 if p < 0 else depths[p] + 1)
        for d in range(max(depths) + 1):
            level = [i for i in range(n) if depths[i] == d]
            read = [self.stand if parents[i] < 0 else node_slots[:, parents[i]] for i in level]
            rows = torch.stack([torch.stack([node_slots[:, i] for i in level], 1), torch.stack(read, 1)], -1)
            rows = rows.reshape(-1, 2).int().contiguous()  # column 0: written, column 1: resumed from
            one = torch.ones(rows.shape[0], dtype=torch.int32, device=self.device)
            out = ssd.ssm_decode_update(
                x[:, level].reshape(-1, SSM_HEADS, SSM_P).contiguous(), dt[:, level].reshape(-1, SSM_HEADS).contiguous(),
                self.A, B[:, level].reshape(-1, 1, SSM_N).contiguous(), C[:, level].reshape(-1, 1, SSM_N).contiguous(),
                self.states, rows, num_accepted_tokens=one, D=self.D, err_word=self.error)
            y[:, level] = out.view(R, len(level), SSM_HEADS, SSM_P)
        return h + y.reshape(R, n, inner) @ self.ssm_out

    def attention_layer(self, h, depths, mask, tables):
        """h [R, n, WIDTH]; returns the layer's output and the new keys and values."""
        R, n, _ = h.shape
        T = R * n
        z = (h @ self.qkv).view(T, -1)
        q, k, v = (t.unflatten(1, (-1, HEAD_DIM)) for t in
                   z.split([HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM], 1))
        position = (self.context[:, None] + depths[None, :]).int().flatten()  # a node's place on its path
        q, k = ssd.kv_qk_norm_rope(q, k, position, self.cos_sin, self.q_weight, self.k_weight, err_word=self.error)
        o = ssd.kv_tree_attention(q, k, v, self.k_cache, self.v_cache, tables["cu_seqlens"], self.context, self.table,
                                  max_new_tokens=n, tree_mask=mask, err_word=self.error)
        return h + (o.view(T, -1) @ self.attn_out).view(R, n, -1), k, v

    def step(self, tokens, parents):
        """Runs a tree of tokens ([R, n], node 0 the last certain token) and keeps the path greedy decoding takes.
        Returns (tokens decoded after each node [R, n], kept path [R, longest], its length [R])."""
        R, n = tokens.shape
        dev = self.device
        depths = []
        ancestors = torch.zeros(n, n, dtype=torch.bool)
        for i, p in enumerate(parents):
            depths.append(0 if p < 0 else depths[p] + 1)
            if p >= 0:
                ancestors[i] = ancestors[p]
            ancestors[i, i] = True
        mask = (ancestors.long() << torch.arange(n)).sum(1).int().to(dev).repeat(R)[:, None].contiguous()
        depths = torch.tensor(depths, device=dev)
        new = torch.full((R,), n, dtype=torch.int32, device=dev)
        tables = ssd.kv_block_tables(self.context, new, self.reserved, self.table, self.ring, self.ring_state, BLOCK,
                                     self.blocks, R * n, err_word=self.error)
        self.reserved, self.ring_state = tables["reserved_lens"], tables["ring_state"]

        # the request's slots behind the one it stands on, in turn
        turn = (self.stand - self.first_slot)[:, None] + 1 + torch.arange(n, device=dev)
        node_slots = self.first_slot[:, None] + turn % (NODES + 1)
        h = self.embed[tokens]
        h = self.ssm_layer(h, parents, node_slots)
        h, k, v = self.attention_layer(h, depths, mask, tables)
        decoded = (h @ self.embed.T).float().argmax(-1)

        # the kept path: from node 0 on to a child that holds what was decoded, as long as there is one
        tok, dec = tokens.tolist(), decoded.tolist()
        paths = []
        for r in range(R):
            path = [0]
            while True:
                nxt = [i for i in range(n) if parents[i] == path[-1] and tok[r][i] == dec[r][path[-1]]]
                if not nxt:
                    break
                path.append(nxt[0])
            paths.append(path)
        longest = max(len(p) for p in paths)
        path = torch.tensor([p + [0] * (longest - len(p)) for p in paths], dtype=torch.int32, device=dev)
        lens = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
        self.context = ssd.kv_commit_tokens(k, v, self.k_cache, self.v_cache, tables["slots"], tables["cu_seqlens"],
                                            self.context, path=path, path_lens=lens, err_word=self.error)
        last = path.gather(1, (lens - 1).long()[:, None])[:, 0].long()
        self.stand = node_slots.gather(1, last[:, None])[:, 0].int()
        return decoded, path, lens


def decode(requests=3, length=24, speculate=True, dtype=torch.float32, seed=0, hints=None):
    """Greedy decoding of ``length`` tokens per request; returns (tokens [requests, length], steps taken).  ``hints``:
    the tokens of an earlier run, which the drafts then hold now and then."""
    model = HybridModel(requests, length + 1, dtype, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    out = [[int(t)] for t in torch.randint(VOCAB, (requests,), generator=g)]
    steps = 0
    while min(len(o) for o in out) < length:
        parents = PARENTS if speculate else [-1]
        tree = torch.randint(VOCAB, (requests, len(parents)), generator=g)
        for r, o in enumerate(out):
            tree[r, 0] = o[-1]
            if hints is not None and speculate:
                for i in range(1, len(parents)):
                    if torch.rand(1, generator=g) < 0.7:
                        tree[r, i] = int(hints[r, min(len(o) - 1 + DEPTHS[i], hints.shape[1] - 1)])
        decoded, path, lens = model.step(tree.cuda(), parents)
        for r, o in enumerate(out):
            o += [int(decoded[r, int(i)]) for i in path[r, :int(lens[r])]]
        steps += 1
        for r, o in enumerate(out):  # requests at their end idle on; their cache must not overflow
            del o[length + 1:]
        if max(int(c) for c in model.context) > length - 1:
            break
    assert int(model.error.item()) == 0, "device error word %d" % int(model.error.item())
    n = min(min(len(o) for o in out), length)
    return torch.tensor([o[:n] for o in out]), steps


def main():
    plain, plain_steps = decode(speculate=False)
    drafted, steps = decode(hints=plain)
    n = min(plain.shape[1], drafted.shape[1])
    same = bool((plain[:, :n] == drafted[:, :n]).all())
    print("%d tokens per request: %d single-token steps, %d steps with drafted trees, same tokens: %s"
          % (n, plain_steps, steps, same))
    return same, n, plain_steps, steps


if __name__ == "__main__":
    ssd.build()
    main()
