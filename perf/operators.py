"""Measured cases of the attention-side serving operators: block tables and slot maps built on the
GPU (``kv_block_tables``), per-head norms of queries and keys with the position rotation
(``kv_qk_norm_rope``), attention of drafted tokens over a paged cache (``kv_tree_attention``) and the
commit of accepted tokens to that cache (``kv_commit_tokens``).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once
at the end) unless ``own`` is true; then it makes the calls a user makes of the library."""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one step of a speculative batch: 256 requests of 1 + 3 tokens, the ordinary decode bookkeeping
        dict(name="tables_spec", op="tables", reqs=256, new_lo=4, new_hi=4, ctx_lo=1, ctx_hi=8192, block=64, dense=0),
        # the long mixed batch: 8 prompts of 65536 tokens beside 384 single-token requests
        dict(name="tables_mixed", op="tables", reqs=392, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=65536, block=16, dense=8),
        # a handful of decode tokens of an fp32 model with odd head sizes and a partial rotation: a latency case
        dict(name="rope_odd", op="rope", tokens=37, hq=12, hkv=4, d=80, rot=40, type="f32", inter=0, block=24),
        # a prefill step of 65536 packed tokens, bf16, the rotation over the whole head
        dict(name="rope_prompt", op="rope", tokens=65536, hq=32, hkv=8, d=128, rot=128, type="bf16", inter=0, block=64),
        # after a tree step: accepted paths of at most 5 of 16 drafted tokens for 256 requests
        dict(name="commit_tree", op="commit", reqs=256, nodes=16, path=5, hkv=8, d=128, type="bf16", block=64),
        # a prompt's keys and values written to the cache as they are: 32768 tokens
        dict(name="commit_prompt", op="commit", reqs=8, nodes=4096, path=0, hkv=8, d=128, type="bf16", block=16),
        # one token of one short request: the smallest decode call
        dict(name="attn_one", op="attn", reqs=1, q_lo=1, q_hi=1, ctx_lo=777, ctx_hi=777, hq=32, hkv=8, d=128,
             type="bf16", block=16, tree=0),
        # one token of one long request (65536 cached): the cache has to be split over the GPU
        dict(name="attn_long", op="attn", reqs=1, q_lo=1, q_hi=1, ctx_lo=65536, ctx_hi=65536, hq=32, hkv=8, d=128,
             type="bf16", block=256, tree=0),
        # the speculative batch: 256 requests of 1 + 3 tokens over ragged caches
        dict(name="attn_spec", op="attn", reqs=256, q_lo=4, q_hi=4, ctx_lo=0, ctx_hi=8192, hq=32, hkv=8, d=128,
             type="bf16", block=64, tree=0),
        # verification of ragged trees of up to 64 drafted tokens, 8 query heads to a key head
        dict(name="attn_tree", op="attn", reqs=24, q_lo=33, q_hi=64, ctx_lo=0, ctx_hi=16384, hq=32, hkv=4, d=128,
             type="bf16", block=32, tree=1),
        # a chunk of prompts behind cached prefixes: new tokens attend to the prefix and to one another
        dict(name="attn_prompt", op="attn", reqs=4, q_lo=512, q_hi=4096, ctx_lo=0, ctx_hi=8192, hq=32, hkv=8, d=128,
             type="bf16", block=64, tree=0),
        # small fp32 trees over pages of an odd size
        dict(name="attn_f32", op="attn", reqs=16, q_lo=1, q_hi=7, ctx_lo=0, ctx_hi=2000, hq=16, hkv=4, d=64,
             type="f32", block=24, tree=1),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    return v - 1 if v == 3 * 1024 else v


def draw(rng):
    """One more case of the listed ranges: requests, lengths, heads, types, page sizes and masks."""
    op = rng.choice(["tables", "rope", "commit", "attn", "attn", "attn"])
    block = rng.choice([8, 16, 16, 24, 32, 48, 64, 128, 256])
    if op == "tables":
        return dict(op=op, reqs=_log(rng, 1, 1024), new_lo=0, new_hi=_log(rng, 1, 256), ctx_lo=0,
                    ctx_hi=_log(rng, 64, 65536), block=block, dense=rng.choice([0, 0, 1, 3]))
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "rope":
        d = rng.choice([64, 80, 112, 128, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]),
                    type=dtype, inter=rng.choice([0, 1]), block=block)
    d = rng.choice([64, 128, 128])
    if op == "commit":
        nodes = _log(rng, 1, 512)
        return dict(op=op, reqs=_log(rng, 1, 64), nodes=nodes, path=rng.choice([0, min(nodes, 6)]), hkv=hkv, d=d,
                    type=dtype, block=block)
    if dtype == "f32":  # the CUDA-core path: small batches
        return dict(op=op, reqs=_log(rng, 1, 16), q_lo=1, q_hi=_log(rng, 1, 8), ctx_lo=0, ctx_hi=_log(rng, 64, 2048),
                    hq=hq, hkv=hkv, d=d, type=dtype, block=block, tree=rng.choice([0, 1]))
    kind = rng.choice(["decode", "tree", "prompt"])
    if kind == "decode":
        return dict(op=op, reqs=_log(rng, 1, 128), q_lo=1, q_hi=rng.choice([1, 2, 4, 8]), ctx_lo=0,
                    ctx_hi=_log(rng, 64, 8192), hq=hq, hkv=hkv, d=d, type=dtype, block=block, tree=0)
    if kind == "tree":
        return dict(op=op, reqs=_log(rng, 1, 24), q_lo=1, q_hi=_log(rng, 2, 64), ctx_lo=0, ctx_hi=_log(rng, 64, 16384),
                    hq=min(hq, 32), hkv=hkv, d=d, type=dtype, block=block, tree=1)
    return dict(op=op, reqs=_log(rng, 1, 4), q_lo=1, q_hi=_log(rng, 16, 2048), ctx_lo=0, ctx_hi=_log(rng, 64, 8192),
                hq=min(hq, 32), hkv=hkv, d=d, type=dtype, block=block, tree=0)


def _lens(case):
    """Request lengths of a case; they are a property of the case, not of the seed of its values."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["reqs"]
    if case["op"] == "tables":
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
        for r in range(min(case["dense"], n)):  # prompts
            new[r], ctx[r] = 65536, 0
        return new, ctx
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    if n > 1:
        ctx[0] = 0  # a request with nothing cached
        new[-1], ctx[-1] = case["q_hi"], case["ctx_hi"]
    return new, ctx


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "tables":
        new, ctx = _lens(case)
        b, n, t = case["block"], case["reqs"], sum(new)
        touched = sum(_cdiv(c + m, b) - c // b for c, m in zip(ctx, new) if m)
        return {"bytes": 24 * n + 16 + 12 * t + 8 * touched, "flops": 0}
    e = 2 if case["type"] == "bf16" else 4
    if op == "rope":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        return {"bytes": t * d * e * (2 * hq + 2 * hkv) + t * 3 * hkv * d * e + t * case["rot"] * 4 + 8 * t,
                "flops": t * (hq + hkv) * d * 8}
    if op == "commit":
        rows = case["reqs"] * (case["path"] or case["nodes"])
        return {"bytes": rows * case["hkv"] * case["d"] * e * 4 + 8 * rows, "flops": 0}
    new, ctx = _lens(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t = sum(new)
    # a tree's tokens see themselves at least; a chain's every token before them
    pairs = sum(m * c + (m if case["tree"] else m * (m + 1) // 2) for c, m in zip(ctx, new))
    return {"bytes": (sum(ctx) + t) * hkv * d * 2 * e + 2 * t * hq * d * e + 4 * t * hq
            + (t * 4 * _cdiv(max(new), 32) if case["tree"] else 0), "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------- inputs --

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _tables(g, lens, block, spare, cols):
    """Block ids of requests whose blocks are scattered over the cache: [reqs, cols], and the number of blocks."""
    need = [_cdiv(n, block) for n in lens]
    total = sum(need) + spare + 1
    perm = torch.randperm(total - 1, generator=g, device=DEV, dtype=torch.int32) + 1  # block 0 stays the null block
    held = _ints(need)
    start = torch.cumsum(held, 0) - held
    col = torch.arange(cols, device=DEV)
    index = (start[:, None] + col[None, :]).clamp(max=max(total - 2, 0))
    return torch.where(col[None, :] < held[:, None], perm[index], 0).to(torch.int32), total, perm[sum(need):]


def _tree_bits(rng, sizes, words):
    """Ancestor masks of random trees, one row of 32-bit words for each token."""
    rows = []
    for r, n in enumerate(sizes):
        masks = []
        for i in range(n):
            up = masks[rng.randrange(max(0, i - 6), i)] if i else 0
            masks.append(up | (1 << i))
        if r == 0 and n > 1:
            masks[-1] = 0  # a padded token that sees none of the new ones
        rows += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in masks]
    rows = [[v - (1 << 32) if v >= (1 << 31) else v for v in row] for row in rows]
    return _ints(rows)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    rng = random.Random(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "tables":
        new, ctx = _lens(case)
        b = case["block"]
        top = max(c + m for c, m in zip(ctx, new)) + 1
        cols = _cdiv(top, b) + 1
        extra = sum(_cdiv(c + m, b) - _cdiv(c, b) for c, m in zip(ctx, new))
        table, total, free = _tables(g, ctx, b, extra + 5, cols)
        cap = free.numel() + 3
        head = rng.randrange(cap)
        ring = torch.zeros(cap, dtype=torch.int32, device=DEV)
        ring[(torch.arange(free.numel(), device=DEV) + head) % cap] = free
        s.update(ctx=_ints(ctx), new=_ints(new), reserved=_ints(ctx), table=table, ring=ring,
                 state=_ints([head, free.numel()]), blocks=total, max_tokens=sum(new) + 13)
        return s
    dtype = TYPES[case["type"]]
    hkv, d, b = case["hkv"], case["d"], case["block"]
    if op == "rope":
        t, hq, rot = case["tokens"], case["hq"], case["rot"]
        blocks = _cdiv(t, b) + 2
        qkv = _randn(g, (t, (hq + 2 * hkv) * d), dtype)  # one packed projection, read through views
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        s["qw"] = 1 + 0.1 * _randn(g, (d,), torch.float32)
        s["kw"] = 1 + 0.1 * _randn(g, (d,), torch.float32)
        top = 8192
        angle = torch.arange(top, device=DEV)[:, None] * (10000.0 ** (-torch.arange(0, rot, 2, device=DEV) / rot))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        first = rng.randrange(top)
        s["positions"] = ((torch.arange(t, device=DEV) + first) % top).to(torch.int32)
        s["slots"] = torch.randperm(blocks * b, generator=g, device=DEV)[:t].to(torch.int32)
        s["kc"] = torch.zeros((blocks, b, hkv, d), dtype=dtype, device=DEV)
        s["vc"] = torch.zeros((blocks, b, hkv, d), dtype=dtype, device=DEV)
        return s
    if op == "commit":
        n, nodes, path = case["reqs"], case["nodes"], case["path"]
        t = n * nodes
        blocks = _cdiv(t, b) + 2
        kv = _randn(g, (t, 2 * hkv * d), dtype)
        s["k"], s["v"] = kv[:, :hkv * d].view(t, hkv, d), kv[:, hkv * d:].view(t, hkv, d)
        s["kc"] = torch.zeros((blocks, b, hkv, d), dtype=dtype, device=DEV)
        s["vc"] = torch.zeros((blocks, b, hkv, d), dtype=dtype, device=DEV)
        s["slots"] = torch.randperm(blocks * b, generator=g, device=DEV)[:t].to(torch.int32)
        s["cu"] = _ints([i * nodes for i in range(n + 1)])
        s["ctx"] = _ints([rng.randrange(8192) for _ in range(n)])
        if path:
            s["path"] = _ints([sorted(rng.sample(range(nodes), path)) for _ in range(n)])
            s["lens"] = _ints([rng.randint(1, path) for _ in range(n)])
        return s
    new, ctx = _lens(case)
    hq, t, n = case["hq"], sum(new), case["reqs"]
    cols = _cdiv(max(ctx), b) + 1
    s["table"], blocks, _ = _tables(g, ctx, b, 3, cols)
    qkv = _randn(g, (t, (hq + 2 * hkv) * d), dtype)
    s["q"] = qkv[:, :hq * d].view(t, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    s["kc"] = _randn(g, (blocks, b, hkv, d), dtype)
    s["vc"] = _randn(g, (blocks, b, hkv, d), dtype)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s["cu"], s["ctx"], s["max_new"], s["max_ctx"] = _ints(cu), _ints(ctx), max(new), max(ctx)
    s["mask"] = _tree_bits(rng, new, _cdiv(max(new), 32)) if case["tree"] else None
    return s


# ------------------------------------------------------------ plain forms --

def _plain_tables(s):
    b, cap, top = s["case"]["block"], s["ring"].numel(), s["max_tokens"]
    ctx, new, held0, table = s["ctx"].long(), s["new"].long(), s["reserved"].long(), s["table"]
    n, cols = table.shape
    total = ctx + new
    held = (held0 + b - 1) // b
    need = torch.maximum(held, (total + b - 1) // b)
    pops = need - held
    before = torch.cumsum(pops, 0) - pops
    col = torch.arange(cols, device=DEV)[None, :]
    taken = (col >= held[:, None]) & (col < need[:, None])
    entry = (s["state"][0] + before[:, None] + col - held[:, None]).remainder(cap)
    table.copy_(torch.where(taken, s["ring"][entry], table))
    popped = pops.sum()
    state = torch.stack([(s["state"][0] + popped).remainder(cap), s["state"][1] - popped]).to(torch.int32)
    ends = torch.cumsum(new, 0)
    cu = torch.cat([ends.new_zeros(1), ends])
    tok = torch.arange(top, device=DEV)
    live = tok < cu[-1]
    req = torch.searchsorted(ends, tok, right=True).clamp(max=n - 1)
    pos = torch.where(live, ctx[req] + tok - cu[req], 0)
    slot = torch.where(live, table[req, (pos // b).clamp(max=cols - 1)] * b + pos % b, -1)
    i32 = torch.int32
    return [table, cu.to(i32), total.to(i32), torch.maximum(held0, total).to(i32), state, slot.to(i32), pos.to(i32),
            torch.where(live, req, -1).to(i32)]


def _rotate(x, cos, sin, rot, inter):
    """x [T, H, D] with its first rot entries rotated in pairs."""
    part, rest = x[..., :rot], x[..., rot:]
    if inter:
        a, c = part[..., 0::2], part[..., 1::2]
        return torch.cat([torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2), rest], -1)
    a, c = part[..., :rot // 2], part[..., rot // 2:]
    return torch.cat([a * cos - c * sin, c * cos + a * sin, rest], -1)


def _plain_rope(s):
    rot, inter, dtype = s["case"]["rot"], s["case"]["inter"], s["q"].dtype
    table = s["cos_sin"][s["positions"].long()]
    cos, sin = table[:, None, :rot // 2], table[:, None, rot // 2:]
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["qw"]
    k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["kw"]
    q, k = _rotate(q, cos, sin, rot, inter).to(dtype), _rotate(k, cos, sin, rot, inter).to(dtype)
    slots = s["slots"].long()
    s["kc"].view(-1, *k.shape[1:])[slots] = k
    s["vc"].view(-1, *k.shape[1:])[slots] = s["v"]
    return [q, k, s["kc"], s["vc"]]


def _plain_commit(s):
    kc, vc = s["kc"].view(-1, *s["k"].shape[1:]), s["vc"].view(-1, *s["v"].shape[1:])
    if "path" not in s:
        slots = s["slots"].long()
        kc[slots], vc[slots] = s["k"], s["v"]
        return [s["kc"], s["vc"], s["ctx"] + (s["cu"][1:] - s["cu"][:-1])]
    path, cu = s["path"].long(), s["cu"][:-1].long()[:, None]
    step = torch.arange(path.shape[1], device=DEV)[None, :]
    live = step < s["lens"][:, None]
    # the steps beyond a path repeat its first one
    src, dst = cu + torch.where(live, path, path[:, :1]), s["slots"][cu + torch.where(live, step, 0)].long()
    kc[dst], vc[dst] = s["k"][src], s["v"][src]
    return [s["kc"], s["vc"], s["ctx"] + s["lens"]]


def _plain_attn(s):
    case = s["case"]
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["block"]
    n, group, most, past = case["reqs"], hq // hkv, s["max_new"], s["max_ctx"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    new = cu[1:] - cu[:-1]
    # queries and new keys padded to the longest request: [n, most, heads, d]
    step = torch.arange(most, device=DEV)
    tok = (cu[:-1, None] + step[None, :]).clamp(max=s["q"].shape[0] - 1)
    has = step[None, :] < new[:, None]
    q = s["q"][tok].float().view(n, most, hkv, group, d)
    pos = torch.arange(past, device=DEV)
    cached = pos[None, :] < ctx[:, None]
    page = s["table"].long()[:, pos // b] * b + pos[None, :] % b
    # keys and values a request does not have count as zeros
    blank, none = ~cached[:, :, None, None], ~has[:, :, None, None]
    k = torch.cat([s["kc"].view(-1, hkv, d)[page].float().masked_fill_(blank, 0),
                   s["k"][tok].float().masked_fill_(none, 0)], 1)
    v = torch.cat([s["vc"].view(-1, hkv, d)[page].float().masked_fill_(blank, 0),
                   s["v"][tok].float().masked_fill_(none, 0)], 1)
    if s["mask"] is None:
        among = (step[None, None, :] <= step[None, :, None]).expand(n, most, most)
    else:
        word = s["mask"][tok][:, :, step // 32]  # [n, most, most]
        among = ((word >> (step % 32)) & 1) != 0
    sees = torch.cat([cached[:, None, :].expand(n, most, past), among & has[:, None, :]], 2)
    score = torch.einsum("nqhgd,nkhd->nhgqk", q, k) * (d ** -0.5)
    score.masked_fill_(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("nhgqk,nkhd->nhgqd", p, v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(n, most, hq)
    return [o[has].to(s["q"].dtype), lse[has]]


# -------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tables": _plain_tables, "rope": _plain_rope, "commit": _plain_commit, "attn": _plain_attn}[op](s)
    import selective_state_space_mamba2_gb300 as ssd
    if op == "tables":
        r = ssd.kv_block_tables(s["ctx"], s["new"], s["reserved"], s["table"], s["ring"], s["state"],
                                block_size=s["case"]["block"], num_blocks=s["blocks"], max_tokens=s["max_tokens"])
        return [s["table"], r["cu_seqlens"], r["seq_lens"], r["reserved_lens"], r["ring_state"], r["slots"],
                r["positions"], r["token_req"]]
    if op == "rope":
        q, k = ssd.kv_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], q_weight=s["qw"], k_weight=s["kw"],
                                   eps=1e-6, interleaved=bool(s["case"]["inter"]), v=s["v"], k_cache=s["kc"],
                                   v_cache=s["vc"], slots=s["slots"])
        return [q, k, s["kc"], s["vc"]]
    if op == "commit":
        lens = ssd.kv_commit_tokens(s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["cu"], s["ctx"],
                                    path=s.get("path"), path_lens=s.get("lens"))
        return [s["kc"], s["vc"], lens]
    return list(ssd.kv_tree_attention(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["cu"], s["ctx"], s["table"],
                                      max_new_tokens=s["max_new"], tree_mask=s["mask"], return_lse=True))


# ------------------------------------------------------------------ exact --

def _exact_rope(s):
    rot, inter = s["case"]["rot"], s["case"]["inter"]
    cs = s["cos_sin"].double().index_select(0, s["positions"].long())
    made = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
        y = x.clone()
        for i in range(rot // 2):
            lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            c, sn = cs[:, i, None], cs[:, rot // 2 + i, None]
            y[:, :, lo] = x[:, :, lo] * c - x[:, :, hi] * sn
            y[:, :, hi] = x[:, :, hi] * c + x[:, :, lo] * sn
        made.append(y)
    kc, vc = s["kc"].double(), s["vc"].double()
    blk, off = s["slots"].long() // s["case"]["block"], s["slots"].long() % s["case"]["block"]
    kc[blk, off] = made[1]
    vc[blk, off] = s["v"].double()
    return [made[0], made[1], kc, vc]


def _exact_attn(s):
    case = s["case"]
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["block"]
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out, lse = [], []
    for r, c in enumerate(ctx):
        n = cu[r + 1] - cu[r]
        pages = s["table"][r, :_cdiv(c, b)].long()
        part = slice(cu[r], cu[r + 1])
        k = torch.cat([s["kc"][pages].reshape(-1, hkv, d)[:c].double(), s["k"][part].double()])
        v = torch.cat([s["vc"][pages].reshape(-1, hkv, d)[:c].double(), s["v"][part].double()])
        if s["mask"] is None:
            among = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        else:
            words = s["mask"][part].long() & 0xFFFFFFFF
            j = torch.arange(n, device=DEV)
            among = (words[:, j // 32] >> (j % 32)[None, :]) % 2 == 1
        sees = torch.cat([torch.ones(n, c, dtype=torch.bool, device=DEV), among], 1)
        o_r = torch.empty(n, hq, d, dtype=torch.float64, device=DEV)
        l_r = torch.empty(n, hq, dtype=torch.float64, device=DEV)
        for h in range(hq):
            kv = h // (hq // hkv)
            score = (s["q"][part, h].double() @ k[:, kv].T) / math.sqrt(d)
            score = torch.where(sees, score, torch.full_like(score, -math.inf))
            l_r[:, h] = torch.logsumexp(score, 1)
            weight = torch.where(sees, torch.exp(score - l_r[:, h, None]), torch.zeros_like(score))
            o_r[:, h] = weight @ v[:, kv]
        out.append(o_r)
        lse.append(l_r)
    return [torch.cat(out), torch.cat(lse)]


def _exact_commit(s):
    """Row by row from the definition: token path[r, i] of request r goes to slot i of its tokens."""
    cu, b = s["cu"].tolist(), s["case"]["block"]
    kc, vc = s["kc"].double(), s["vc"].double()
    src, dst = [], []
    for r in range(len(cu) - 1):
        kept = range(cu[r + 1] - cu[r]) if "path" not in s else s["path"][r, :int(s["lens"][r])].tolist()
        src += [cu[r] + j for j in kept]
        dst += [cu[r] + i for i in range(len(kept))]
    slot, src = s["slots"].long()[dst], torch.tensor(src, device=DEV)
    kc[slot // b, slot % b] = s["k"][src].double()
    vc[slot // b, slot % b] = s["v"][src].double()
    return [kc, vc, None]


def exact(case, seed):
    if case["op"] == "tables" or work(case)["flops"] > 4e12:
        return None  # whole numbers; or over the time a comparison may take
    s = prepare(case, seed)
    return {"rope": _exact_rope, "commit": _exact_commit, "attn": _exact_attn}[case["op"]](s)
