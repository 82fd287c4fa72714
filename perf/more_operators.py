"""Measured cases of decoding over a paged cache that is held in 8 bits, a scale for each block of tokens and head:
keys and values quantised as they are written (``kv_commit_tokens_fp8``) and read back (``kv_read_tokens_fp8``), attention
of new tokens over that cache (``kv_tree_attention_fp8``), and the verification of drafted tokens against the target's
probabilities from given random numbers (``kv_verify_tokens``).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, in 64 where whole numbers hang on a
sum) unless ``own`` is true; then it makes the calls a user makes of the library."""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
LEAST, MOST = -64, 119  # exponents of the scales


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # after a step of a speculative batch: accepted paths of at most 5 of 16 drafted tokens for 256 requests
        dict(name="commit_tree", op="commit", reqs=256, nodes=16, path=5, ctx_hi=8192, hkv=8, d=128, type="bf16", block=64),
        # prompts written as they are, 8 of 4096 tokens behind ragged prefixes
        dict(name="commit_prompt", op="commit", reqs=8, nodes=4096, path=0, ctx_hi=500, hkv=8, d=128, type="bf16", block=16),
        # a few short rows of an fp32 model with odd head and block sizes: a latency case
        dict(name="read_odd", op="read", reqs=3, lo=1, hi=37, start=90, hkv=5, d=80, type="f32", block=24),
        # cached prefixes of 16 requests back to bf16
        dict(name="read_prefix", op="read", reqs=16, lo=500, hi=8192, start=0, hkv=8, d=128, type="bf16", block=64),
        # one token of one short request: the smallest decode call
        dict(name="attn_one", op="attn", reqs=1, q_lo=1, q_hi=1, ctx_lo=777, ctx_hi=777, hq=32, hkv=8, d=128,
             type="bf16", block=16, tree=0),
        # one token of one long request (65536 cached): the cache has to be split over the GPU
        dict(name="attn_long", op="attn", reqs=1, q_lo=1, q_hi=1, ctx_lo=65536, ctx_hi=65536, hq=32, hkv=8, d=128,
             type="bf16", block=256, tree=0),
        # the speculative batch: 256 requests of 1 + 3 tokens over ragged caches
        dict(name="attn_spec", op="attn", reqs=256, q_lo=4, q_hi=4, ctx_lo=0, ctx_hi=8192, hq=32, hkv=8, d=128,
             type="bf16", block=64, tree=0),
        # ragged trees of up to 64 drafted tokens, 8 query heads to a key head
        dict(name="attn_tree", op="attn", reqs=24, q_lo=33, q_hi=64, ctx_lo=0, ctx_hi=16384, hq=32, hkv=4, d=128,
             type="bf16", block=32, tree=1),
        # a chunk of prompts behind cached prefixes: new tokens attend to the prefix and to one another
        dict(name="attn_prompt", op="attn", reqs=4, q_lo=512, q_hi=4096, ctx_lo=0, ctx_hi=8192, hq=32, hkv=8, d=128,
             type="bf16", block=64, tree=0),
        # small fp32 trees over pages of an odd size
        dict(name="attn_f32", op="attn", reqs=16, q_lo=1, q_hi=7, ctx_lo=0, ctx_hi=2000, hq=16, hkv=4, d=64,
             type="f32", block=24, tree=1),
        # drafts of a speculative batch, 1 + 3 tokens a request, drawn from a draft model's probabilities
        dict(name="verify_chain", op="verify", reqs=256, nodes=4, vocab=65536, tree=0, draft=1, type="f32"),
        # drafted trees of a handful of requests, their tokens the likeliest ones of a draft
        dict(name="verify_tree", op="verify", reqs=5, nodes=24, vocab=50021, tree=1, draft=0, type="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    """One more case of the listed ranges: requests, lengths, heads, types, page sizes, masks, vocabularies."""
    op = rng.choice(["commit", "read", "attn", "attn", "attn", "verify"])
    if op == "verify":
        vocab = _log(rng, 1000, 65536)
        tree = rng.choice([0, 1])
        return dict(op=op, reqs=_log(rng, 1, 64 if tree else 256), nodes=_log(rng, 1, 32) if tree else rng.choice([1, 2, 4, 8]),
                    vocab=vocab, tree=tree, draft=rng.choice([0, 1]), type=rng.choice(["f32", "f32", "bf16"]))
    block = rng.choice([8, 16, 16, 24, 32, 48, 64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "commit":
        nodes = _log(rng, 1, 512)
        return dict(op=op, reqs=_log(rng, 1, 64), nodes=nodes, path=rng.choice([0, min(nodes, 6)]), ctx_hi=_log(rng, 1, 8192),
                    hkv=hkv, d=rng.choice([64, 80, 128, 128]), type=dtype, block=block)
    if op == "read":
        return dict(op=op, reqs=_log(rng, 1, 64), lo=0, hi=_log(rng, 1, 2048), start=rng.choice([0, _log(rng, 1, 1000)]), hkv=hkv,
                    d=rng.choice([64, 80, 128, 128]), type=dtype, block=block)
    d = rng.choice([64, 128, 128])
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


def _cdiv(a, b):
    return -(-a // b)


def _lens(case):
    """Request lengths of a case; they are a property of the case, not of the seed of its values."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["reqs"]
    if case["op"] == "commit":
        return [case["nodes"]] * n, [rng.randint(0, case["ctx_hi"]) for _ in range(n)]
    if case["op"] == "read":
        new = [rng.randint(case["lo"], case["hi"]) for _ in range(n)]
        new[-1] = case["hi"]
        return new, [rng.randint(0, case["start"]) for _ in range(n)]
    if case["op"] == "verify":
        new = [rng.randint(1, case["nodes"]) if case["tree"] else case["nodes"] for _ in range(n)]
        new[-1] = case["nodes"]
        return new, [0] * n
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    if n > 1:
        ctx[0] = 0  # a request with nothing cached
        new[-1], ctx[-1] = case["q_hi"], case["ctx_hi"]
    return new, ctx


def work(case):
    op = case["op"]
    e = 2 if case["type"] == "bf16" else 4
    new, ctx = _lens(case)
    t, n = sum(new), case["reqs"]
    if op == "verify":
        # the row that the next token is drawn from, of target and draft, and a few words a drafted token
        return {"bytes": n * case["vocab"] * e * (1 + case["draft"]) + t * (12 + 2 * e) + 4 * n * (case["nodes"] + 3), "flops": 0}
    hkv, d, b = case["hkv"], case["d"], case["block"]
    if op == "commit":
        rows = n * case["path"] if case["path"] else t
        pages = sum(_cdiv(c + (case["path"] or m), b) - c // b for c, m in zip(ctx, new))
        return {"bytes": rows * hkv * d * 2 * (e + 1) + pages * (8 * hkv + 4) + 8 * rows, "flops": 0}
    if op == "read":
        pages = sum(_cdiv(c + m, b) - c // b for c, m in zip(ctx, new))
        return {"bytes": t * hkv * d * 2 * (e + 1) + pages * (8 * hkv + 4), "flops": 0}
    hq = case["hq"]
    # a tree's tokens see themselves at least; a chain's every token before them
    pairs = sum(m * c + (m if case["tree"] else m * (m + 1) // 2) for c, m in zip(ctx, new))
    pages = sum(_cdiv(c, b) for c in ctx)
    return {"bytes": sum(ctx) * hkv * d * 2 + t * hkv * d * 2 * e + 2 * t * hq * d * e + 4 * t * hq + pages * (8 * hkv + 4)
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
    return torch.where(col[None, :] < held[:, None], perm[index], 0).to(torch.int32), total


def _scale(top):
    """The smallest power of two that brings magnitudes of at most ``top`` into e4m3."""
    m, e = torch.frexp(top.float())
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(LEAST, MOST)
    return torch.where(top > 0, torch.exp2(e.double()), 2.0 ** LEAST).float()


def _cache(g, blocks, b, hkv, d):
    """A cache as it stands after some steps: codes and scales of blocks whose heads differ in size."""
    codes = torch.empty((blocks, b, hkv, d), dtype=E4M3, device=DEV)
    size = torch.exp2(_randn(g, (blocks, hkv), torch.float32))
    scale = torch.empty((blocks, hkv), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (b * hkv * d))
    for i in range(0, blocks, step):
        x = _randn(g, (min(step, blocks - i), b, hkv, d), torch.float32) * size[i:i + step, None, :, None]
        scale[i:i + step] = _scale(x.abs().amax((1, 3)))
        codes[i:i + step] = (x / scale[i:i + step, None, :, None]).to(E4M3)
    return codes, scale


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


def _drafts(s, g, rng, new, cu):
    """Target probabilities, and trees of tokens drafted from a model that is near the target."""
    case = s["case"]
    t, vocab, dtype = sum(new), case["vocab"], TYPES[case["type"]]
    logits = 2.5 * _randn(g, (t, vocab), torch.float32)
    near = torch.softmax(logits + 0.5 * _randn(g, (t, vocab), torch.float32), -1).to(dtype)
    s["p"] = torch.softmax(logits, -1).to(dtype)
    parent = [[-1] + [rng.randrange(max(0, i - 3), i) if case["tree"] else i - 1 for i in range(1, n)] for n in new]
    at = torch.tensor([cu[r] + max(k, 0) for r, up in enumerate(parent) for k in up], device=DEV)
    rank = [[sum(1 for k in up[1:i] if k == up[i]) if i else 0 for i in range(len(up))] for up in parent]
    if case["draft"]:
        pick = torch.multinomial(near.float(), max(new), replacement=True, generator=g)  # with replacement, as drawn
        s["q"] = near
    else:
        pick = near.topk(max(new), -1).indices
        s["q"] = None
    s["tokens"] = pick[at, torch.tensor([k for up in rank for k in up], device=DEV)].to(torch.int32)
    s["parents"] = _ints([k for up in parent for k in up]) if case["tree"] else None
    s["uniform"] = torch.rand(t, generator=g, device=DEV)
    s["most"] = max(new)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    rng = random.Random(seed)
    op = case["op"]
    s = dict(case=case)
    new, ctx = _lens(case)
    t, n = sum(new), case["reqs"]
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s["cu"], s["ctx"], s["most"] = _ints(cu), _ints(ctx), max(new)
    if op == "verify":
        _drafts(s, g, rng, new, cu)
        return s
    dtype = TYPES[case["type"]]
    hkv, d, b = case["hkv"], case["d"], case["block"]
    held = ctx if op == "attn" else [c + m for c, m in zip(ctx, new)]
    s["table"], blocks = _tables(g, held, b, 3, _cdiv(max(held), b) + 1)
    s["kc"], s["ks"] = _cache(g, blocks, b, hkv, d)
    s["vc"], s["vs"] = _cache(g, blocks, b, hkv, d)
    if op == "read":
        return s
    hq = case["hq"] if op == "attn" else 0
    qkv = _randn(g, (t, (hq + 2 * hkv) * d), dtype)  # one packed projection, read through views
    s["q"] = qkv[:, :hq * d].view(t, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    if op == "attn":
        s["most_ctx"] = max(ctx)
        s["mask"] = _tree_bits(rng, new, _cdiv(max(new), 32)) if case["tree"] else None
    elif case["path"]:
        s["path"] = _ints([sorted(rng.sample(range(case["nodes"]), case["path"])) for _ in range(n)])
        s["lens"] = _ints([rng.randint(1, case["path"]) for _ in range(n)])
    return s


# ------------------------------------------------------------ plain forms --

def _codes(codes, *at):
    """Entries of a cache in 8 bits."""
    return codes.view(torch.uint8)[at].view(E4M3)


def _plain_commit(s):
    b, hkv, d = s["case"]["block"], s["case"]["hkv"], s["case"]["d"]
    table, cu, ctx = s["table"].long(), s["cu"].long(), s["ctx"].long()
    n, cols = table.shape
    if "path" in s:
        lens = s["lens"].long()
        step = torch.arange(s["path"].shape[1], device=DEV)[None, :].expand(n, -1)
        row = cu[:-1, None] + s["path"].long()
    else:
        lens = cu[1:] - cu[:-1]
        step = torch.arange(s["most"], device=DEV)[None, :].expand(n, -1)
        row = cu[:-1, None] + step
    live = step < lens[:, None]
    req = torch.arange(n, device=DEV)[:, None].expand_as(step)[live]
    row, pos = row[live], ctx[req] + step[live]
    page, off = table[req, pos // b], pos % b
    # a request's first block may hold rows already
    first, fill = table[torch.arange(n, device=DEV), (ctx // b).clamp(max=cols - 1)], ctx % b
    fill = torch.where(lens > 0, fill, 0)
    outs = []
    for x, codes, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x[row].float()
        top = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV).index_fill_(0, page, True)
        keeps = torch.zeros_like(touched).index_fill_(0, first[fill > 0], True)
        need = _scale(top)
        need = torch.where(keeps[:, None], torch.maximum(need, scale), need)
        now = torch.where(touched[:, None], need, scale)
        old = _codes(codes, first).float()
        ratio = (scale / now)[first][:, None, :, None]
        again = torch.arange(b, device=DEV)[None, :] < fill[:, None]
        at = again.nonzero(as_tuple=True)
        codes.view(torch.uint8)[first[at[0]], at[1]] = (old * ratio).to(E4M3).view(torch.uint8)[at]
        codes.view(torch.uint8)[page, off] = (x / now[page][:, :, None]).to(E4M3).view(torch.uint8)
        scale.copy_(now)
        outs += [codes, scale]
    return outs + [(ctx + lens).to(torch.int32)]


def _plain_read(s):
    b = s["case"]["block"]
    table, cu, start = s["table"].long(), s["cu"].long(), s["ctx"].long()
    tok = torch.arange(int(sum(_lens(s["case"])[0])), device=DEV)
    req = torch.searchsorted(cu[1:], tok, right=True)
    pos = start[req] + tok - cu[req]
    page, off = table[req, pos // b], pos % b
    dtype = TYPES[s["case"]["type"]]
    return [(_codes(codes, page, off).float() * scale[page][:, :, None]).to(dtype)
            for codes, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]


def _plain_attn(s):
    case = s["case"]
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["block"]
    n, group, most, past = case["reqs"], hq // hkv, s["most"], s["most_ctx"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    new = cu[1:] - cu[:-1]
    # queries and new keys padded to the longest request: [n, most, heads, d]
    step = torch.arange(most, device=DEV)
    tok = (cu[:-1, None] + step[None, :]).clamp(max=s["q"].shape[0] - 1)
    has = step[None, :] < new[:, None]
    q = s["q"][tok].float().view(n, most, hkv, group, d)
    pos = torch.arange(past, device=DEV)
    cached = pos[None, :] < ctx[:, None]
    page = s["table"].long()[:, pos // b]
    off = (pos % b)[None, :].expand(n, -1)
    # keys and values a request does not have count as zeros
    blank, none = ~cached[:, :, None, None], ~has[:, :, None, None]
    kc = _codes(s["kc"], page, off).float() * s["ks"][page][:, :, :, None]
    k = torch.cat([kc.masked_fill_(blank, 0), s["k"][tok].float().masked_fill_(none, 0)], 1)
    del kc
    vc = _codes(s["vc"], page, off).float() * s["vs"][page][:, :, :, None]
    v = torch.cat([vc.masked_fill_(blank, 0), s["v"][tok].float().masked_fill_(none, 0)], 1)
    del vc
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


def _fixed(x):
    """Weights as whole numbers of 2^-44, whose sums do not depend on their order."""
    return (x.clamp(0, 1) * 2.0 ** 44).to(torch.int64)


def _plain_verify(s):
    cu, tokens, p, q = s["cu"].long(), s["tokens"].long(), s["p"], s["q"]
    n, most = cu.numel() - 1, s["most"]
    all_r = torch.arange(n, device=DEV)
    lens = cu[1:] - cu[:-1]
    cur = torch.zeros(n, dtype=torch.long, device=DEV)  # the last accepted token
    depth = (lens > 0).long()
    path = torch.full((n, most), -1, dtype=torch.long, device=DEV)
    path[:, 0] = torch.where(lens > 0, 0, -1)
    over = torch.zeros(n, dtype=torch.float64, device=DEV)   # the factor of the draft in the residual
    left = torch.ones(n, dtype=torch.float64, device=DEV)    # the residual's sum
    p_row = p[cu[:-1]].float()
    q_row = q[cu[:-1]].float() if q is not None else torch.zeros_like(p_row)
    for j in range(1, most):  # children follow their parents
        at = (cu[:-1] + j).clamp(max=tokens.numel() - 1)
        up = s["parents"][at].long() if s["parents"] is not None else torch.full_like(at, j - 1)
        tried = (j < lens) & (up == cur)
        tok, u = tokens[at], s["uniform"][at].double()
        pt, qt = p_row[all_r, tok], q_row[all_r, tok]
        if q is None:  # a drafted token was certain to be drafted; rejected ones have no weight any more
            takes = tried & (u * left < pt.double())
        else:
            rest = (pt - over.float() * qt).clamp(min=0)
            takes = tried & (u * qt.double() * left < rest.double())
        drops = tried & ~takes
        cur = torch.where(takes, j, cur)
        path[all_r, torch.where(takes, depth, 0)] = torch.where(takes, j, path[:, 0])
        depth = depth + takes
        if q is None:
            left = torch.where(drops, (left - pt.double()).clamp(min=0), left)
            p_row[all_r, tok] = torch.where(drops, 0, pt)
        else:
            over = torch.where(drops, over + left, over)
            rest = _fixed(p_row - over.float()[:, None] * q_row).sum(1).double() * 2.0 ** -44
            left = torch.where(drops, rest, left)
            q_row = torch.where(takes[:, None], q[cu[:-1] + cur].float(), q_row)
        p_row = torch.where(takes[:, None], p[cu[:-1] + cur].float(), p_row)
        over, left = torch.where(takes, 0, over), torch.where(takes, 1, left)
    weight = _fixed(p_row - over.float()[:, None] * q_row if q is not None else p_row)
    ends = weight.cumsum(1)
    total = ends[:, -1]
    draw24 = (s["uniform"][cu[:-1]] * 2.0 ** 24).to(torch.int64)
    mark = (total >> 24) * draw24 + (((total & 0xFFFFFF) * draw24) >> 24)
    nxt = torch.searchsorted(ends, mark[:, None], right=True)[:, 0]
    i32 = torch.int32
    return [path.to(i32), depth.to(i32), (depth - 1).clamp(min=0).to(i32), nxt.to(i32)]


# -------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"commit": _plain_commit, "read": _plain_read, "attn": _plain_attn, "verify": _plain_verify}[op](s)
    import selective_state_space_mamba2_gb300 as ssd
    if op == "commit":
        lens = ssd.kv_commit_tokens_fp8(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["ctx"],
                                        path=s.get("path"), path_lens=s.get("lens"))
        return [s["kc"], s["ks"], s["vc"], s["vs"], lens]
    if op == "read":
        return list(ssd.kv_read_tokens_fp8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["ctx"],
                                           total_tokens=int(sum(_lens(s["case"])[0])), dtype=TYPES[s["case"]["type"]]))
    if op == "attn":
        return list(ssd.kv_tree_attention_fp8(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["cu"], s["ctx"],
                                              s["table"], max_new_tokens=s["most"], tree_mask=s["mask"], return_lse=True))
    r = ssd.kv_verify_tokens(s["tokens"], s["p"], s["uniform"], s["cu"], max_path=s["most"], draft_probs=s["q"],
                             parents=s["parents"])
    return [r["path"], r["path_lens"], r["accepted"], r["next_tokens"]]


# ------------------------------------------------------------------ exact --

def _to_e4m3(y):
    """Doubles rounded to the nearest value of e4m3, ties to the even one."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_commit(s):
    """Request by request and block by block from the definition."""
    b, table = s["case"]["block"], s["table"].tolist()
    cu, ctx, outs, lens = s["cu"].tolist(), s["ctx"].tolist(), [], []
    paths = [list(range(cu[r + 1] - cu[r])) for r in range(len(ctx))]
    if "path" in s:
        paths = [row[:k] for row, k in zip(s["path"].tolist(), s["lens"].tolist())]
    for x, codes, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        codes, scale = codes.double(), scale.double()
        for r, path in enumerate(paths):
            for col in range(ctx[r] // b, (ctx[r] + len(path) - 1) // b + 1):
                lo, hi = max(ctx[r], col * b), min(ctx[r] + len(path), (col + 1) * b)
                page, fill = table[r][col], lo - col * b
                rows = x[torch.tensor(path[lo - ctx[r]:hi - ctx[r]], device=DEV) + cu[r]].double()
                k = torch.ceil(torch.log2(rows.abs().amax((0, 2)).clamp(min=1e-300) / 448)).clamp(LEAST, MOST)
                now = torch.exp2(k)
                if fill:
                    now = torch.maximum(now, scale[page])
                    codes[page, :fill] = _to_e4m3(codes[page, :fill] * (scale[page] / now)[:, None])
                scale[page] = now
                codes[page, fill:fill + hi - lo] = _to_e4m3(rows / now[:, None])
        outs += [codes, scale]
    return outs + [None]


def _exact_read(s):
    b, outs = s["case"]["block"], []
    cu, start = s["cu"].tolist(), s["ctx"].tolist()
    for codes, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        parts = []
        for r, c in enumerate(start):
            n = cu[r + 1] - cu[r]
            pages = s["table"][r, :_cdiv(c + n, b)].long()
            rows = _codes(codes, pages).double() * scale[pages].double()[:, None, :, None]
            parts.append(rows.reshape(-1, *rows.shape[2:])[c:c + n])
        outs.append(torch.cat(parts))
    return outs


def _exact_attn(s):
    case = s["case"]
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["block"]
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out, lse = [], []
    for r, c in enumerate(ctx):
        n = cu[r + 1] - cu[r]
        pages = s["table"][r, :_cdiv(c, b)].long()
        part = slice(cu[r], cu[r + 1])
        k, v = (torch.cat([(_codes(codes, pages).double() * scale[pages].double()[:, None, :, None]).reshape(-1, hkv, d)[:c],
                           fresh[part].double()])
                for codes, scale, fresh in ((s["kc"], s["ks"], s["k"]), (s["vc"], s["vs"], s["v"])))
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


def exact(case, seed):
    if case["op"] == "verify" or work(case)["flops"] > 4e12:
        return None  # whole numbers; or over the time a comparison may take
    s = prepare(case, seed)
    return {"commit": _exact_commit, "read": _exact_read, "attn": _exact_attn}[case["op"]](s)
