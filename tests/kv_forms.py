"""Plain 64-bit forms of the attention-side calls, request by request, and the error bounds their
results are held to.

The bounds come from the kernels' arithmetic alone.  u = 2^-24 is fp32's unit roundoff and b = 2^-8
bf16's.  A score is D products and sums in fp32: off by at most (D + 4) u scale sum |q||k|.  A weight
exp(s) carries that error relatively (twice: its own score and the maximum's), 2^-21 of the
exponential and, on the tensor cores, b for the weight's rounding to bf16; sums over n keys add n u.
The output is a weighted mean, so it is off by those relative errors times sum w |v|, plus its own
rounding."""
import numpy as np
import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8


def poison(shape, dtype, device):
    """NaN everywhere: a row that is read, or multiplied by a zero weight, shows."""
    return torch.full(shape, float("nan"), dtype=dtype, device=device)


def block_tables(ctx, new, reserved, table, ring, state, b, num_blocks, max_tokens, null=0):
    """kv_block_tables on lists; returns (ok, dict)."""
    S, cols = table.shape
    table = table.copy()
    head, count = state
    cdiv = lambda x: -(-x // b)
    bad = any(c < 0 or n < 0 or v < 0 for c, n, v in zip(ctx, new, reserved)) or sum(new) > max_tokens
    if not bad:
        need = [max(cdiv(v), cdiv(c + n)) for c, n, v in zip(ctx, new, reserved)]
        pops = sum(m - cdiv(v) for m, v in zip(need, reserved))
        bad = any(m > cols for m in need) or pops > count
    out = dict(slots=[-1] * max_tokens, positions=[0] * max_tokens, token_req=[-1] * max_tokens)
    if bad:
        out.update(table=table, cu_seqlens=[0] * (S + 1), seq_lens=list(ctx), reserved_lens=list(reserved),
                   ring_state=[head, count])
        return False, out
    cu, at, bad_slot = [0], head, False
    for r in range(S):
        for col in range(cdiv(reserved[r]), need[r]):
            table[r, col] = ring[at % len(ring)]
            at += 1
        for j in range(new[r]):
            t, pos = cu[-1] + j, ctx[r] + j
            blk = int(table[r, pos // b])
            out["positions"][t], out["token_req"][t] = pos, r
            if blk != null and 0 <= blk < num_blocks:
                out["slots"][t] = blk * b + pos % b
            elif blk != null:
                bad_slot = True
        cu.append(cu[-1] + new[r])
    out.update(table=table, cu_seqlens=cu, seq_lens=[c + n for c, n in zip(ctx, new)],
               reserved_lens=[max(v, c + n) for c, n, v in zip(ctx, new, reserved)],
               ring_state=[at % len(ring) if at != head else head, count - (at - head)])
    out["bad_slot"] = bad_slot
    return True, out


def norm_rope(x, weight, cos_sin, positions, eps, interleaved):
    """x [T, H, D] -> float64, and the bound's scale sum |terms| per entry."""
    x = x.double().cpu()
    T, H, D = x.shape
    n = x
    if weight is not None:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    y, mag = n.clone(), n.abs()
    if cos_sin is not None:
        R = cos_sin.shape[1]
        cs = cos_sin.double().cpu()[positions.long().cpu()]
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            c, s = cs[:, i, None], cs[:, R // 2 + i, None]
            y[:, :, a] = n[:, :, a] * c - n[:, :, b] * s
            y[:, :, b] = n[:, :, b] * c + n[:, :, a] * s
            mag[:, :, a] = (n[:, :, a] * c).abs() + (n[:, :, b] * s).abs()
            mag[:, :, b] = (n[:, :, b] * c).abs() + (n[:, :, a] * s).abs()
    return y, mag


def rope_bound(y, mag, D, dtype):
    # mean of D squares, rsqrt (2 ulp), weight, angle, two products and a sum: (D / 2 + 10) u at most;
    # then the rounding of the result
    return (D / 2 + 10) * U32 * mag + (UBF if dtype == torch.bfloat16 else U32) * y.abs() * 1.01 + 1e-30


def attention(q, k_new, v_new, k_cache, v_cache, cu, ctx, table, mask, scale):
    """Per request and head in float64: out, lse, and sum w|v|, the largest scale sum |q||k| and the
    number of keys of each row (for the bound)."""
    T, H, D = q.shape
    Hkv = k_new.shape[1]
    b = k_cache.shape[1]
    out, mag = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64)
    big, keys = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    q, k_new, v_new = q.double().cpu(), k_new.double().cpu(), v_new.double().cpu()
    for r in range(len(ctx)):
        n, c = cu[r + 1] - cu[r], ctx[r]
        blocks = [int(table[r, j]) for j in range(-(-c // b))]
        kc = k_cache[blocks].reshape(-1, Hkv, D)[:c].double().cpu()
        vc = v_cache[blocks].reshape(-1, Hkv, D)[:c].double().cpu()
        for i in range(n):
            t = cu[r] + i
            if mask is None:
                sees = list(range(i + 1))
            else:
                sees = [j for j in range(n) if (int(mask[t, j // 32]) >> (j % 32)) & 1]
            rows = torch.tensor([cu[r] + j for j in sees], dtype=torch.long)
            k = torch.cat([kc, k_new[rows]])
            v = torch.cat([vc, v_new[rows]])
            keys[t] = k.shape[0]
            if k.shape[0] == 0:
                continue
            for h in range(H):
                g = h // (H // Hkv)
                s = scale * (k[:, g] @ q[t, h])
                lse[t, h] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[t, h])
                # where a weight is zero the value does not count
                out[t, h] = w @ v[:, g]
                mag[t, h] = w @ v[:, g].abs()
                big[t, h] = (k[:, g].abs() @ q[t, h].abs()).max() * abs(scale)
    return out, lse, mag, big, keys


def attention_bound(out, lse, mag, big, keys, D, dtype):
    score = (D + 4) * U32 * big  # of a score
    rel = 2 * score + 2.0 ** -21 + (keys[:, None] + 8) * U32
    weight = rel + (UBF if dtype == torch.bfloat16 else 0.0)
    tol = 1.01 * weight[..., None] * mag + 1.01 * (UBF if dtype == torch.bfloat16 else U32) * out.abs() + 1e-30
    finite = torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))
    return tol, rel + 4 * U32 * finite.abs()


def rand_pages(lens, b, cols, spare, rng):
    """Scattered block ids for requests of these lengths; returns (table, number of blocks)."""
    need = [-(-n // b) for n in lens]
    total = sum(need) + spare + 1
    ids = rng.permutation(np.arange(1, total))
    table = np.zeros((len(lens), cols), np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, total, ids[at:].astype(np.int32)
