"""The attention-side calls (kv_block_tables, kv_qk_norm_rope, kv_tree_attention, kv_commit_tokens) on
the GPU against plain 64-bit forms, with NaN in every cache row, page and draft that must not count."""
import numpy as np
import pytest
import torch

import selective_state_space_mamba2_gb300 as ssd
from tests import kv_forms as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ssd.build()
    torch.cuda.init()


def _i(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ tables --

def _tables(ctx, new, reserved, b, cols, max_tokens, free, head, null=0, spare_ring=3, seed=0, mangle=None):
    rng = np.random.default_rng(seed)
    table, total, ids = F.rand_pages(reserved, b, cols, free, rng)
    if mangle:
        mangle(table)
    cap = free + spare_ring
    ring = np.full(cap, -7, np.int32)
    for i in range(free):
        ring[(head + i) % cap] = ids[i]
    ok, want = F.block_tables(ctx, new, reserved, table, ring, (head, free), b, total, max_tokens, null)
    t, r, err = _i(table), _i(ring), _err()
    got = ssd.kv_block_tables(_i(ctx), _i(new), _i(reserved), t, r, _i([head, free]), b, total, max_tokens,
                              null_block_id=null, err_word=err)
    torch.cuda.synchronize()
    for key in ("cu_seqlens", "seq_lens", "reserved_lens", "ring_state", "slots", "positions", "token_req"):
        assert got[key].tolist() == list(want[key]), key
    assert np.array_equal(t.cpu().numpy(), want["table"])
    assert np.array_equal(r.cpu().numpy(), ring)
    return ok, want, int(err.item())


@pytest.mark.parametrize("seed", range(6))
def test_tables_random_batches(seed):
    """Ragged batches: empty requests, contexts inside and at block ends, rows with blocks to spare, a context beyond
    what is reserved, a ring that wraps, padding rows; more requests than a CTA has threads."""
    rng = np.random.default_rng(100 + seed)
    S = [1, 7, 256, 257, 600, 33][seed]
    b = [16, 1, 64, 5, 16, 256][seed]
    top = [40, 9, 130, 30, 20, 3000][seed]
    ctx = rng.integers(0, top, S)
    new = rng.integers(0, top, S) * (rng.random(S) < 0.8)
    reserved = np.maximum(0, ctx + rng.integers(-b, 3 * b, S))
    cols = int((ctx + new).max() // b + 5)
    free = int(sum(-(-(c + n) // b) for c, n in zip(ctx, new))) + 2
    ok, _, err = _tables(ctx.tolist(), new.tolist(), reserved.tolist(), b, cols, int(new.sum()) + 11, free,
                         head=free + 1, seed=seed)
    assert ok and err == 0


def test_tables_long_prompts_beside_decodes():
    """Requests over several token tiles beside single tokens, and a request that ends exactly with the output."""
    new = [1, 5000, 1, 0, 1024, 9, 8, 1, 2048]
    ctx = [17, 3, 0, 5, 64, 0, 7, 16, 100]
    b = 16
    free = sum(-(-(c + n) // b) for c, n in zip(ctx, new))
    ok, _, err = _tables(ctx, new, ctx, b, 400, sum(new), free, head=0)
    assert ok and err == 0


@pytest.mark.parametrize("case,bit", [("blocks", 32), ("cols", 32), ("tokens", 2), ("negative", 2), ("ring", 2)])
def test_tables_refuse_as_a_whole(case, bit):
    """A step that cannot be served changes nothing and comes back empty."""
    ctx, new, reserved, b, cols, top, free = [10, 20, 5], [30, 1, 2], [10, 20, 5], 8, 8, 64, 20
    head = 2
    if case == "blocks":
        free = 2
    elif case == "cols":
        cols = 4
    elif case == "tokens":
        top = 32
    elif case == "negative":
        new = [30, -1, 2]
    elif case == "ring":
        head = 23  # free + spare_ring entries: none at 23
    rng = np.random.default_rng(0)
    table, total, ids = F.rand_pages(reserved, b, cols, 20, rng)
    ring = np.concatenate([ids[:20], np.full(3, -7, np.int32)])
    t, r, err, state = _i(table), _i(ring), _err(), _i([head, free])
    got = ssd.kv_block_tables(_i(ctx), _i(new), _i(reserved), t, r, state, b, total, top, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bit
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), ring)
    assert got["cu_seqlens"].tolist() == [0] * 4 and got["slots"].tolist() == [-1] * top
    assert got["token_req"].tolist() == [-1] * top and got["positions"].tolist() == [0] * top
    assert got["seq_lens"].tolist() == ctx and got["reserved_lens"].tolist() == reserved
    assert got["ring_state"].tolist() == [head, free]


def test_tables_null_and_bad_entries():
    """A held entry that is the null block gives slot -1; one that is no block does too, and is reported."""
    def null(t):
        t[0, 1] = 9999

    def none(t):
        t[0, 1] = 0
    ok, want, err = _tables([10, 3], [4, 2], [16, 8], 8, 4, 9, 3, 0, mangle=none)
    assert ok and err == 0 and want["slots"][:4] == [-1] * 4
    ok, want, err = _tables([10, 3], [4, 2], [16, 8], 8, 4, 9, 3, 0, mangle=null)
    assert ok and want["bad_slot"] and err == 1


def test_tables_steps_chain_on_another_stream():
    """Two steps, each reading what the one before it wrote, on a stream of the caller's."""
    s = torch.cuda.Stream()
    b, S = 4, 3
    table, ring, state = _i(np.zeros((S, 6))), _i([5, 6, 7, 8, 9, 1, 2, 3]), _i([6, 8])
    ctx, new, zero = _i([0, 0, 0]), _i([3, 5, 0]), _i([0, 0, 0])
    s.wait_stream(torch.cuda.current_stream())
    one = ssd.kv_block_tables(ctx, new, zero, table, ring, state, b, 10, 8, stream=s)
    two = ssd.kv_block_tables(one["seq_lens"], _i([2, 0, 1]), one["reserved_lens"], table, ring, one["ring_state"], b,
                              10, 8, stream=s)
    s.synchronize()
    # ring from entry 6: 2, 3, 5, 6, 7 ...: request 0 takes 2; request 1 takes 3 and 5; then 0 takes 6 and 2 takes 7
    assert table[0, :2].tolist() == [2, 6] and table[1, :2].tolist() == [3, 5] and table[2, 0].item() == 7
    assert two["slots"].tolist() == [2 * 4 + 3, 6 * 4, 7 * 4, -1, -1, -1, -1, -1]
    assert two["ring_state"].tolist() == [3, 3]


def test_tables_without_requests():
    got = ssd.kv_block_tables(_i([]), _i([]), _i([]), _i(np.zeros((0, 3))), _i([1, 2]), _i([1, 1]), 8, 4, 5)
    torch.cuda.synchronize()
    assert got["cu_seqlens"].tolist() == [0] and got["slots"].tolist() == [-1] * 5
    assert got["ring_state"].tolist() == [1, 1]


# -------------------------------------------------------------------- rope --

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 32, False), (80, 40, False), (8, 2, False), (8, 8, True),
                                         (256, 64, True), (112, 112, False), (256, 256, False), (40, 6, True),
                                         (128, 0, False)])
@pytest.mark.parametrize("H,Hkv,T", [(5, 1, 7), (32, 8, 3), (2, 2, 1)])
def test_norm_rope(dtype, D, rot, inter, H, Hkv, T):
    """Head sizes, rotated parts that end inside a lane's entries, both pairings; q, k and v as views of one packed
    projection; tokens without a slot; rows of the cache that are not written keep their bits."""
    g = torch.Generator(device=DEV).manual_seed(D * 31 + rot + T)
    qkv = torch.randn(T, (H + 2 * Hkv) * D + 8, generator=g, device=DEV).to(dtype)
    q = qkv[:, :H * D].view(T, H, D) if T == 1 else qkv[:, :H * D].unflatten(1, (H, D))
    k = qkv[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
    v = qkv[:, (H + Hkv) * D:(H + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    qw = torch.randn(D, generator=g, device=DEV)
    kw = torch.randn(D, generator=g, device=DEV)
    cs = torch.randn(50, rot, generator=g, device=DEV) if rot else None
    pos = _i(np.arange(T) * 7 % 50) if rot else None
    kv = F.poison((6, 2, 3, Hkv, D), dtype, DEV)  # keys and values of a block side by side
    kc, vc = kv[:, 0], kv[:, 1]
    slots = _i([(5 * t + 4) % 18 if t != 1 else -1 for t in range(T)])
    err = _err()
    qo, ko = ssd.kv_qk_norm_rope(q, k, pos, cs, qw, kw, 1e-5, inter, v, kc, vc, slots, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want, mag = F.norm_rope(x, w, cs, pos, 1e-5, inter)
        assert ((got.double().cpu() - want).abs() <= F.rope_bound(want, mag, D, dtype)).all()
    used = torch.zeros(18, dtype=torch.bool)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            used[s] = True
            assert torch.equal(kc[s // 3, s % 3], ko[t]) and torch.equal(vc[s // 3, s % 3], v[t])
    rest = kv.transpose(1, 2).reshape(18, 2, Hkv, D)[~used.to(DEV)]
    assert torch.isnan(rest).all()


@pytest.mark.parametrize("dtype,D,rot,inter", [(BF, 128, 128, False), (F32, 80, 40, False), (BF, 64, 64, True)])
def test_norm_rope_more_tokens_than_ctas(dtype, D, rot, inter):
    """Tokens beyond the grid: every CTA walks over several, one of them with a position that is none."""
    T, H, Hkv = 2500, 3, 1
    g = torch.Generator(device=DEV).manual_seed(D)
    q, k = torch.randn(T, H, D, generator=g, device=DEV).to(dtype), torch.randn(T, Hkv, D, generator=g, device=DEV).to(dtype)
    w = torch.randn(D, generator=g, device=DEV)
    cs = torch.randn(3000, rot, generator=g, device=DEV)
    at = np.arange(T)
    at[7] = 3000
    kc, vc = F.poison((320, 8, Hkv, D), dtype, DEV), F.poison((320, 8, Hkv, D), dtype, DEV)
    slots = np.random.default_rng(0).permutation(2560)[:T]
    qo, ko, err = F.poison(q.shape, dtype, DEV), F.poison(k.shape, dtype, DEV), _err()
    ssd.kv_qk_norm_rope(q, k, _i(at), cs, w, w, 1e-6, inter, k, kc, vc, _i(slots), q_out=qo, k_out=ko, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 2 and torch.isnan(qo[7]).all() and torch.isnan(ko[7]).all()
    keep = torch.arange(T) != 7
    at[7] = 0
    for got, x in ((qo, q), (ko, k)):
        want, mag = F.norm_rope(x, w, cs, _i(at), 1e-6, inter)
        assert ((got.double().cpu() - want).abs() <= F.rope_bound(want, mag, D, dtype))[keep].all()
    rows = torch.from_numpy(slots[keep.numpy()]).to(DEV)
    assert torch.equal(kc.flatten(0, 1)[rows], ko[keep.to(DEV)]) and torch.equal(vc.flatten(0, 1)[rows], k[keep.to(DEV)])


@pytest.mark.parametrize("dtype,D,rot,inter,H,Hkv", [
    (BF, 64, 64, False, 8, 2), (BF, 64, 16, True, 20, 4), (BF, 128, 128, False, 16, 16), (BF, 64, 40, False, 4, 1),
    (F32, 64, 64, False, 8, 1), (F32, 128, 12, True, 4, 4), (BF, 8, 8, True, 33, 1), (BF, 256, 256, False, 8, 4),
])
def test_norm_rope_tokens_side_by_side(dtype, D, rot, inter, H, Hkv):
    """Few heads and many tokens, of which a CTA has several at a time: the last ones alone, in place, some without a slot,
    with a slot or a position that is none."""
    T = 4803
    g = torch.Generator(device=DEV).manual_seed(D + H)
    q, k = torch.randn(T, H, D, generator=g, device=DEV).to(dtype), torch.randn(T, Hkv, D, generator=g, device=DEV).to(dtype)
    v = torch.randn(T, Hkv, D, generator=g, device=DEV).to(dtype)
    w = torch.randn(D, generator=g, device=DEV)
    cs = torch.randn(5000, rot, generator=g, device=DEV)
    at = np.arange(T) + 17
    at[[5, 2402]] = [-1, 5000]
    kc, vc = F.poison((T // 8 + 2, 8, Hkv, D), dtype, DEV), F.poison((T // 8 + 2, 8, Hkv, D), dtype, DEV)
    slots = np.random.default_rng(1).permutation(T)
    slots[[3, 4800]] = -1
    slots[4000] = (T // 8 + 2) * 8
    err, was = _err(), (q.clone(), k.clone())
    qo, ko = ssd.kv_qk_norm_rope(q, k, _i(at), cs, w, w, 1e-6, inter, v, kc, vc, _i(slots), q_out=q, k_out=k, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == ssd.DEVERR_METADATA | ssd.DEVERR_SLOT
    keep = torch.ones(T, dtype=torch.bool)
    keep[[5, 2402]] = False
    at[[5, 2402]] = 0
    for got, x in ((qo, was[0]), (ko, was[1])):
        want, mag = F.norm_rope(x, w, cs, _i(at), 1e-6, inter)
        assert ((got.double().cpu() - want).abs() <= F.rope_bound(want, mag, D, dtype))[keep].all()
        assert torch.equal(got[~keep.to(DEV)], x[~keep.to(DEV)])
    keep[[3, 4800, 4000]] = False
    rows = torch.from_numpy(slots[keep.numpy()]).to(DEV)
    assert torch.equal(kc.flatten(0, 1)[rows], ko[keep.to(DEV)]) and torch.equal(vc.flatten(0, 1)[rows], v[keep.to(DEV)])
    rest = torch.ones(kc.shape[0] * 8, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert torch.isnan(kc.flatten(0, 1)[rest]).all() and torch.isnan(vc.flatten(0, 1)[rest]).all()


@pytest.mark.parametrize("rot", [64, 40])
def test_norm_rope_in_place_and_without_norm(rot):
    T, H, Hkv, D = 9, 3, 3, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn(T, H, D, generator=g, device=DEV)
    k = torch.randn(T, Hkv, D, generator=g, device=DEV)
    cs = torch.randn(20, rot, generator=g, device=DEV)
    pos = _i(np.arange(T) + 3)
    wq, mq = F.norm_rope(q, None, cs, pos, 0, False)
    wk, mk = F.norm_rope(k, None, cs, pos, 0, False)
    a, b = ssd.kv_qk_norm_rope(q, k, pos, cs, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert a is q and ((a.double().cpu() - wq).abs() <= F.rope_bound(wq, mq, D, F32)).all()
    assert b is k and ((b.double().cpu() - wk).abs() <= F.rope_bound(wk, mk, D, F32)).all()


def test_norm_rope_reports_bad_positions_and_slots():
    T, H, D = 4, 2, 64
    q = torch.randn(T, H, D, device=DEV)
    cs = torch.randn(10, D, device=DEV)
    kc, vc = F.poison((2, 4, H, D), F32, DEV), F.poison((2, 4, H, D), F32, DEV)
    qo, ko, err = F.poison((T, H, D), F32, DEV), F.poison((T, H, D), F32, DEV), _err()
    ssd.kv_qk_norm_rope(q, q, _i([0, 10, -1, 9]), cs, v=q, k_cache=kc, v_cache=vc, slots=_i([0, 1, 2, 8]), q_out=qo,
                        k_out=ko, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 3
    assert torch.isnan(qo[1:3]).all() and torch.isfinite(qo[0]).all() and torch.isfinite(qo[3]).all()
    assert torch.isfinite(kc[0, 0]).all() and torch.isnan(kc.flatten(0, 1)[1:]).all() and torch.isnan(vc.flatten(0, 1)[1:]).all()


def test_norm_rope_zero_row_and_large_values():
    """An all-zero head stays zero (eps keeps the root finite); values near fp32's square root of the largest number."""
    q = torch.zeros(2, 1, 64, device=DEV)
    q[1] = 1e18
    qo, _ = ssd.kv_qk_norm_rope(q, q.clone(), q_weight=torch.ones(64, device=DEV))
    torch.cuda.synchronize()
    assert (qo[0] == 0).all() and torch.allclose(qo[1], torch.ones(1, 64, device=DEV), rtol=1e-5)


# --------------------------------------------------------------- attention --

def _tree(rng, n, words):
    rows, bits = [], []
    for i in range(n):
        up = bits[rng.integers(max(0, i - 5), i)] if i else 0
        bits.append(up | 1 << i)
    for m in bits:
        rows.append([(m >> 32 * w) & 0xFFFFFFFF for w in range(words)])
    return np.array(rows, np.uint32).reshape(n, words)


def _attn(dtype, H, Hkv, D, b, new, ctx, tree, seed=0, empty_rows=(), poison_new=(), scale=None, qk_gain=1.0,
          max_new=None, pack=True, extra_words=0):
    """Inputs with NaN in every page row that holds no cached token, and in front of and behind the packed tokens."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 77)
    S, T = len(new), sum(new)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    cols = max(-(-max(ctx) // b), 1) + 1
    table, total, _ = F.rand_pages(ctx, b, cols, 2, rng)
    table[table == 0] = 10 ** 6  # entries behind the context are never read
    kc, vc = F.poison((total, b, Hkv, D), dtype, DEV), F.poison((total, b, Hkv, D), dtype, DEV)
    for r in range(S):
        for j in range(-(-ctx[r] // b)):
            n = min(b, ctx[r] - j * b)
            kc[int(table[r, j]), :n] = torch.randn(n, Hkv, D, generator=g, device=DEV).to(dtype)
            vc[int(table[r, j]), :n] = torch.randn(n, Hkv, D, generator=g, device=DEV).to(dtype)
    pad = 3
    qkv = F.poison((T + 2 * pad, (H + 2 * Hkv) * D), dtype, DEV)
    qkv[pad:pad + T] = torch.randn(T, (H + 2 * Hkv) * D, generator=g, device=DEV).to(dtype)
    qkv[:, :H * D] *= qk_gain
    part = qkv[pad:pad + T]
    q = part[:, :H * D].unflatten(1, (H, D))
    k = part[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
    v = part[:, (H + Hkv) * D:].unflatten(1, (Hkv, D))
    if not pack:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    mask = None
    if tree:
        words = -(-max(max(new), 1) // 32) + extra_words
        mask = np.concatenate([_tree(rng, n, words) for n in new])
        for r, i in empty_rows:
            mask[cu[r] + i] = 0
        for r, i in poison_new:  # nobody but itself may see it
            t = cu[r] + i
            k[t], v[t] = float("nan"), float("nan")
            for j in range(new[r]):
                if j != i:
                    mask[cu[r] + j, i // 32] &= ~np.uint32(1 << i % 32)
    sc = D ** -0.5 if scale is None else scale
    return dict(q=q, k=k, v=v, kc=kc, vc=vc, cu=cu, ctx=ctx, table=table, mask=mask, scale=sc, new=new,
                max_new=max(new) if max_new is None else max_new)


def _run(c, err, **kw):
    mask = None if c["mask"] is None else torch.from_numpy(c["mask"].view(np.int32)).to(DEV)
    return ssd.kv_tree_attention(c["q"], c["k"], c["v"], c["kc"], c["vc"], _i(c["cu"]), _i(c["ctx"]), _i(c["table"]),
                                 c["max_new"], tree_mask=mask, scale=c["scale"], return_lse=True, err_word=err, **kw)


def _near(c, out, rows):
    """The output rows (a slice) are inside the bound."""
    want, wlse, mag, big, keys = F.attention(c["q"], c["k"], c["v"], c["kc"], c["vc"], c["cu"], c["ctx"], c["table"],
                                             c["mask"], c["scale"])
    tol, _ = F.attention_bound(want, wlse, mag, big, keys, c["q"].shape[2], c["q"].dtype)
    return bool(((out.double().cpu() - want).abs() <= tol)[rows].all())


def _check(c, nan_rows=()):
    err = _err()
    out, lse = _run(c, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    dtype, D = c["q"].dtype, c["q"].shape[2]
    want, wlse, mag, big, keys = F.attention(c["q"], c["k"], c["v"], c["kc"], c["vc"], c["cu"], c["ctx"], c["table"],
                                             c["mask"], c["scale"])
    tol, ltol = F.attention_bound(want, wlse, mag, big, keys, D, dtype)
    out, lse = out.double().cpu(), lse.double().cpu()
    live = torch.ones(out.shape[0], dtype=torch.bool)
    for t in nan_rows:
        live[t] = False
        assert torch.isnan(out[t]).all()
    bad = ((out - want).abs() > tol)[live]
    assert not torch.isnan(out[live]).any() and not bad.any(), float(((out - want).abs() / tol)[live].max())
    none = keys == 0
    assert (out[none] == 0).all() and torch.isneginf(lse[none]).all()
    some = live & ~none
    assert ((lse - wlse).abs() <= ltol)[some].all(), float(((lse - wlse).abs() / ltol)[some].max())
    return out


LAYOUTS = [  # dtype, query heads, key heads, head size, block size
    (BF, 8, 2, 128, 16), (BF, 4, 4, 64, 8), (BF, 8, 1, 128, 48), (BF, 10, 2, 64, 256), (BF, 5, 1, 128, 32),
    (BF, 16, 1, 128, 64), (BF, 40, 1, 128, 128), (BF, 128, 1, 64, 16),
    (F32, 8, 2, 128, 16), (F32, 4, 4, 64, 5), (F32, 3, 1, 256, 1), (F32, 20, 1, 40, 24),
    (BF, 8, 2, 128, 20), (BF, 2, 1, 256, 16), (BF, 6, 2, 96, 16), (BF, 130, 1, 64, 16),
]


@pytest.mark.parametrize("dtype,H,Hkv,D,b", LAYOUTS)
@pytest.mark.parametrize("tree", [False, True])
def test_attention_layouts(dtype, H, Hkv, D, b, tree):
    """Every kernel, head size, group and page size on a ragged batch: no context, contexts of one token, at and around
    page and tile ends, requests without new tokens, single tokens and several; stale page rows are NaN."""
    new = [1, 3, 0, 7, 2, 5, 1, 4]
    ctx = [0, 1, 40, 63, 64, 65, 300, b]
    _check(_attn(dtype, H, Hkv, D, b, new, ctx, tree, seed=D + H))


@pytest.mark.parametrize("dtype,D,group", [(BF, 128, 4), (BF, 64, 1), (BF, 128, 5), (BF, 128, 16), (F32, 64, 2)])
@pytest.mark.parametrize("n", [1, 15, 31, 33, 64, 65, 129])
def test_attention_tree_sizes(dtype, D, group, n):
    """Trees up to several mask words and key tiles; rows that see nothing at all and rows that see no draft."""
    c = _attn(dtype, group, 1, D, 16, [n, max(1, n // 2)], [0, 100], True, seed=n, extra_words=n % 2,
              empty_rows=[(0, n - 1), (1, 0)])
    _check(c)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("new,ctx", [([200], [0]), ([1], [0]), ([130, 1, 67], [70, 2000, 0]), ([257], [129])])
def test_attention_prompts(dtype, D, new, ctx):
    """Chains over several query tiles, behind a prefix or none."""
    _check(_attn(dtype, 4, 2, D, 16, new, ctx, False, seed=3))


@pytest.mark.parametrize("dtype,H,Hkv,D", [(BF, 8, 2, 128), (BF, 32, 1, 64), (F32, 4, 1, 128)])
def test_attention_long_caches_are_split(dtype, H, Hkv, D):
    """One long request beside short ones: its keys are cut over many CTAs and joined."""
    _check(_attn(dtype, H, Hkv, D, 16, [1, 2, 1], [20011, 5, 700], False, seed=9))


@pytest.mark.parametrize("dtype,H,Hkv,D", [(BF, 2, 1, 64), (BF, 4, 4, 128), (F32, 2, 1, 64)])
def test_attention_many_requests(dtype, H, Hkv, D):
    """More requests than a CTA has threads, most of them without new tokens, so that runs begin and end anywhere."""
    rng = np.random.default_rng(31)
    S = 450
    new = (rng.integers(1, 4, S) * (rng.random(S) < 0.3)).tolist()
    new[-1] = 2
    ctx = rng.integers(0, 150, S).tolist()
    _check(_attn(dtype, H, Hkv, D, 16, new, ctx, False, seed=31))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64)])
def test_attention_nan_drafts_stay_out(dtype, D):
    """A draft whose key and value are NaN touches nobody but itself."""
    c = _attn(dtype, 4, 1, D, 16, [9, 40], [33, 0], True, seed=4, poison_new=[(0, 4), (1, 0), (1, 35)])
    _check(c, nan_rows=[int(c["cu"][0]) + 4, int(c["cu"][1]), int(c["cu"][1]) + 35])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_infinite_values(dtype):
    """An infinite value that is seen gives infinity (or NaN against its opposite) in its column, and only there."""
    c = _attn(dtype, 4, 1, 64, 16, [6], [20], True, seed=8)
    c["v"][2, 0, 5] = float("inf")
    c["v"][3, 0, 9] = float("-inf")
    out, _ = _run(c, _err())
    torch.cuda.synchronize()
    bits = c["mask"][:, 0]
    for i in range(6):
        row = out[i]
        for col, j, inf in ((5, 2, float("inf")), (9, 3, float("-inf"))):
            if bits[i] >> j & 1:
                assert (row[:, col] == inf).all()
            else:
                assert torch.isfinite(row[:, col]).all()
        keep = [e for e in range(64) if e not in (5, 9)]
        assert torch.isfinite(row[:, keep]).all()


@pytest.mark.parametrize("H,D,new,ctx,tree", [
    (4, 128, [1], [777], False), (1, 64, [1, 2, 4], [63, 0, 129], True), (8, 128, [4, 4], [20000, 70], False),
    (32, 64, [1] * 40, list(range(40, 1640, 40)), False), (4, 64, [8, 3, 0, 5], [0, 300, 7, 64], True),
])
def test_attention_few_rows_keep_their_weights(H, D, new, ctx, tree):
    """Tiles of at most 32 rows hold the weights to 2^-15 (8 bits cut off, what is left rounded to 8).  Half of the keys have a weight that bf16 rounds down and
    values of 1, half one that it rounds up and values of -1: the outputs nearly cancel, and 8 bits would leave 2^-8 of
    the weights' sum, beside a rounding of the outputs of 2^-8 of their own, much smaller, size."""
    c = _attn(BF, H, 1, D, 16, new, ctx, tree, seed=48, scale=1.0)
    c["q"].zero_()
    c["q"][..., 0], c["q"][..., 1] = 1.0, 2.0 ** -8
    scores = [np.log(0.5 * (1 + f / 128)) for f in (0.4, 0.6)]

    def fill(k, v, at):  # rows at positions `at` of a request
        for odd in (0, 1):
            rows = [i for i, p in enumerate(at) if p % 2 == odd]
            first = torch.tensor(scores[odd]).to(BF)
            k[rows] = 0.0
            k[rows, :, 0] = first.to(DEV)
            k[rows, :, 1] = float((scores[odd] - first.double()) * 256)
            v[rows] = 1.0 - 2.0 * odd
    for r, n in enumerate(ctx):
        for j in range(-(-n // 16)):
            page, here = int(c["table"][r, j]), min(16, n - 16 * j)
            fill(c["kc"][page, :here], c["vc"][page, :here], range(16 * j, 16 * j + here))
            if j == 0:  # one key of weight 1 sets the maximum
                c["kc"][page, 0], c["vc"][page, 0] = 0.0, 0.0
        fill(c["k"][c["cu"][r]:c["cu"][r + 1]], c["v"][c["cu"][r]:c["cu"][r + 1]], range(n, n + new[r]))
    c["k"][c["cu"][:-1][np.array(new) > 0]] = 0.0  # here too, of the first new token
    c["v"][c["cu"][:-1][np.array(new) > 0]] = 0.0
    err = _err()
    out, _ = _run(c, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want, wlse, mag, big, keys = F.attention(c["q"], c["k"], c["v"], c["kc"], c["vc"], c["cu"], c["ctx"], c["table"],
                                             c["mask"], c["scale"])
    _, rel = F.attention_bound(want, wlse, mag, big, keys, D, F32)
    tol = 1.01 * (rel + 2.0 ** -15)[..., None] * mag + 1.01 * F.UBF * want.abs() + 1e-30
    assert ((out.double().cpu() - want).abs() <= tol).all(), float(((out.double().cpu() - want).abs() / tol).max())


@pytest.mark.parametrize("dtype,H,D,new", [(BF, 4, 128, [1, 3]), (BF, 8, 64, [4, 1]), (BF, 8, 128, [30, 9]), (F32, 4, 64, [2, 2])])
def test_attention_infinite_cached_values(dtype, H, D, new):
    """An infinite value of the cache gives infinity in its column, whatever its weight's parts: one, none or several of
    them, and their signs."""
    c = _attn(dtype, H, 1, D, 16, new, [200, 1000], False, seed=49)
    for r, (pos, col, inf) in enumerate([(70, 3, float("inf")), (999, 40, float("-inf"))]):
        c["vc"][int(c["table"][r, pos // 16]), pos % 16, 0, col] = inf
    out, _ = _run(c, _err())
    torch.cuda.synchronize()
    first = out[:new[0]], out[new[0]:]
    for part, col, inf in ((first[0], 3, float("inf")), (first[1], 40, float("-inf"))):
        assert (part[..., col] == inf).all()
        assert torch.isfinite(part[..., :col]).all() and torch.isfinite(part[..., col + 1:]).all()


@pytest.mark.parametrize("dtype,D", [(BF, 64), (BF, 96), (F32, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_values_of_vanishing_weights_count(dtype, D, bad):
    """A key that is seen, but so far below the others that its weight is zero in fp32: its value is no number, and neither
    is the result of those that see it; the others' columns and rows are."""
    c = _attn(dtype, 4, 1, D, 16, [6, 2], [20, 5], True, seed=47)
    c["mask"][:] = [[0b1], [0b11], [0b101], [0b1001], [0b10011], [0b100101], [0b1], [0b11]]
    c["q"][..., 0] = 1000.0
    far = c["k"][:, 0, 0]
    far.fill_(0.0)
    for r in range(2):
        for page in c["table"][r, :-(-c["ctx"][r] // 16)]:
            c["kc"][int(page), :, 0, 0] = torch.where(torch.isnan(c["kc"][int(page), :, 0, 0]), float("nan"), 0.0)
    far[1] = -1000.0  # seen by tokens 1 and 4
    c["v"][1, 0, 3] = bad
    last = c["kc"][int(c["table"][1, 0]), 4, 0]  # the second request's last cached token
    last[0] = -1000.0
    c["vc"][int(c["table"][1, 0]), 4, 0, 7] = bad
    out, lse = _run(c, _err())
    torch.cuda.synchronize()
    sees = torch.zeros_like(out, dtype=torch.bool)
    sees[[1, 4], :, 3] = True
    sees[6:, :, 7] = True
    assert torch.equal(~torch.isfinite(out), sees) and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype,gain", [(BF, 60.0), (F32, 60.0), (BF, 0.0), (F32, 1e-3)])
def test_attention_score_ranges(dtype, gain):
    """Peaked scores (hundreds apart, so running maxima jump), and equal ones."""
    _check(_attn(dtype, 8, 2, 128, 16, [4, 1, 33], [500, 1000, 77], False, seed=6, qk_gain=gain))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
def test_attention_scales(dtype, scale):
    """Any finite scale, zero (the mean of what is seen) and negative ones among them."""
    _check(_attn(dtype, 4, 2, 64, 16, [3, 1, 20], [100, 40, 0], True, seed=14, scale=scale))


def test_attention_outputs_made_for_another_stream():
    """Outputs and workspace that a call allocates itself, used on a stream other than the current one, are not handed
    out again while that stream still works on them."""
    c = _attn(BF, 8, 2, 128, 16, [2, 1, 30], [3000, 40, 900], False, seed=23)
    want, lse = _run(c, _err())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mask = None
    args = (c["q"], c["k"], c["v"], c["kc"], c["vc"], _i(c["cu"]), _i(c["ctx"]), _i(c["table"]), c["max_new"])
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        out, l2 = ssd.kv_tree_attention(*args, tree_mask=mask, return_lse=True, stream=s)
        outs.append((out, l2))
        del out, l2
        for size in (1 << 12, 1 << 20, 1 << 22):  # would land in the freed workspace
            torch.full((size,), float("nan"), device=DEV)
    torch.cuda.synchronize()
    for out, l2 in outs:
        assert torch.equal(out, want) and torch.equal(l2, lse)


def test_attention_does_not_depend_on_the_hint():
    """max_new_tokens sizes the tiles; every value of it gives a result inside the bound."""
    for hint in (0, 1, 10, 33, 1000):
        _check(_attn(BF, 4, 1, 128, 16, [40, 3, 1], [50, 200, 0], True, seed=12, max_new=hint))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_is_repeatable_and_stream_ordered(dtype):
    """The same bits every time, on another stream, and with a workspace full of NaN."""
    c = _attn(dtype, 8, 2, 128, 16, [2, 1, 30], [3000, 40, 900], False, seed=21)
    a, la = _run(c, _err())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    b, lb = _run(c, _err(), stream=s, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_reports_bad_metadata(dtype):
    """A context beyond the table, more drafts than mask bits, decreasing offsets: the request's rows stay unwritten and
    the others come out right.  A block id that is none reads as zeros."""
    def case(new=(2, 3)):
        return _attn(dtype, 4, 2, 64, 16, list(new), [30, 50], True, seed=2)

    c, good = case(), case()
    c["ctx"] = [30, 16 * c["table"].shape[1] + 1]
    out, err = F.poison(c["q"].shape, dtype, DEV), _err()
    _run(c, err, out=out)
    torch.cuda.synchronize()
    assert int(err.item()) == 2 and _near(good, out, slice(0, 2)) and torch.isnan(out[2:]).all()

    c, good = case((2, 40)), case((2, 40))
    c["mask"] = c["mask"][:, :1].copy()
    out, err = F.poison(c["q"].shape, dtype, DEV), _err()
    _run(c, err, out=out)
    torch.cuda.synchronize()
    assert int(err.item()) == 2 and _near(good, out, slice(0, 2)) and torch.isnan(out[2:]).all()

    c = case()
    c["cu"] = np.array([0, 9, 5], np.int32)
    out, err = F.poison(c["q"].shape, dtype, DEV), _err()
    _run(c, err, out=out)
    torch.cuda.synchronize()
    assert int(err.item()) == 2 and torch.isnan(out).all()

    c = case()
    c["table"][1, 1] = -5
    err = _err()
    out, _ = _run(c, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 1
    c["kc"] = torch.cat([c["kc"], torch.zeros_like(c["kc"][:1])])
    c["vc"] = torch.cat([c["vc"], torch.zeros_like(c["vc"][:1])])
    c["table"][1, 1] = c["kc"].shape[0] - 1
    assert _near(c, out, slice(0, 5))


def test_attention_cache_views_and_far_blocks():
    """Keys and values interleaved block by block, with a block stride that puts the last blocks beyond 2^31
    elements."""
    c = _attn(BF, 4, 1, 128, 16, [3, 1], [100, 40], False, seed=5)
    nb, b, H, D = c["kc"].shape
    stride = (1 << 32) // nb // 8 * 8
    big = torch.empty(stride * (nb - 1) + 2 * b * H * D, dtype=BF, device=DEV)
    kc = big.as_strided((nb, b, H, D), (stride, H * D, D, 1), 0)
    vc = big.as_strided((nb, b, H, D), (stride, H * D, D, 1), b * H * D)
    kc.copy_(c["kc"])
    vc.copy_(c["vc"])
    c["kc"], c["vc"] = kc, vc
    _check(c)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_waits_are_bounded(D):
    """With a limit of a few cycles the tensor-core kernel's waits give up: the call returns, the timeout is reported and
    the next call on the same context is right."""
    c = _attn(BF, 8, 2, D, 16, [2, 1, 30], [3000, 40, 900], False, seed=22)
    err = _err()
    _run(c, err, wait_limit_cycles=20)
    torch.cuda.synchronize()
    assert int(err.item()) == ssd.DEVERR_TIMEOUT
    _check(c)


PAIRS = [  # query heads, key heads, head size, block size, tree, new tokens, cached
    (8, 1, 128, 16, True, [17, 33, 0, 100, 48, 16, 64], [0, 5000, 7, 64, 130, 0, 2049]),
    (16, 2, 64, 32, False, [49, 1, 16, 31, 0, 90], [700, 64, 0, 3000, 100, 1]),
    (5, 1, 128, 64, False, [26, 51, 400, 2], [65, 1000, 0, 3]),
    (4, 4, 64, 16, True, [300, 129], [100, 0]),
    (40, 1, 128, 16, False, [4, 7, 3, 13], [40, 0, 9000, 500]),
    (128, 1, 64, 8, True, [1, 2, 3, 4], [63, 1, 300, 0]),
]


@pytest.mark.parametrize("H,Hkv,D,b,tree,new,ctx", PAIRS)
def test_attention_pairs_of_row_tiles(H, Hkv, D, b, tree, new, ctx):
    """Requests of more rows than a tensor-core tile on the average, which two tiles work on together: requests that end
    in the first tile or the second, or have one token or none, few rows of a tile in use, and several items a request."""
    c = _attn(BF, H, Hkv, D, b, new, ctx, tree, seed=len(new) + H, empty_rows=[(0, 0)] if tree else ())
    _check(c)


def test_attention_pairs_keep_bad_values_apart():
    """NaN drafts and an infinite value in the second tile of a pair, and in keys that only one of the tiles sees."""
    c = _attn(BF, 8, 1, 128, 16, [40, 30], [33, 200], True, seed=40, poison_new=[(0, 2), (0, 39), (1, 20)])
    _check(c, nan_rows=[2, 39, 60])
    c = _attn(BF, 8, 1, 64, 16, [40], [100], False, seed=41)
    c["v"][20, 0, 7] = float("inf")  # a token of the second tile: the first one's rows stay finite
    out, _ = _run(c, _err())
    torch.cuda.synchronize()
    assert torch.isfinite(out[:20]).all() and (out[20:, :, 7] == float("inf")).all()
    assert torch.isfinite(out[20:, :, :7]).all() and torch.isfinite(out[20:, :, 8:]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("limit", [20, 20000])
def test_attention_waits_of_pairs_are_bounded(D, limit):
    """As above, where two tiles share their loads: one that gives up ends the other's waits, too."""
    c = _attn(BF, 8, 1, D, 16, [40, 30, 64, 17], [3000, 400, 0, 900], False, seed=42)
    err = _err()
    _run(c, err, wait_limit_cycles=limit)
    torch.cuda.synchronize()
    assert int(err.item()) == ssd.DEVERR_TIMEOUT or (limit > 20 and int(err.item()) == 0)
    _check(c)


@pytest.mark.parametrize("H,D,new,ctx", [(8, 64, [2, 1, 30], [300, 40, 90]), (4, 128, [1] * 40, [100] * 40),
                                         (8, 128, [40, 30, 64, 17], [300, 400, 0, 90])])
def test_attention_that_gave_up_leaves_nothing_behind(H, D, new, ctx):
    """Waits that give up at any time, in runs of so few tiles that all copies are asked for before: the next call, queued at
    once, gets the shared memory that copies of the one before would still be written to, and is right."""
    c = _attn(BF, H, 1, D, 16, new, ctx, False, seed=45)
    good, lse = _run(c, _err())
    errs, outs = [], []
    for limit in [1, 20, 100, 300] + list(range(500, 6000, 250)):
        errs.append(_err())
        _run(c, errs[-1], wait_limit_cycles=limit)
        outs.append(_run(c, None))
    torch.cuda.synchronize()
    assert all(int(e.item()) in (0, ssd.DEVERR_TIMEOUT) for e in errs) and int(errs[0].item()) == ssd.DEVERR_TIMEOUT
    for o, l in outs:
        assert torch.equal(o, good) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype,H,Hkv,D,new,ctx", [
    (BF, 5, 1, 64, [20011, 3, 4096], [100, 70000, 0]), (BF, 8, 1, 128, [9001, 517], [33, 64]),
    (BF, 1, 1, 64, [30000], [0]), (F32, 3, 1, 64, [3001, 1], [65, 5000]),
])
def test_attention_long_prompts_are_means(dtype, H, Hkv, D, new, ctx):
    """Chains of many row tiles, which runs begin and end in anywhere.  With queries of zero every weight is one: a token's
    output is the mean of the values up to it, and its lse the logarithm of their number.  Sums of n terms in fp32 are
    off by n 2^-24 of the mean magnitude at most, before the output's own rounding."""
    rng = np.random.default_rng(51)
    g = torch.Generator(device=DEV).manual_seed(51)
    T, b = sum(new), 16
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table, total, _ = F.rand_pages(ctx, b, -(-max(ctx) // b) + 1, 1, rng)
    kc = torch.randn(total, b, Hkv, D, generator=g, device=DEV).to(dtype)
    vc, k, v = torch.randn_like(kc), *(torch.randn(T, Hkv, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    q = torch.zeros(T, H, D, dtype=dtype, device=DEV)
    err = _err()
    out, lse = ssd.kv_tree_attention(q, k, v, kc, vc, _i(cu), _i(ctx), _i(table), max(new), return_lse=True, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for r in range(len(new)):
        pages = torch.from_numpy(table[r, :-(-ctx[r] // b)].astype(np.int64)).to(DEV)
        cached = vc[pages].reshape(-1, Hkv, D)[:ctx[r]].double()
        mine = torch.cat([cached, v[cu[r]:cu[r + 1]].double()])
        count = torch.arange(1, len(mine) + 1, device=DEV, dtype=torch.float64)[:, None, None]
        want, mag = (mine.cumsum(0) / count)[ctx[r]:], (mine.abs().cumsum(0) / count)[ctx[r]:]
        n = count[ctx[r]:]
        tol = (2 * n + 8) * F.U32 * mag + (F.UBF if dtype == BF else F.U32) * want.abs()
        got = out[cu[r]:cu[r + 1]].double().unflatten(1, (Hkv, H // Hkv))
        assert ((got - want[:, :, None]).abs() <= tol[:, :, None]).all()
        want_lse = n[:, 0].log()
        assert ((lse[cu[r]:cu[r + 1]].double() - want_lse).abs() <= 16 * F.U32 * (1 + want_lse)).all()


def test_attention_pairs_do_not_depend_on_the_hint():
    """Tiles of as many tokens as a request is said to have, two of them side by side; and a batch where two tiles would
    work together, but no token belongs to a request."""
    for hint in (0, 1, 7, 1000):
        _check(_attn(BF, 8, 1, 128, 16, [40, 64, 1], [50, 0, 200], True, seed=43, max_new=hint))
    c = _attn(BF, 8, 1, 128, 16, [40], [100], False, seed=44)
    c["cu"] = np.array([0, 0], np.int32)
    out = F.poison((40, 8, 128), BF, DEV)
    _run(c, _err(), out=out)
    torch.cuda.synchronize()
    assert torch.isnan(out).all()


def test_attention_without_tokens():
    c = _attn(BF, 4, 1, 128, 16, [0, 0], [100, 40], False, seed=5)
    out, lse = _run(c, _err())
    torch.cuda.synchronize()
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    # tokens behind the last request: nothing is theirs, nothing is written
    c = _attn(BF, 4, 1, 128, 16, [5], [100], False, seed=5)
    c["cu"] = np.array([0, 0], np.int32)
    out = F.poison((5, 4, 128), BF, DEV)
    _run(c, _err(), out=out)
    torch.cuda.synchronize()
    assert torch.isnan(out).all()


# ------------------------------------------------------------------ commit --

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hkv,D", [(8, 128), (1, 8), (3, 40)])
def test_commit_paths(dtype, Hkv, D):
    g = torch.Generator(device=DEV).manual_seed(1)
    new = [5, 0, 16, 1, 9]
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    kv = torch.randn(T, 2 * Hkv * D, generator=g, device=DEV).to(dtype)
    k, v = kv[:, :Hkv * D].unflatten(1, (Hkv, D)), kv[:, Hkv * D:].unflatten(1, (Hkv, D))
    path = np.array([[0, 2, 4], [9, 9, 9], [1, 7, 15], [0, 5, 5], [8, 8, 8]])
    lens, ctx = [3, 0, 2, 1, 0], [10, 20, 30, 40, 50]
    slots = np.random.default_rng(0).permutation(60)[:T]
    slots[cu[2] + 1] = -1  # a token without a slot
    kc, vc, err = F.poison((12, 5, Hkv, D), dtype, DEV), F.poison((12, 5, Hkv, D), dtype, DEV), _err()
    out = ssd.kv_commit_tokens(k, v, kc, vc, _i(slots), _i(cu), _i(ctx), _i(path), _i(lens), err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and out.tolist() == [13, 20, 32, 41, 50]
    wk, wv = F.poison((60, Hkv, D), dtype, DEV), F.poison((60, Hkv, D), dtype, DEV)
    for r in range(5):
        for i in range(lens[r]):
            s = slots[cu[r] + i]
            if s >= 0:
                wk[s], wv[s] = k[cu[r] + path[r, i]], v[cu[r] + path[r, i]]
    bits = torch.int16 if dtype == BF else torch.int32
    assert torch.equal(kc.view(60, Hkv, D).view(bits), wk.view(bits))
    assert torch.equal(vc.view(60, Hkv, D).view(bits), wv.view(bits))


def test_commit_all_tokens_and_errors():
    T, Hkv, D = 11, 2, 64
    k = torch.randn(T, Hkv, D, device=DEV)
    kc, vc = F.poison((4, 4, Hkv, D), F32, DEV), F.poison((4, 4, Hkv, D), F32, DEV)
    slots = _i([15, 3, 2, 1, 0, 4, 5, 6, 7, 8, 9, -1, -1])  # a padded slot map
    assert ssd.kv_commit_tokens(k, -k, kc, vc, slots) is None
    torch.cuda.synchronize()
    assert torch.equal(kc.flatten(0, 1)[15], k[0]) and torch.equal(vc.flatten(0, 1)[9], -k[10])
    assert torch.isnan(kc.flatten(0, 1)[10:15]).all()
    kc, vc, err = F.poison((4, 4, Hkv, D), F32, DEV), F.poison((4, 4, Hkv, D), F32, DEV), _err()
    out = ssd.kv_commit_tokens(k, k, kc, vc, _i([0, 1, 2, 3, 4, 5, 99, 7, 8, 9, 10]), _i([0, 3, 6, 9, 11]), _i([1, 1, 1, 1]),
                               _i([[0, 1], [0, 3], [0, 1], [1, 0]]), _i([3, 2, 2, 1]), err_word=err)
    torch.cuda.synchronize()
    # request 0: more steps than columns; 1: a step that is none of its tokens; 2: a slot that is none
    assert int(err.item()) == 3 and out.tolist() == [1, 3, 3, 2]
    flat = kc.flatten(0, 1)
    assert torch.isnan(flat[:3]).all() and torch.equal(flat[3], k[3]) and torch.isnan(flat[4]).all()
    assert torch.equal(flat[7], k[7]) and torch.equal(flat[9], k[10])


def test_commit_of_paths_without_requests():
    k, kc = torch.ones(3, 1, 8, device=DEV), torch.zeros(1, 4, 1, 8, device=DEV)
    out = ssd.kv_commit_tokens(k, k, kc, kc.clone(), _i([0, 1, 2]), _i([0]), _i([]), _i(np.zeros((0, 2))), _i([]))
    torch.cuda.synchronize()
    assert out.shape == (0,) and (kc == 0).all()


# ------------------------------------------------------------------ binding --

@pytest.mark.parametrize("word", [torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int16),
                                  torch.zeros(1, dtype=torch.uint8), torch.zeros(1)])
def test_an_error_word_is_32_bits(word):
    k, kc = torch.zeros(2, 1, 8, device=DEV), torch.zeros(1, 2, 1, 8, device=DEV)
    with pytest.raises(ValueError, match="err_word"):
        ssd.kv_commit_tokens(k, k, kc, kc.clone(), _i([0, 1]), err_word=word.to(DEV))


def test_a_workspace_with_gaps_is_refused():
    """Its bytes do not lie side by side: the kernels would write between them, and beyond the last."""
    c = _attn(BF, 4, 1, 64, 16, [2], [20], False, seed=46)
    room = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        _run(c, None, workspace=room[::2])
    with pytest.raises(ssd.SSDError):
        _run(c, None, workspace=room[:1])
    out, _ = _run(c, None, workspace=room)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()


class _Fresh(dict):
    """A mapping whose values live no longer than who asks for them keeps them: views of one buffer, counted."""
    alive = 0

    class View(torch.Tensor):
        def __del__(self):
            _Fresh.alive -= 1

    def __getitem__(self, key):
        if key == "ring_state":
            _Fresh.seen = _Fresh.alive  # of the values asked for before
        v = super().__getitem__(key).view(-1).as_subclass(self.View)
        _Fresh.alive += 1
        return v


def test_outputs_made_on_access_are_kept_for_the_call():
    """Values of ``out`` are held until the call is queued, and an error in looking one up is the caller's to see."""
    args = (_i([3, 0]), _i([2, 1]), _i([3, 0]), _i([[1, 0], [0, 0]]), _i([2, 3, 4]), _i([0, 3]), 4, 9, 5)
    want = ssd.kv_block_tables(*args)
    args = args[:3] + (_i([[1, 0], [0, 0]]),) + args[4:]
    room = _Fresh({k: torch.zeros_like(v) for k, v in want.items()})
    assert ssd.kv_block_tables(*args, out=room) is room and _Fresh.seen == 3 and _Fresh.alive == 0
    torch.cuda.synchronize()
    for k, v in want.items():
        assert torch.equal(dict.__getitem__(room, k), v), k
    del room["token_req"]
    ssd.kv_block_tables(*args, out=room)
    torch.cuda.synchronize()

    class Broken(dict):
        def __getitem__(self, key):
            if key == "token_req":
                raise RuntimeError("no access")
            return super().__getitem__(key)

    with pytest.raises(RuntimeError, match="no access"):
        ssd.kv_block_tables(*args, out=Broken(room))


def test_a_flag_without_a_truth_value_is_refused():
    """The exception is the flag's own, and nothing is queued."""
    q = torch.zeros(1, 1, 8, device=DEV)
    with pytest.raises(ValueError, match="truth value"):
        ssd.kv_qk_norm_rope(q, q, interleaved=np.zeros(2))
    c = _attn(BF, 4, 1, 64, 16, [2], [20], False, seed=46)
    with pytest.raises(ValueError, match="truth value"):
        ssd.kv_tree_attention(c["q"], c["k"], c["v"], c["kc"], c["vc"], _i(c["cu"]), _i(c["ctx"]), _i(c["table"]), 2,
                              return_lse=np.zeros(2))


def _four_calls(stream):
    """The four calls on the same inputs; everything that they allocate."""
    g = torch.Generator(device=DEV).manual_seed(50)
    k = torch.randn(3, 2, 64, generator=g, device=DEV)
    kc = torch.randn(4, 16, 2, 64, generator=g, device=DEV)
    q = torch.randn(3, 4, 64, generator=g, device=DEV)
    cu, ctx, table, one = _i([0, 1, 3]), _i([20, 9]), _i([[1, 2], [3, 0]]), _i([1, 2])
    args = (ctx, one, ctx, table.clone(), _i([2, 3, 4]), _i([0, 3]), 16, 9, 5)
    slots, kn, vn = _i([5, 7, 9]), kc.clone(), kc.clone()
    torch.cuda.synchronize()

    def run():
        tables = ssd.kv_block_tables(*args, stream=stream)
        return [tables[key] for key in sorted(tables)] + list(ssd.kv_qk_norm_rope(q, k, stream=stream)) + \
            list(ssd.kv_tree_attention(q, k, k, kc, kc, cu, ctx, table, 2, return_lse=True, stream=stream)) + \
            [ssd.kv_commit_tokens(k, k, kn, vn, slots, cu, ctx, stream=stream)]
    return run


@pytest.mark.parametrize("as_number", [False, True])
def test_outputs_for_another_stream_have_no_work_to_come(as_number):
    """Memory that the current stream has yet to write for its last owner is not what a call on another stream gets."""
    want = _four_calls(None)()
    s = torch.cuda.Stream()
    run = _four_calls(s.cuda_stream if as_number else s)
    torch.cuda.empty_cache()
    torch.cuda._sleep(40_000_000)
    for _ in range(4):  # freed at once, filled when the current stream gets there
        last = [torch.full((n,), 7, dtype=torch.int32, device=DEV) for n in (4, 100, 128, 300, 500, 1000, 1 << 16, 1 << 20)]
        del last
    got = run()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_mask_without_words_is_refused():
    """A tensor of no elements has no pointer: it is not a chain's missing mask."""
    c = _attn(BF, 4, 1, 64, 16, [2, 3], [20, 0], True, seed=52)
    c["mask"] = c["mask"][:, :0].copy()
    with pytest.raises(ValueError, match="tree_mask must have a word"):
        _run(c, None)
    out, lse = _run(_attn(BF, 4, 1, 64, 16, [0, 0], [20, 0], False, seed=52) | dict(mask=np.zeros((0, 0), np.uint32)), None)
    assert out.shape[0] == 0 and lse.shape[0] == 0


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        cuda_stream, device_index = 0, torch.cuda.current_device() + 1

    k, kc = torch.zeros(2, 1, 8, device=DEV), torch.zeros(1, 2, 1, 8, device=DEV)
    with pytest.raises(ValueError, match="stream is on cuda"):
        ssd.kv_commit_tokens(k, k, kc, kc.clone(), _i([0, 1]), stream=Elsewhere())
    torch.cuda.synchronize()
    assert (kc == 0).all()


def _refused(call, good, over, error, match):
    """The call with good arguments passes; with some of them replaced it is refused by the right exception."""
    call(**good)
    with pytest.raises(error, match=match):
        call(**{**good, **over(good)})
    torch.cuda.synchronize()


def _gaps(t):  # the same values, with rows that are not dense
    return torch.stack([t, t], -1)[..., 0]


@pytest.mark.parametrize("over,error,match", [
    (lambda a: dict(new_lens=_i([1])), ValueError, "new_lens must be int32 of shape"),
    (lambda a: dict(context_lens=a["context_lens"].long()), ValueError, "context_lens must be int32"),
    (lambda a: dict(block_table=a["block_table"][0]), ValueError, "block_table must be int32"),
    (lambda a: dict(block_table=_gaps(a["block_table"])), ValueError, "block_table must be contiguous"),
    (lambda a: dict(ring_state=_i([0, 3, 0])), ValueError, "ring_state"),
    (lambda a: dict(max_tokens=-1), ValueError, "max_tokens must not be negative"),
    (lambda a: dict(max_tokens=1 << 40), ValueError, "max_tokens must fit 32 bits"),
    (lambda a: dict(block_size=0), ssd.SSDError, "kv_block_tables"),
    (lambda a: dict(block_size="16"), TypeError, "integer"),
    (lambda a: dict(out={}), KeyError, "cu_seqlens"),
    (lambda a: dict(reserved_lens=a["reserved_lens"].cpu()), ValueError, "reserved_lens must be a CUDA tensor"),
    (lambda a: dict(free_ring=None), ValueError, "free_ring is required"),
])
def test_tables_refuse_bad_tensors(over, error, match):
    good = dict(context_lens=_i([3, 0]), new_lens=_i([2, 1]), reserved_lens=_i([3, 0]), block_table=_i([[1, 0], [0, 0]]),
                free_ring=_i([2, 3, 4]), ring_state=_i([0, 3]), block_size=4, num_blocks=9, max_tokens=5)
    _refused(ssd.kv_block_tables, good, over, error, match)


@pytest.mark.parametrize("over,error,match", [
    (lambda a: dict(q=a["q"][0]), ValueError, "q and k must be"),
    (lambda a: dict(q=a["q"].half()), ValueError, "q must be bfloat16 or float32"),
    (lambda a: dict(k=a["k"].float()), ValueError, "k must be bfloat16"),
    (lambda a: dict(k=a["k"][:2]), ValueError, "k must be"),
    (lambda a: dict(q=_gaps(a["q"])), ValueError, "rows of q must be dense"),
    (lambda a: dict(v=a["v"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "rows of v must be dense"),
    (lambda a: dict(q=torch.zeros(5 * 4 * 64 + 1, dtype=BF, device=DEV)[1:].view(5, 4, 64)), ssd.SSDError, "kv_qk_norm_rope"),
    (lambda a: dict(q=torch.zeros(5, 4 * 64 + 4, dtype=BF, device=DEV)[:, :256].unflatten(1, (4, 64))), ssd.SSDError, "kv_qk"),
    (lambda a: dict(q=torch.zeros(5, 3, 64, dtype=BF, device=DEV)), ssd.SSDError, "kv_qk_norm_rope"),
    (lambda a: dict(positions=a["positions"].long()), ValueError, "positions must be int32"),
    (lambda a: dict(positions=None), ValueError, "positions is required"),
    (lambda a: dict(cos_sin=a["cos_sin"].to(BF)), ValueError, "cos_sin must be float32"),
    (lambda a: dict(cos_sin=a["cos_sin"][:, :63].contiguous()), ssd.SSDError, "kv_qk_norm_rope"),
    (lambda a: dict(q_weight=a["q_weight"][:32].contiguous()), ValueError, "q_weight must be float32"),
    (lambda a: dict(k_weight=a["k_weight"].to(BF)), ValueError, "k_weight must be float32"),
    (lambda a: dict(slots=a["slots"][:4]), ValueError, "slots must be int32"),
    (lambda a: dict(v_cache=None), ValueError, "v_cache is required"),
    (lambda a: dict(v_cache=a["v_cache"].float()), ValueError, "k_cache and v_cache must be"),
    (lambda a: dict(k_cache=a["k_cache"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "blocks of k_cache"),
    (lambda a: dict(k_cache=torch.zeros(4, 8, 2, 64, dtype=BF, device=DEV)[:, :4]), ValueError, "same block stride"),
    (lambda a: dict(q_out=torch.zeros(5, 4, 64, device=DEV)), ValueError, "q_out must be bfloat16"),
    (lambda a: dict(k_out=_gaps(a["k"])), ValueError, "k_out must be contiguous"),
    (lambda a: dict(eps="x"), TypeError, "real number|float"),
])
def test_norm_rope_refuses_bad_tensors(over, error, match):
    x = torch.zeros(5, 8, 64, dtype=BF, device=DEV)
    good = dict(q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], positions=_i(range(5)), cos_sin=torch.ones(8, 64, device=DEV),
                q_weight=torch.ones(64, device=DEV), k_weight=torch.ones(64, device=DEV), slots=_i(range(5)),
                k_cache=torch.zeros(4, 4, 2, 64, dtype=BF, device=DEV), v_cache=torch.zeros(4, 4, 2, 64, dtype=BF, device=DEV))
    _refused(ssd.kv_qk_norm_rope, good, over, error, match)


@pytest.mark.parametrize("over,error,match", [
    (lambda a: dict(q=a["q"][0]), ValueError, "q and k_new must be"),
    (lambda a: dict(k_new=a["k_new"].float()), ValueError, "k_new must be bfloat16"),
    (lambda a: dict(v_new=a["v_new"][:2]), ValueError, "v_new must be"),
    (lambda a: dict(q=_gaps(a["q"])), ValueError, "rows of q must be dense"),
    (lambda a: dict(k_cache=a["k_cache"][:, :, :1]), ValueError, "k_cache and v_cache must be"),
    (lambda a: dict(cu_seqlens=_i([])), ValueError, "cu_seqlens must have an entry more"),
    (lambda a: dict(cu_seqlens=_i([0, 1, 3, 3])), ValueError, "context_lens must be int32"),
    (lambda a: dict(context_lens=a["context_lens"].long()), ValueError, "context_lens must be int32"),
    (lambda a: dict(block_table=a["block_table"][:1]), ValueError, "block_table must be int32"),
    (lambda a: dict(tree_mask=a["tree_mask"][:2]), ValueError, "tree_mask must be int32"),
    (lambda a: dict(tree_mask=a["tree_mask"].long()), ValueError, "tree_mask must be int32"),
    (lambda a: dict(max_new_tokens=-1), ssd.SSDError, "kv_tree_attention"),
    (lambda a: dict(max_new_tokens=1 << 31), ValueError, "max_new_tokens must fit 32 bits"),
    (lambda a: dict(scale=float("inf")), ssd.SSDError, "kv_tree_attention"),
    (lambda a: dict(wait_limit_cycles=-1), ssd.SSDError, "kv_tree_attention"),
    (lambda a: dict(out=torch.zeros(3, 4, 64, device=DEV)), ValueError, "out must be bfloat16"),
    (lambda a: dict(lse=torch.zeros(3, 3, device=DEV)), ValueError, "lse must be float32"),
])
def test_attention_refuses_bad_tensors(over, error, match):
    x, c = torch.zeros(3, 8, 64, dtype=BF, device=DEV), torch.zeros(4, 8, 2, 64, dtype=BF, device=DEV)
    good = dict(q=x[:, :4], k_new=x[:, 4:6], v_new=x[:, 6:], k_cache=c, v_cache=c.clone(), cu_seqlens=_i([0, 1, 3]),
                context_lens=_i([9, 0]), block_table=_i([[1, 2], [3, 0]]), max_new_tokens=2, tree_mask=_i([[1], [1], [3]]))
    _refused(ssd.kv_tree_attention, good, over, error, match)


@pytest.mark.parametrize("over,error,match", [
    (lambda a: dict(k_new=a["k_new"][0]), ValueError, "k_new must be"),
    (lambda a: dict(v_new=a["v_new"].float()), ValueError, "v_new must be bfloat16"),
    (lambda a: dict(slots=a["slots"][:2]), ValueError, "slots must have an entry for each"),
    (lambda a: dict(slots=a["slots"].long()), ValueError, "slots must be int32"),
    (lambda a: dict(cu_seqlens=None), ValueError, "cu_seqlens is required"),
    (lambda a: dict(cu_seqlens=_i([])), ValueError, "cu_seqlens must have an entry more"),
    (lambda a: dict(path=a["path"][:, :0].contiguous()), ValueError, "path must have a column"),
    (lambda a: dict(path=a["path"][:1]), ValueError, "path must be int32"),
    (lambda a: dict(path_lens=None), ValueError, "path_lens is required"),
    (lambda a: dict(context_lens=_i([1])), ValueError, "context_lens must be int32"),
    (lambda a: dict(context_out=_i([1, 2, 3])), ValueError, "context_out must be int32"),
    (lambda a: dict(v_cache=a["v_cache"][:3]), ValueError, "k_cache and v_cache must be"),
])
def test_commit_refuses_bad_tensors(over, error, match):
    x, c = torch.zeros(3, 4, 64, dtype=BF, device=DEV), torch.zeros(4, 8, 2, 64, dtype=BF, device=DEV)
    good = dict(k_new=x[:, :2], v_new=x[:, 2:], k_cache=c, v_cache=c.clone(), slots=_i([1, 2, 3, -1]), cu_seqlens=_i([0, 1, 3]),
                context_lens=_i([9, 0]), path=_i([[0], [1]]), path_lens=_i([1, 1]))
    _refused(ssd.kv_commit_tokens, good, over, error, match)


# ----------------------------------------------------------------- together --

def test_hybrid_tree_decode_example():
    """The four calls beside ssm_decode_update on drafted trees give the tokens that single-token steps give, in fewer
    steps."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_tree_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_tree_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    same, n, plain_steps, steps = example.main()
    assert same and n >= 12 and steps < plain_steps


def test_calls_replay_as_a_graph():
    """A decode step's four calls captured once: replays with new lengths, tokens and tables in the same buffers give
    the bits of eager calls."""
    b, S, H, G, D, n = 16, 3, 4, 2, 128, 2
    g = torch.Generator(device=DEV).manual_seed(3)
    T = S * n
    ctx, new = _i([37, 0, 90]), _i([n] * S)
    kc = torch.randn(40, b, G, D, generator=g, device=DEV).to(BF)
    vc = torch.randn(40, b, G, D, generator=g, device=DEV).to(BF)
    table = _i(np.zeros((S, 12)))
    ring, state = _i(np.random.default_rng(0).permutation(np.arange(1, 40))), _i([5, 39])
    qkv = torch.randn(T, (H + 2 * G) * D, generator=g, device=DEV).to(BF)
    cs = torch.randn(256, D, generator=g, device=DEV)
    zero = _i([0] * S)
    keep = {}

    def step():
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, G * D, G * D], 1))
        m = ssd.kv_block_tables(ctx, new, zero, table, ring, state, b, 40, T)
        q, k = ssd.kv_qk_norm_rope(q, k, m["positions"], cs)
        o, lse = ssd.kv_tree_attention(q, k, v, kc, vc, m["cu_seqlens"], ctx, table, n, return_lse=True)
        c = ssd.kv_commit_tokens(k, v, kc, vc, m["slots"], m["cu_seqlens"], ctx)
        keep.update(m=m, o=o, lse=lse, c=c)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = dict(keep)
    ctx.copy_(_i([80, 3, 17]))
    qkv.normal_(generator=g)
    before = kc.clone(), vc.clone(), table.clone()
    graph.replay()
    torch.cuda.synchronize()
    after = kc.clone(), vc.clone(), table.clone()
    for t, old in zip((kc, vc, table), before):
        t.copy_(old)
    step()
    torch.cuda.synchronize()
    for key in keep["m"]:
        assert torch.equal(keep["m"][key], captured["m"][key]), key
    assert torch.equal(keep["o"], captured["o"]) and torch.equal(keep["lse"], captured["lse"])
    assert torch.equal(keep["c"], captured["c"])
    for t, got in zip((kc, vc, table), after):
        assert torch.equal(t, got)
