"""kv_tree_attention_fp8 where a few keys have most of the weight: what is left counts in full.

One cached key has the share p of a row's weight and a value of nothing, so that the output is the mean of all the others'
values times 1 - p.  All values are positive (0.5 to 1.5): the output is the sum of w |v|, and errors of the weights, each
relative to its own, are errors relative to the output, however many keys there are.  Counted up, relative to the output:

* weights rounded to 16-bit floats, at least as fine as fp16's: 2^-11 of themselves, or 2^-36 of the row's largest, that is
  N 2^-36 p 1.5 in all against an output of (1 - p) 0.5 at least; new tokens' weights to bf16, one part: 2^-8 of their share
* scores: queries have 3 significant bits (one e4m3 part, nothing is lost), so D products and sums in fp32 as on a 16-bit cache,
  (D + 4) 2^-24 of sum |q||k|, in the weight and in the sum of weights; the exponential 2^-21
* sums in fp32, no chain of them longer than N / 32 + 64: (N / 32 + 64) 2^-24, in both sums
* the output's rounding, 2^-8."""
import math

import numpy as np
import pytest
import torch

import selective_state_space_mamba2_gb300 as ssd
from tests import kv8_forms as F8
from tests.test_kv_gpu import _err, _i

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ssd.build()
    torch.cuda.init()


def _case(H, D, n, N, share, at, b, spread, seed, dtype=BF):
    """One request of n new tokens, H query heads to a key head, N cached keys; the dominating key at position `at`."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = (1 + 0.25 * torch.randint(0, 4, (n, H, D), generator=g, device=DEV)) * (2.0 ** torch.randint(-1, 1, (n, H, D), generator=g, device=DEV))
    q *= torch.randint(0, 2, (n, H, D), generator=g, device=DEV) * 2 - 1
    q[:, :, 0] = 1.5
    scale = spread / (1.2 * D ** 0.5)  # q k scale has a deviation of about `spread`
    k = torch.randn(N + n, 1, D, generator=g, device=DEV, dtype=torch.float64)
    k[:, :, 0] = 0  # the first entry is the dominating key's
    v = 0.5 + torch.rand(N + n, 1, D, generator=g, device=DEV, dtype=torch.float64)
    blocks = -(-N // b)
    table = np.random.default_rng(seed).permutation(blocks)[None]
    ks = torch.full((blocks, 1), 2.0 ** -6, device=DEV)
    vs = torch.full((blocks, 1), 2.0 ** -8, device=DEV)
    # what the others come to, and the score that has `share` beside it
    s = (torch.einsum("nhd,kd->nhk", q.double(), k[:, 0]) * scale)
    top = float(torch.logsumexp(s, -1).mean()) + math.log(share / (1 - share))
    page = int(table[0, at // b])
    ks[page] = max(top / (scale * 1.5 * 96), 2.0 ** -6)  # its entry is 96 of its block's scale, or what comes near
    entry = top / (scale * 1.5)
    k[at], v[at] = 0, 0
    k[at, 0, 0] = entry
    kc = torch.zeros(blocks * b, 1, D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros(blocks * b, 1, D, dtype=torch.uint8, device=DEV)
    pages = torch.from_numpy(table[0]).to(DEV)
    rows = (pages[:, None] * b + torch.arange(b, device=DEV)).reshape(-1)[:N]
    kc[rows] = (k[:N] / ks[rows // b, 0].double()[:, None, None]).clamp(-448, 448).to(F8.E4M3).view(torch.uint8)
    vc[rows] = (v[:N] / vs[rows // b, 0].double()[:, None, None]).to(F8.E4M3).view(torch.uint8)
    return dict(q=q.to(dtype), k=k[N:].to(dtype), v=v[N:].to(dtype), kc=kc.view(blocks, b, 1, D).view(F8.E4M3), vc=vc.view(blocks, b, 1, D).view(F8.E4M3),
                ks=ks, vs=vs, table=table, N=N, n=n, scale=scale, rows=rows)


def _want(c):
    """64-bit output, log of the sum of weights, largest weight and largest scale sum |q||k| of each row."""
    N, n = c["N"], c["n"]
    D = c["q"].shape[2]

    def full(codes, scale, new):
        x = codes.view(-1, D).double()[c["rows"]] * scale[c["rows"] // codes.shape[1], 0].double()[:, None]
        return torch.cat([x, new[:, 0].double()])
    k, v = full(c["kc"], c["ks"], c["k"]), full(c["vc"], c["vs"], c["v"])
    s = torch.einsum("nhd,kd->nhk", c["q"].double(), k) * c["scale"]
    sees = torch.arange(N + n, device=DEV)[None, :] <= N + torch.arange(n, device=DEV)[:, None]
    s = torch.where(sees[:, None], s, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[..., None])
    big = (torch.einsum("nhd,kd->nhk", c["q"].double().abs(), k.abs()) * c["scale"]).amax(-1)
    return w @ v, lse, w[..., :N].amax(-1), w[..., N:].sum(-1), big


def _run(c, copies):
    """Of `copies` requests that are all the same and share their blocks."""
    err = _err()
    n = c["n"]
    q, k, v = (c[x].repeat(copies, 1, 1) for x in "qkv")
    out, lse = ssd.kv_tree_attention_fp8(q, k, v, c["kc"], c["vc"], c["ks"], c["vs"], _i(np.arange(copies + 1) * n), _i([c["N"]] * copies),
                                         _i(np.repeat(c["table"], copies, 0)), n, scale=c["scale"], return_lse=True, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out.double().unflatten(0, (copies, n)), lse.double().unflatten(0, (copies, n))


def _check(c, copies=1):
    want, wlse, top, new, big = _want(c)
    out, lse = _run(c, copies)
    N, D = c["N"], c["q"].shape[2]
    u = 2.0 ** -24
    score = 2 * (D + 4) * u * big + 2.0 ** -21 + 2 * (N / 32 + 64) * u
    left = want.amin(-1)  # of a row's outputs, each at least half of the others' weight
    rel = 2.0 ** -11 + score + 2.0 ** -8 * 1.5 * new / left + N * 2.0 ** -36 * top * 1.5 / left + 2.0 ** -8
    err = (out / want - 1).abs()
    assert (err <= 1.01 * rel[..., None]).all(), (float(err.max()), float(rel.max()))
    assert ((lse - wlse).abs() <= score + 4 * u * wlse.abs()).all()
    return float(err.max())


KINDS = [(4, 1), (3, 5), (8, 4), (17, 1), (8, 30), (4, 70)]  # query heads, new tokens: row tiles of 16, 32, 128 and two of 128


@pytest.mark.parametrize("share", [0.5, 0.9, 0.97, 0.99, 0.999])
@pytest.mark.parametrize("H,n", KINDS)
@pytest.mark.parametrize("D,N,at,b", [(128, 8192, 0, 64), (64, 16384, 5000, 16), (128, 2048, 2047, 128), (64, 8191, 0, 8)])
def test_one_key_with_most_of_the_weight(H, n, D, N, share, at, b):
    _check(_case(H, D, n, N, share, at, b, 1.0, seed=N + H))


@pytest.mark.parametrize("H,n", KINDS)
def test_one_key_beside_equal_ones(H, n):
    """Weights that are all the same are all off in the same direction."""
    for share in (0.9, 0.99, 0.999):
        _check(_case(H, 128, n, 16384, share, 3, 64, 2.0 ** -20, seed=7))


@pytest.mark.parametrize("share", [0.5, 0.9, 0.99, 0.999])
@pytest.mark.parametrize("H,n", [(4, 1), (8, 4), (8, 30)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_key_in_a_batch(H, n, D, share):
    """So many requests that a CTA has all of one's keys, or of several requests'."""
    _check(_case(H, D, n, 8192, share, 0, 64, 1.0, seed=3), copies=700 if n < 5 else 200)
    _check(_case(H, D, n, 3000, share, 2000, 16, 2.0 ** -20, seed=4), copies=700 if n < 5 else 200)


@pytest.mark.parametrize("H,n", [(8, 30), (4, 70), (4, 1), (8, 4)])
@pytest.mark.parametrize("share", [0.999, 0.9999])
def test_one_key_beside_very_many(H, n, share):
    """Weights as far below the largest as long caches have them."""
    _check(_case(H, 64, n, 65536, share, 100, 64, 2.0 ** -20, seed=5), copies=60 if n > 5 else 400)
    _check(_case(H, 128, n, 65536, share, 65535, 16, 0.5, seed=6), copies=1)
