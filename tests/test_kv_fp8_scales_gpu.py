"""kv_tree_attention_fp8 over values' scales as far apart as one request may have them, 2^96 with the 1 of its new tokens among
them: a key counts in the sum of weights whatever its value's scale, in an item and in one that is cut over many CTAs."""
import numpy as np
import pytest
import torch

import selective_state_space_mamba2_gb300 as ssd
from tests.test_kv_fp8_gpu import BF, F32, _attn, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ssd.build()
    torch.cuda.init()


LAYOUTS = [  # type, query heads, key heads, head size, block size, new, cached: row tiles of 16, 32, 128 rows, two of them, CUDA cores
    (BF, 4, 1, 128, 8, [1, 3, 2], [40, 333, 1000]), (BF, 8, 2, 64, 64, [1, 4], [700, 5000]), (BF, 8, 1, 128, 16, [4, 3], [1000, 65]),
    (BF, 32, 1, 64, 128, [1], [20011]), (BF, 8, 1, 128, 8, [30, 5], [900, 100]), (BF, 4, 1, 64, 64, [70, 9, 33], [300, 3000, 0]),
    (BF, 8, 2, 128, 32, [40, 17], [5000, 129]), (F32, 4, 2, 64, 16, [3, 1], [700, 40]), (BF, 4, 1, 96, 16, [2, 5], [300, 90]),
]


def _exponents(what, lo, hi, rng, blocks):
    """Of the scales of a request's blocks, in order."""
    j = np.arange(blocks)
    return {"in turn": np.where(j % 2 == 0, hi, lo), "one large first": np.where(j == 0, hi, lo), "large last": np.where(j == blocks - 1, hi, lo),
            "one small": np.where(j == blocks // 2, lo, hi), "any": rng.integers(lo, hi + 1, blocks), "small first": np.minimum(lo + 20 * j, hi)}[what]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("what", ["in turn", "one large first", "large last", "one small", "any", "small first"])
@pytest.mark.parametrize("lo,hi", [(-64, 32), (0, 96), (-30, 66)])
@pytest.mark.parametrize("queries", ["zero", "usual", "far"])
def test_attention_value_scales_far_apart_in_a_request(layout, what, lo, hi, queries):
    dtype, H, Hkv, D, b, new, ctx = layout
    c = _attn(dtype, H, Hkv, D, b, new, ctx, False, seed=len(what) + D + b, qk_gain=8.0 if queries == "far" else 1.0)
    rng = np.random.default_rng(b)
    for r, n in enumerate(ctx):
        blocks = -(-n // b)
        if blocks:
            c["vs"][c["table"][r, :blocks]] = 2.0 ** _exponents(what, lo, hi, rng, blocks).astype(np.float64)[:, None]
    if queries == "zero":
        c["q"][:] = 0
    _check(c)
