"""kv_commit_tokens_fp8 where a CTA has many blocks to write, empty places among them: codes and scales exactly, call after call."""
import numpy as np
import pytest
import torch

import selective_state_space_mamba2_gb300 as ssd
from tests import kv8_forms as F8
from tests.test_kv_fp8_gpu import _check_commit, _commit, _commit_case, _err

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ssd.build()
    torch.cuda.init()


def _batch(S, H, b, dtype, path, seed):
    """Requests of 0 to 6 tokens whose magnitudes differ from request to request."""
    rng = np.random.default_rng(seed)
    c = _commit_case(dtype, H, 128, b, rng.integers(0, 7, S).tolist(), rng.integers(0, 4 * b, S).tolist(), seed=seed, path=path)
    for r in range(S):
        c["kv"][c["cu"][r]:c["cu"][r + 1]] *= 2.0 ** int(rng.integers(-12, 13))
    return c


def _repeats(c, times=8):
    """The same call over again from the same cache gives the same bytes."""
    first = None
    start = [a.copy() for a in c["codes"]], [a.copy() for a in c["scales"]]
    for _ in range(times):
        c["codes"], c["scales"] = [a.copy() for a in start[0]], [a.copy() for a in start[1]]
        _, dev = _commit(c, _err())
        bits = [t.view(torch.uint8) if t.dtype == F8.E4M3 else t.view(torch.int32) for t in dev]
        first = first or bits
        assert all(torch.equal(x, y) for x, y in zip(bits, first))


@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("S,H,b,dtype", [(3000, 1, 16, BF), (2000, 2, 64, BF), (1500, 2, 16, F32), (1000, 1, 64, F32), (2500, 3, 16, BF)])
def test_commit_many_short_requests(S, H, b, dtype, path):
    """Several blocks a CTA, teams of more than a warp: a place that is empty does not bring two blocks' maxima together."""
    c = _batch(S, H, b, dtype, path, seed=S + H + b)
    _repeats(c)
    _check_commit(c)


@pytest.mark.parametrize("H,b", [(4, 64), (2, 32)])
def test_commit_long_prompts_of_several_blocks_a_cta(H, b):
    new = [5000, 1, 0, 9001, 64, 7000, 3, 11000]
    c = _commit_case(BF, H, 128, b, new, [0, 5, 3, 77, 64, 63, 500, 31], seed=b, loud=(3, 6))
    _repeats(c, 4)
    _check_commit(c)


@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("b,dtype", [(16, BF), (4, F32), (1, BF)])
@pytest.mark.parametrize("pad", [1, 17, 200])
def test_commit_behind_rows_of_no_request(b, dtype, path, pad):
    """cu_seqlens that does not begin with 0: the rows before its first entry are no request's, and every block is written once."""
    c = _commit_case(dtype, 2, 64, b, [5, 3, 0, 9], [3, 2 * b + 1, 7, b - 1], seed=pad + b, path=path, loud=(0, 3))
    c["kv"] = torch.cat([torch.full((pad, c["kv"].shape[1]), float("nan"), dtype=dtype), c["kv"], torch.full((2, c["kv"].shape[1]), float("nan"), dtype=dtype)])
    c["cu"] = c["cu"] + np.int32(pad)
    _repeats(c)
    _check_commit(c)
