"""kv_tree_attention_fp8 on batches with requests without tokens behind the last one and packed rows that no request has: the
requests' own rows within the bounds of their arithmetic, entry by entry, as without the padding."""
import numpy as np
import pytest
import torch

import selective_state_space_mamba2_gb300 as ssd
from tests import kv8_forms as F8
from tests.test_kv_fp8_gpu import BF, F32, _attn, _err, _run, _tensor_cores

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ssd.build()
    torch.cuda.init()


@pytest.mark.parametrize("dtype,H,Hkv,D,b,new,ctx,hint", [
    (BF, 8, 2, 128, 16, [3, 1, 0, 2], [300, 77, 40, 0], 3), (BF, 8, 2, 64, 16, [3, 70, 0, 2], [5000, 77, 40, 0], 70),
    (BF, 8, 1, 128, 32, [3, 40, 0, 64], [300, 3000, 40, 0], 64), (BF, 4, 1, 64, 64, [1, 1, 0, 1], [9000, 1, 5, 400], 1),
    (F32, 4, 2, 64, 16, [3, 1, 0, 2], [300, 2000, 40, 0], 3), (BF, 4, 2, 96, 24, [3, 30, 0, 2], [300, 77, 40, 0], 30)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("front", [0, 5])
def test_attention_padded_batches_entry_by_entry(dtype, H, Hkv, D, b, new, ctx, hint, tree, front):
    c = _attn(dtype, H, Hkv, D, b, new, ctx, tree, seed=9 + front, max_new=hint)
    want, wlse, tol, ltol, keys = F8.attention_bound(c, F8.values(c["kcodes"], c["ks"]), F8.values(c["vcodes"], c["vs"]), _tensor_cores(c))
    T, more = sum(new), 9
    p = dict(c, cu=np.concatenate([c["cu"] + front, [T + front] * 3]).astype(np.int32), ctx=list(c["ctx"]) + [50, 0, 7],
             table=np.concatenate([c["table"], c["table"][:3]]))
    for x in "qkv":
        nan = torch.full((front + more, *c[x].shape[1:]), float("nan"), dtype=dtype, device=DEV)
        p[x] = torch.cat([nan[:front], c[x], nan[front:]])
    if tree:
        ones = np.full((front + more, c["mask"].shape[1]), 2 ** 32 - 1, np.uint32)
        p["mask"] = np.concatenate([ones[:front], c["mask"], ones[front:]])
    out = torch.full((front + T + more, H, D), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((front + T + more, H), 7.0, device=DEV)
    err = _err()
    _run(p, err, out=out, lse=lse)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for t in (out, lse):
        assert (t[:front] == 7).all() and (t[front + T:] == 7).all()
    got, gl = out[front:front + T].double().cpu(), lse[front:front + T].double().cpu()
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
    assert (got[keys == 0] == 0).all() and torch.isneginf(gl[keys == 0]).all()
    some = keys > 0
    assert ((gl - wlse).abs() <= ltol)[some].all()
