"""Attention over the cache where segments are cut into parts, with and without page
lists, against the fp64 definition with bounds that a lost or misplaced page cannot
meet (test_cache_exact.py shows that they reject it)."""
import numpy as np
import pytest
import torch

from cache_common import values
from cache_exact import CASES, SCALE, build, tolerances
from gpu_common import need_gpu
from oracle import cache as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", list(CASES))
def test_exact_sums(name):
    fm = need_gpu()
    B, H, Hk, N, d, lens, most, kind, Hm = CASES[name]
    q, k8, kscale, v8, vscale, table, lens, vectors = build(name)
    cache = fm.KVCache(k8.cuda(), v8.cuda(), kscale.cuda(), vscale.cuda())
    mask = None if kind is None else fm.DeviceMask(*[None if t is None else t.cuda() for t in vectors], True)
    ws = fm.alloc_cache_workspace(B, H, Hk, N, d, most)
    args = (q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), ws)
    o, lse = fm.flashmask_fwd_cache(*args, mask=mask, scale=SCALE)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    lts, lte, uts, ute = (None if t is None else t.numpy() for t in vectors)
    ref_o, ref_l, pv, _, _ = C.attend(q.double().numpy(), values(k8), kscale.numpy(), values(v8), vscale.numpy(),
                                      table.numpy(), lens, None, SCALE, True, lts, lte, uts, ute)
    tol_o, tol_l = tolerances(ref_o, ref_l, pv)
    none = np.isneginf(ref_l)
    got_o, got_l = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got_l), none) and (got_o[none] == 0).all()
    err_o, err_l = np.abs(got_o - ref_o) - tol_o, np.abs(got_l[~none] - ref_l[~none]) - tol_l[~none]
    assert err_o.max() <= 0 and err_l.max() <= 0, (err_o.max(), err_l.max())
    # the workspace's counters are as they were: the same bits again
    o2, lse2 = fm.flashmask_fwd_cache(*args, mask=mask, scale=SCALE)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
