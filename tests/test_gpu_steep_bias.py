"""GPU: a distance bias so steep that the nearest key a query sees takes all the weight, however far away it is."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
from test_gpu_score_mod import BF, F8, I4, held, make_pool, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, F8, I4])
@pytest.mark.parametrize("slope", [50.0, 1e20, 1e31])
@pytest.mark.parametrize("n", [1, 40])
def test_decode_sees_only_far_keys(fmt, slope, n):
    L, n_q, hq, hkv, d, last = 300, 2, 32, 8, 64, 10
    pool = make_pool(fmt, hkv, d, 0, 1, 64, 1, 5)
    pt = torch.arange(5, dtype=torch.int32).view(1, 5).cuda()
    k, v, q = randn(1, L, hkv, d), randn(2, L, hkv, d), randn(3, n, n_q, hq, d)
    hs.kv_pool_append(pool, 0, k[None].cuda(), v[None].cuda(), torch.tensor([0]).cuda(), page_table=pt)
    new = torch.zeros(n, n_q, hkv, d, dtype=torch.bfloat16).cuda()
    mod = hs.ScoreMod(dist_slope=torch.full((hq,), slope).cuda(), key_end=torch.full((n, n_q), last).cuda())
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_q, hq, L), dtype=torch.uint8, device="cuda")
    o = hs.hybrid_decode_mod_fwd(pool, 0, q.cuda(), new, new, torch.full((n,), L).cuda(), L, mod, ws,
                                 page_table=pt.expand(n, 5).contiguous())
    assert hs.hswa_pool_check_error(pool) == 0
    # all other weights are below e^-40: the nearest row's value, rounded to bf16 once, and its code's weight to f16
    hv = held(fmt, v, False)[last - 1].repeat_interleave(hq // hkv, 0)
    size = hv.abs() + (hv.amax(-1) - hv.amin(-1))[:, None]
    assert ((o.cpu().double() - hv).abs() <= 2.0 ** -8 * hv.abs() + (2.0 ** -11 + 1e-4) * size).all()
