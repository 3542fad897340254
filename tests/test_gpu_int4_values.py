"""GPU: decode over 4-bit pools with V rows of very different sizes: rows far larger than the others along a long
context."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref
from test_gpu_int4 import make_pool, rows, table

pytestmark = pytest.mark.gpu


def exact(q, k, v, lo, hi, pos0=0):
    x = ref.int4_values(v)
    return ref.attention(q, ref.int4_values(k), x, torch.clamp(lo, min=0), hi, pos0, weight_eps=ref.F16,
                         v_range=x.amax(-1) - x.amin(-1))


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (32, 8, 64), (16, 4, 128)])
@pytest.mark.parametrize("size", [1e3, 3e4])
@pytest.mark.parametrize("first", [0, 1])
def test_large_v_rows_along_a_long_context(hq, hkv, d, size, first):
    # splits of 8192 keys; the first row of every page (or the second) is `size` times the others. In two of three KV
    # heads those rows carry no weight (scores of -40), so they add nothing to the tolerance either, which scales
    # with weights x values and weights x ranges.
    n, n_qt, L = 320 // hkv, 2, 32768
    pool = make_pool(hkv, d, 0, 1, 1, 1, L // 64)
    pt = table(5, 1, L // 64, L // 64)
    k, v, q = rows(1, L + n_qt, hkv, d), rows(2, L + n_qt, hkv, d), rows(3, n_qt, hq, d)
    at = torch.arange(first, L, 64)
    v[at] = (v[at].float() * size).to(torch.bfloat16)
    for g in range(hkv):
        if g % 3 != 2:  # one query for all rows of the group, of which these keys have score -40
            group = hq // hkv
            q[:, g * group: (g + 1) * group] = q[0, g * group].clone()
            u = q[0, g * group].float()
            k[at, g] = (-40.0 * d ** 0.5 * u / (u @ u)).to(torch.bfloat16)
    hs.kv_pool_append(pool, 0, k[None, :L].cuda(), v[None, :L].cuda(), torch.tensor([0]).cuda(), page_table=pt.cuda())
    lens = [L] + [0] * (n - 1)
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_qt, hq, L), dtype=torch.uint8, device="cuda")
    args = [x[None].expand(n, *x.shape).contiguous().cuda() for x in (q, k[L:], v[L:])]
    o = hs.hybrid_decode_fwd(pool, 0, *args, torch.tensor(lens).cuda(), L, ws,
                             page_table=pt.expand(n, L // 64).contiguous().cuda())
    assert hs.hswa_pool_check_error(pool) == 0
    lo, hi = ref.ranges(n_qt, L, L + n_qt)
    ref.check(o[0], exact(q, k, v, lo, hi), "long context")
