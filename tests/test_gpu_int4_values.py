"""GPU: decode over 4-bit pools with V rows of very different sizes: rows far larger than the others along a long
context, and far larger values where only another token of the step sees them."""
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


@pytest.mark.parametrize("n,hq,hkv,d", [(1, 4, 2, 128), (40, 32, 8, 64), (40, 64, 8, 128)])
@pytest.mark.parametrize("large_first", [False, True])
@pytest.mark.parametrize("size", [1e4, 1e12])
def test_ranges_apart_do_not_share_a_scale(n, hq, hkv, d, large_first, size):
    # token 0 and token 1 see different documents; V of token 1's is `size` times larger; token 2 sees nothing
    L, cut, n_qt = 900, 410, 3
    pool = make_pool(hkv, d, 0, 1, 1, 1, 15)
    pt = table(6, 1, 15, 15)
    k, v, q = rows(4, L + n_qt, hkv, d), rows(5, L + n_qt, hkv, d), rows(6, n_qt, hq, d)
    big = torch.arange(L + n_qt) < cut if large_first else torch.arange(L + n_qt) >= cut
    v[big] = (v[big].float() * size).to(torch.bfloat16)
    a, b = (cut, L + n_qt), (0, cut)
    if not large_first:
        a, b = b, a
    begin, end = torch.tensor([a[0], b[0], 7]), torch.tensor([a[1], b[1], 7])
    hs.kv_pool_append(pool, 0, k[None, :L].cuda(), v[None, :L].cuda(), torch.tensor([0]).cuda(), page_table=pt.cuda())
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_qt, hq, L), dtype=torch.uint8, device="cuda")
    args = [x[None].expand(n, *x.shape).contiguous().cuda() for x in (q, k[L:], v[L:], begin, end)]
    o = hs.hybrid_decode_mod_fwd(pool, 0, *args[:3], torch.full((n,), L).cuda(), L,
                                 hs.ScoreMod(key_begin=args[3], key_end=args[4]), ws,
                                 page_table=pt.expand(n, 15).contiguous().cuda())
    assert hs.hswa_pool_check_error(pool) == 0
    lo, hi = ref.ranges(n_qt, L, L + n_qt, key_begin=begin, key_end=end)
    r = exact(q, k, v, lo, hi)
    for s in {0, n - 1}:
        ref.check(o[s], r, f"seq {s}")


@pytest.mark.parametrize("n,hq,hkv,d,W", [(2, 4, 2, 128, 0), (40, 32, 8, 64, 0), (3, 16, 2, 128, 70), (90, 8, 4, 64, 70)])
@pytest.mark.parametrize("size", [1e4, 1e12])
def test_a_large_draft_token_or_a_large_key_that_left_the_window(n, hq, hkv, d, W, size):
    # the last new token is seen by itself alone; in a ring the oldest key is seen by the first token alone
    L, n_qt = 71, 4
    pool = make_pool(hkv, d, 1 if W else 0, 0 if W else 1, W or 1, n, 2)
    pt = torch.tensor([[1, 0]], dtype=torch.int32)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    lo = max(0, L - W) if W else 0
    k, v, q = rows(7, L + n_qt - lo, hkv, d), rows(8, L + n_qt - lo, hkv, d), rows(9, n_qt, hq, d)
    for row in [L + n_qt - 1] + ([L - W + 1] if W else []):
        v[row - lo] = (v[row - lo].float() * size).to(torch.bfloat16)
    for s in range(n if W else 1):
        hs.kv_pool_append(pool, 0, k[None, : L - lo].cuda(), v[None, : L - lo].cuda(), torch.tensor([lo]).cuda(),
                          seq_ids=ids[s:s + 1] if W else None, page_table=None if W else pt.cuda())
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_qt, hq, L), dtype=torch.uint8, device="cuda")
    args = [x[None].expand(n, *x.shape).contiguous().cuda() for x in (q, k[L - lo:], v[L - lo:])]
    o = hs.hybrid_decode_fwd(pool, 0, *args, torch.full((n,), L).cuda(), L, ws, seq_ids=ids if W else None,
                             page_table=None if W else pt.expand(n, 2).contiguous().cuda())
    assert hs.hswa_pool_check_error(pool) == 0
    a, e = ref.ranges(n_qt, L, L + n_qt, W)
    r = exact(q, k, v, a, e, lo)
    for s in {0, n - 1}:
        ref.check(o[s], r, f"seq {s}")
