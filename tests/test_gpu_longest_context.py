"""GPU: decode at the longest context length that the calls accept, with one page of entries behind almost all of the
page table. The keys of the last page have scores 40 above the others', which sum to 2^31 e^-40 < 1e-8 of the weights."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref
from test_gpu_score_mod import BF, I4, held, make_pool, randn

pytestmark = pytest.mark.gpu
LONGEST = 2 ** 31 - 1 - 4096


@pytest.mark.parametrize("fmt", [I4, BF])
@pytest.mark.parametrize("L", [LONGEST, LONGEST - 4096, LONGEST - 12345])
def test_the_last_split_of_the_longest_contexts(fmt, L):
    hq, hkv, d = 2, 1, 64
    pool = make_pool(fmt, hkv, d, 0, 1, 64, 1, 2)
    last = (L - 1) // 64
    pt = torch.zeros(1, last + 1, dtype=torch.int32, device="cuda")
    pt[0, last] = 1
    n = L - 64 * last
    k, v = torch.zeros(64, hkv, d, dtype=torch.bfloat16), randn(1, 64 + n, hkv, d)
    near = torch.full((n, hkv, d), 5.0, dtype=torch.bfloat16)  # q k / sqrt(d) = 40 for a q of ones
    hs.kv_pool_append(pool, 0, k[None].cuda(), v[None, :64].contiguous().cuda(), torch.tensor([0]).cuda(), page_table=pt)
    two = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    hs.kv_pool_append(pool, 0, near[None].cuda(), v[None, 64:].contiguous().cuda(), torch.tensor([64]).cuda(), page_table=two)
    q, new = torch.ones(1, 1, hq, d, dtype=torch.bfloat16).cuda(), torch.zeros(1, 1, hkv, d, dtype=torch.bfloat16).cuda()
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 1, 1, hq, L), dtype=torch.uint8, device="cuda")
    o = hs.hybrid_decode_mod_fwd(pool, 0, q, new, new, torch.tensor([L]).cuda(), L, hs.ScoreMod(), ws, page_table=pt)
    assert hs.hswa_pool_check_error(pool) == 0
    hv = held(fmt, v[64:], False)
    r = ref.attention(q[0].cpu(), near.double(), hv, torch.zeros(1, dtype=torch.int64), torch.full((1,), n),
                      weight_eps=ref.F16 if fmt == I4 else ref.BF16,
                      v_range=hv.amax(-1) - hv.amin(-1) if fmt == I4 else None)
    ref.check(o[0], r, f"L={L}")
