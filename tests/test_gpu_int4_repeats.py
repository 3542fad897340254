"""GPU: decode over 4-bit pools gives the same bits every time, whatever order its block copies land in and
whichever CTA takes an item."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref
from test_gpu_int4 import make_pool, rows

pytestmark = pytest.mark.gpu


def entries(seed, n, hkv, d):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, hkv, d, generator=g, device="cuda").to(torch.bfloat16)


# lengths, new tokens, query and KV heads, head dim, window (0: pages)
@pytest.mark.parametrize("lens,n_qt,hq,hkv,d,W", [
    ([30011], 1, 8, 1, 128, 0),                              # one long context, 8 rows, four readers
    ([9000, 20011, 64, 0, 3001], 4, 32, 8, 128, 0),          # 16 rows
    ([7001 * (i % 4) + 61 * i for i in range(40)], 4, 16, 2, 128, 0),  # 32 rows, pairs of warps, its own work list
    ([5003 * (i % 3) + 77 * i for i in range(36)], 1, 6, 2, 64, 0),
    ([60 + 9 * i for i in range(48)], 1, 64, 8, 128, 0),     # whole contexts to single warps
    ([50 * i for i in range(100)], 4, 64, 8, 128, 128),      # rings to pairs of warps
    ([50 * i for i in range(100)], 2, 32, 8, 64, 500)])
def test_decode_gives_the_same_bits_every_time(lens, n_qt, hq, hkv, d, W):
    n = len(lens)
    used = [-(-length // 64) for length in lens]
    total = max(1, sum(used)) * 3
    # pages scattered over three times the memory they need
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    pt = torch.zeros(n, max(max(used), 1), dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        pt[b, :u] = perm[at: at + u]
        at += u
    pt, ids = pt.cuda(), torch.arange(n, dtype=torch.int32, device="cuda")
    pool = make_pool(hkv, d, 1 if W else 0, 0 if W else 1, W or 1, n, 0 if W else total)
    held = []
    for b, length in enumerate(lens):
        lo = max(0, length - W) if W else 0
        k, v = entries(2 * b, length - lo, hkv, d), entries(2 * b + 1, length - lo, hkv, d)
        held.append((k, v, lo))
        if length > lo:
            hs.kv_pool_append(pool, 0, k[None], v[None], torch.tensor([lo], device="cuda"),
                              seq_ids=ids[b:b + 1] if W else None, page_table=None if W else pt[b:b + 1].contiguous())
    q, kn, vn = (rows(s, n * n_qt, h, d).view(n, n_qt, h, d).cuda() for s, h in ((7, hq), (8, hkv), (9, hkv)))
    ctx = torch.tensor(lens, device="cuda")
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_qt, hq, max(lens)), dtype=torch.uint8, device="cuda")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for rep in range(12):
        if rep % 3 == 0:
            flush.fill_(rep)  # entries come from memory
        o = hs.hybrid_decode_fwd(pool, 0, q, kn, vn, ctx, max(lens), ws, seq_ids=ids if W else None,
                                 page_table=None if W else pt)
        first = o.clone() if first is None else first
        assert torch.equal(o, first), rep
    assert hs.hswa_pool_check_error(pool) == 0
    for b in {0, n // 2, n - 1}:
        k, v, lo = held[b]
        kk, vv = torch.cat([k, kn[b]]).cpu(), torch.cat([v, vn[b]]).cpu()
        a, e = ref.ranges(n_qt, lens[b], lens[b] + n_qt, W)
        x = ref.int4_values(vv)
        ref.check(first[b], ref.attention(q[b].cpu(), ref.int4_values(kk), x, torch.clamp(a, min=0), e, lo,
                                          weight_eps=ref.F16, v_range=x.amax(-1) - x.amin(-1)), f"seq {b}")
