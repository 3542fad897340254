"""GPU: calls on two streams at once, each with its own workspace, give what they give one after the other."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
from test_gpu_score_mod import BF, F8, I4, make_pool, randn, slopes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, F8, I4])
def test_decode_and_prefill_on_two_streams(fmt):
    hq, hkv, d, n, n_q = 16, 4, 128, 40, 200
    lens = [(211 * i * i + 17 * i) % 3000 for i in range(n)]
    pool = make_pool(fmt, hkv, d, 1, 1, 96, n, 47 * n)
    pt = torch.randperm(47 * n, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(n, 47).cuda()
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    k, v = randn(1, n, 3000, hkv, d).cuda(), randn(2, n, 3000, hkv, d).cuda()
    zero = torch.zeros(n, dtype=torch.int64, device="cuda")
    hs.kv_pool_append(pool, 1, k, v, zero, page_table=pt)
    hs.kv_pool_append(pool, 0, k, v, zero, seq_ids=ids)
    q, kn, vn = randn(3, n, 2, hq, d).cuda(), randn(4, n, 2, hkv, d).cuda(), randn(5, n, 2, hkv, d).cuda()
    qp = randn(6, 3, n_q, hq, d).cuda()
    ctx, sl = torch.tensor(lens, device="cuda"), slopes(hq).cuda()
    i = torch.arange(1000, 1000 + n_q, device="cuda")
    begin = torch.where(i < 1100, 0, 1100).expand(3, n_q).contiguous()
    start = torch.full((3,), 1000, device="cuda")
    rope = hs.RopeDesc([0.01 * (f + 1) for f in range(32)], [f % 2 for f in range(32)], 2)
    pos = torch.stack([torch.arange(3 * n_q), torch.arange(3 * n_q) // 7]).cuda()

    def calls(ws, wp):
        few = hs.hybrid_decode_mod_fwd(pool, 1, q[:5].contiguous(), kn[:5].contiguous(), vn[:5].contiguous(),
                                       ctx[:5].contiguous(), 3000, hs.ScoreMod(10.0, sl), ws, page_table=pt[:5].contiguous())
        many = hs.hybrid_decode_fwd(pool, 1, q, kn, vn, ctx, 3000, ws, page_table=pt)
        ring = hs.hybrid_decode_fwd(pool, 0, q, kn, vn, torch.full_like(ctx, 3000), 3000, ws, seq_ids=ids)
        pre = hs.full_prefill_mod_fwd(pool, 1, qp, pt[:3].contiguous(), hs.ScoreMod(20.0, key_begin=begin), wp,
                                      start_pos=start)
        turned = hs.rope_fwd(rope, qp, qp[:, :, :4].contiguous(), pos)
        return few, many, ring, pre, *turned

    size = hs.hybrid_decode_workspace_size(pool, n, 2, hq, 3000)
    room = lambda b: torch.empty(b, dtype=torch.uint8, device="cuda")
    wp_size = hs.prefill_mod_workspace_size(pool, 3, n_q)
    want = [x.clone() for x in calls(room(size), room(wp_size))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [(room(size), room(wp_size)) for _ in streams]
    got = [[], []]
    for _ in range(6):
        for s, w, g in zip(streams, work, got):
            with torch.cuda.stream(s):
                g.append(calls(*w))
    torch.cuda.synchronize()
    assert hs.hswa_pool_check_error(pool) == 0
    for g in got:
        for outs in g:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
