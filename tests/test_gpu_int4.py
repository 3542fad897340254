"""GPU: pools of 4-bit entries: commit bit for bit, decode over pages and rings, prefill, gather."""
import numpy as np
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref

pytestmark = pytest.mark.gpu


def rows(seed, n, hkv, d, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    mean = torch.randn(hkv, d, generator=g) * 0.5
    return ((torch.randn(n, hkv, d, generator=g) + mean) * spread).to(torch.bfloat16)


def make_pool(hkv, d, n_swa, n_full, W, seqs, pages):
    pool = hs.kv_pool_create(hs.PoolDesc(n_swa_layers=n_swa, n_full_layers=n_full, window=W, n_kv_heads=hkv, head_dim=d,
                                         max_seqs=seqs, pages_per_full_layer=pages, kv_format=hs.HSWA_KV_INT4))
    pool.data.fill_(0xFF)  # what was never written reads as NaN
    return pool


def table(seed, n, per, total):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(total, generator=g)[: n * per].view(n, per).to(torch.int32)


@pytest.mark.parametrize("hkv,d,n_tok,start", [(1, 64, 1, 0), (3, 128, 130, 60), (8, 128, 65, 63), (2, 64, 200, 1)])
def test_commit_to_pages_is_exact(hkv, d, n_tok, start):
    per = (start + n_tok + 63) // 64
    pool = make_pool(hkv, d, 1, 2, 128, 2, 2 * per + 3)
    pt = table(5, 2, per, 2 * per + 3)
    k, v = (torch.stack([rows(s + 10 * b, n_tok, hkv, d) for b in range(2)]) for s in (1, 2))
    # rows that are hard to hold: constant, tiny range, huge, and one with an infinity and a NaN
    k[0, 0, 0] = 1.5
    v[1, n_tok - 1, 0] = torch.tensor([1e-38, 3e-38] * (d // 2)).to(torch.bfloat16)
    k[1, 0, 0, 0], k[1, 0, 0, 1] = 3e38, -3e38
    v[0, 0, hkv - 1, 5] = float("inf")
    if n_tok > 1:
        v[0, 1, 0, 7] = float("nan")
        k[0, 1, 0] *= 1e30
    layer = 2  # the second full layer
    hs.kv_pool_append(pool, layer, k.cuda(), v.cuda(), torch.tensor([start, start]).cuda(), page_table=pt.cuda())
    assert hs.hswa_pool_check_error(pool) == 0
    for kv, x in enumerate((k, v)):
        codes, step, low = ref.int4_rows(x)
        got_c, got_p = ref.int4_blocks(pool.pages[kv, 1], 64, d)
        for b in range(2):
            for t in range(n_tok):
                p = start + t
                page, r = int(pt[b, p // 64]), p % 64
                want = torch.cat([step[b, t], low[b, t]], -1)
                got = got_p[page, :, r].view(torch.bfloat16)
                nan = torch.isnan(want.float())
                assert torch.equal(torch.isnan(got.float()), nan), (kv, b, t)
                assert torch.equal(got.float()[~nan], want.float()[~nan]), (kv, b, t)
                assert torch.equal(got_c[page, :, r], codes[b, t]), (kv, b, t)
    # nothing else was written: every row that no token of the call owns still holds 0xFF bytes
    owned = torch.zeros(2 * per + 3, 64, dtype=torch.bool)
    for b in range(2):
        for p in range(start, start + n_tok):
            owned[int(pt[b, p // 64]), p % 64] = True
    raw_c, raw_p = ref.int4_blocks(pool.pages[0, 1], 64, d)
    assert (raw_c.transpose(1, 2)[~owned] == 15).all() and (raw_p.transpose(1, 2)[~owned] == -1).all()
    assert (pool.pages[:, 0] == 0xFF).all() and (pool.ring == 0xFF).all()


@pytest.mark.parametrize("W,n_tok,start", [(5, 3, 4), (5, 40, 2), (128, 128, 77), (300, 299, 1000), (1, 2, 0)])
def test_commit_to_ring_is_exact(W, n_tok, start):
    hkv, d = 2, 128
    pool = make_pool(hkv, d, 2, 0, W, 3, 0)
    k, v = rows(3, n_tok, hkv, d)[None], rows(4, n_tok, hkv, d)[None]
    hs.kv_pool_append(pool, 1, k.cuda(), v.cuda(), torch.tensor([start]).cuda(),
                      seq_ids=torch.tensor([2], dtype=torch.int32).cuda())
    assert hs.hswa_pool_check_error(pool) == 0
    for kv, x in enumerate((k, v)):
        codes, step, low = ref.int4_rows(x)
        got_c, got_p = ref.int4_blocks(pool.ring[kv, 2, 1], W, d)
        for t in range(max(0, n_tok - W), n_tok):
            slot = (start + t) % W
            assert torch.equal(got_c[:, slot], codes[0, t])
            assert torch.equal(got_p[:, slot].view(torch.bfloat16), torch.cat([step[0, t], low[0, t]], -1))
    assert (pool.ring[:, :2] == 0xFF).all() and (pool.ring[:, 2, 0] == 0xFF).all()


def test_gather_ring_moves_rows_as_stored():
    W, hkv, d = 9, 2, 64
    pool = make_pool(hkv, d, 1, 0, W, 3, 0)
    pool.data.copy_(torch.randint(0, 256, pool.data.shape, dtype=torch.uint8, device="cuda"))
    before = pool.ring.clone()
    src = torch.tensor([0, -1, 2, 1, 0, 2, 2, -1, 1], dtype=torch.int32)
    hs.kv_pool_gather_ring(pool, 0, 1, src.cuda())
    assert hs.hswa_pool_check_error(pool) == 0
    for kv in range(2):
        c0, p0 = ref.int4_blocks(before[kv, :, 0], W, d)
        c1, p1 = ref.int4_blocks(pool.ring[kv, :, 0], W, d)
        for s in range(W):
            want = int(src[s]) if src[s] >= 0 else 1
            assert torch.equal(c1[1, :, s], c0[want, :, s]) and torch.equal(p1[1, :, s], p0[want, :, s])
    assert torch.equal(pool.ring[:, 0], before[:, 0]) and torch.equal(pool.ring[:, 2], before[:, 2])


def decode_case(seed, lens, n_qt, hq, hkv, d, W, spread=1.0, q_scale=1.0):
    """W > 0: the ring layer; 0: the paged layer. Returns output rows and references."""
    n = len(lens)
    per = (max(lens) + n_qt + 63) // 64
    pool = make_pool(hkv, d, 1, 1, W or 128, n + 1, n * per + 2)
    layer = 0 if W else 1
    pt = table(seed, n, per, n * per + 2).cuda()
    ids = torch.arange(n, dtype=torch.int32).flip(0).contiguous().cuda()
    refs, qs, kn, vn = [], [], [], []
    for b, L in enumerate(lens):
        lo = max(0, L - W) if W else 0
        k, v = rows(seed + 3 * b, L + n_qt - lo, hkv, d, spread), rows(seed + 3 * b + 1, L + n_qt - lo, hkv, d, spread)
        q = (rows(seed + 3 * b + 2, n_qt, hq, d) * q_scale).to(torch.bfloat16)
        if L > lo:
            hs.kv_pool_append(pool, layer, k[None, : L - lo].cuda(), v[None, : L - lo].cuda(), torch.tensor([lo]).cuda(),
                              seq_ids=ids[b:b + 1] if W else None, page_table=None if W else pt[b:b + 1].contiguous())
        first, end = ref.ranges(n_qt, L, L + n_qt, W)
        vr = ref.int4_values(v).amax(-1) - ref.int4_values(v).amin(-1)
        refs.append(ref.attention(q, ref.int4_values(k), ref.int4_values(v), first, end, lo, weight_eps=ref.F16, v_range=vr))
        qs.append(q); kn.append(k[L - lo:]); vn.append(v[L - lo:])
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_qt, hq, max(lens)), dtype=torch.uint8, device="cuda")
    ws.fill_(0xAB)
    args = [torch.stack(x).cuda() for x in (qs, kn, vn)]
    o = hs.hybrid_decode_fwd(pool, layer, *args, torch.tensor(lens).cuda(), max(lens), ws,
                             seq_ids=ids if W else None, page_table=None if W else pt)
    assert hs.hswa_pool_check_error(pool) == 0
    return o, refs


@pytest.mark.parametrize("lens,n_qt,hq,hkv,d", [
    ([0, 1, 5], 1, 8, 1, 128),                      # nothing cached, a single key; 8 rows
    ([63, 64, 65, 255, 256, 257], 1, 4, 2, 128),    # page and split boundaries; 2 rows
    ([300, 17, 1000], 4, 32, 8, 128),               # 16 rows
    ([700, 4097], 4, 16, 2, 128),                   # 32 rows: two row groups
    ([511, 129], 3, 20, 4, 128),                    # 15 rows, odd group of 5
    ([90, 1500], 3, 21, 3, 64),                     # 21 rows, d = 64
    ([2047, 33, 64, 0], 1, 12, 3, 64),
    ([40000], 1, 8, 8, 128),                        # MHA; one sequence over many splits
    ([9000, 100, 70000], 2, 8, 1, 128),
])
def test_decode_over_pages(lens, n_qt, hq, hkv, d):
    o, refs = decode_case(11, lens, n_qt, hq, hkv, d, 0)
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"seq {b} L={lens[b]}")


@pytest.mark.parametrize("W", [1, 4, 63, 128, 300])
@pytest.mark.parametrize("n_qt,hq,hkv,d", [(1, 8, 1, 128), (4, 16, 2, 128), (2, 6, 2, 64)])
def test_decode_over_ring(W, n_qt, hq, hkv, d):
    lens = [0, 1, 3, 127, 128, 129, 1000, 4099]
    o, refs = decode_case(12, lens, n_qt, hq, hkv, d, W)
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"W={W} seq {b} L={lens[b]}")


def test_decode_of_more_sequences_than_a_warp():
    # past 32 sequences the work list comes from its own kernel
    lens = [(37 * i * i + 5 * i) % 700 for i in range(41)] + [9000]
    o, refs = decode_case(17, lens, 2, 4, 2, 64, 0)
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"seq {b} L={lens[b]}")
    o, refs = decode_case(18, lens[:40], 1, 4, 2, 64, 128)
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"ring seq {b} L={lens[b]}")


# many short contexts, more items (sequences x KV heads) than the CTAs take at once, several to a team of warps
@pytest.mark.parametrize("W,longest,n,n_qt,hq,hkv,d", [
    (128, 5000, 100, 8, 64, 16, 128),   # 32 rows, two warps a team; rings that wrap
    (100, 300, 90, 1, 64, 32, 64),      # 2 rows, one warp a team
    (512, 2000, 80, 3, 32, 8, 128),     # 12 rows, contexts up to the longest that are not split
    (3, 50, 75, 7, 24, 8, 64),          # 21 rows, a ring smaller than a page
    (0, 500, 100, 1, 32, 16, 128),      # pages; tails inside a page
    (0, 63, 76, 4, 64, 8, 64),          # at most one page
    (0, 512, 75, 2, 64, 8, 128)])
def test_decode_of_many_short_contexts(W, longest, n, n_qt, hq, hkv, d):
    lens = [0, 1, longest, longest - 1] + [(41 * i * i + 13 * i) % (longest + 1) for i in range(n - 4)]
    o, refs = decode_case(23, lens, n_qt, hq, hkv, d, W)
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"W={W} seq {b} L={lens[b]}")


@pytest.mark.parametrize("spread,q_scale", [(1e-4, 3e3), (300.0, 3e-3), (1e4, 1e-4), (1e-20, 1e20)])
def test_decode_range_of_values(spread, q_scale):
    # scores of ordinary size from entries far from 1: the f16 operands are scaled per row and per step
    o, refs = decode_case(13, [400, 77], 2, 8, 2, 128, 0, spread, q_scale)
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"spread {spread}")


def test_decode_steps_that_grow_along_the_sequence():
    # V rows whose steps grow by 2^30 along the sequence, peaked and flat weights
    hq = hkv = 2
    d, L = 128, 600
    pool = make_pool(hkv, d, 0, 1, 1, 1, 12)
    pt = table(3, 1, 11, 12).cuda()
    k, v = rows(31, L + 1, hkv, d), rows(32, L + 1, hkv, d)
    grow = torch.pow(2.0, torch.arange(L + 1) * 30.0 / L - 15.0)
    v = (v * grow[:, None, None]).to(torch.bfloat16)
    q = rows(33, 1, hq, d)
    hs.kv_pool_append(pool, 0, k[None, :L].cuda(), v[None, :L].cuda(), torch.tensor([0]).cuda(), page_table=pt)
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 1, 1, hq, L), dtype=torch.uint8, device="cuda")
    o = hs.hybrid_decode_fwd(pool, 0, q[None].cuda(), k[None, L:].contiguous().cuda(), v[None, L:].contiguous().cuda(),
                             torch.tensor([L]).cuda(), L, ws, page_table=pt)
    vv = ref.int4_values(v)
    lo, hi = ref.ranges(1, L, L + 1)
    r = ref.attention(q, ref.int4_values(k), vv, lo, hi, weight_eps=ref.F16, v_range=vv.amax(-1) - vv.amin(-1))
    ref.check(o[0], r, "growing steps")


def test_decode_noalloc_equals_decode_and_repeats():
    hq, hkv, d, lens = 16, 4, 128, [130, 900, 1280]
    pool = make_pool(hkv, d, 0, 1, 1, 1, 64)
    pt = table(7, 3, 20, 64).cuda()
    k, v = (torch.stack([rows(s + b, 1280, hkv, d) for b in range(3)]) for s in (50, 60))
    for b, L in enumerate(lens):
        hs.kv_pool_append(pool, 0, k[b:b + 1, :L].contiguous().cuda(), v[b:b + 1, :L].contiguous().cuda(),
                          torch.tensor([0]).cuda(), page_table=pt[b:b + 1].contiguous())
    q, kn, vn = rows(70, 3, hq, d)[:, None].cuda(), rows(71, 3, hkv, d)[:, None].cuda(), rows(72, 3, hkv, d)[:, None].cuda()
    ctx = torch.tensor(lens).cuda()
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 3, 1, hq, 1280), dtype=torch.uint8, device="cuda")
    a = hs.hybrid_decode_fwd(pool, 0, q, kn, vn, ctx, 1280, ws, page_table=pt)
    b2 = torch.empty_like(a)
    hs.hybrid_decode_fwd_noalloc(pool, 0, q, kn, vn, ctx, 1280, b2, page_table=pt)
    c = hs.hybrid_decode_fwd(pool, 0, q, kn, vn, ctx, 1280, ws, page_table=pt)
    assert hs.hswa_pool_check_error(pool) == 0
    assert torch.equal(a, b2) and torch.equal(a, c)


def test_bad_page_and_ring_row_are_reported():
    pool = make_pool(1, 64, 1, 1, 64, 1, 4)
    pool.data.zero_()
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 1, 1, 1, 100), dtype=torch.uint8, device="cuda")
    ctx = torch.tensor([100], device="cuda")
    pt = torch.tensor([[1, 9]], dtype=torch.int32, device="cuda")
    hs.hybrid_decode_fwd(pool, 1, q, q, q, ctx, 100, ws, page_table=pt)
    assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS
    hs.hybrid_decode_fwd(pool, 0, q, q, q, ctx, 100, ws, seq_ids=torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS
    hs.hybrid_decode_fwd(pool, 0, q, q, q, ctx, 99, ws, seq_ids=torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS
    hs.kv_pool_append(pool, 1, q, q, torch.tensor([64], device="cuda"), page_table=pt)
    assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS
    assert (pool.data == 0).all()


def test_a_bad_ring_row_among_many_leaves_the_others_right():
    n, hkv, hq, d, W, n_qt = 90, 8, 32, 64, 100, 4
    pool = make_pool(hkv, d, 1, 0, W, n, 1)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    start = torch.zeros(n, dtype=torch.int64, device="cuda")
    k, v = rows(1, n * 150, hkv, d).view(n, 150, hkv, d).cuda(), rows(2, n * 150, hkv, d).view(n, 150, hkv, d).cuda()
    hs.kv_pool_append(pool, 0, k, v, start, seq_ids=ids)
    q = rows(3, n * n_qt, hq, d).view(n, n_qt, hq, d).cuda()
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_qt, hq, 150), dtype=torch.uint8, device="cuda")
    args = (pool, 0, q, k[:, :n_qt].contiguous(), v[:, :n_qt].contiguous(), start + 150, 150, ws)
    good = hs.hybrid_decode_fwd(*args, seq_ids=ids)
    assert hs.hswa_pool_check_error(pool) == 0
    wrong = ids.clone()
    wrong[37], wrong[80] = n, -1
    o = torch.empty_like(q)
    hs.hybrid_decode_fwd(*args, seq_ids=wrong, o=o)
    assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS
    keep = [b for b in range(n) if b not in (37, 80)]
    assert torch.equal(o[keep], good[keep])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hs.hybrid_decode_fwd(*args, seq_ids=wrong, o=o)
    wrong.copy_(ids)
    g.replay()
    assert hs.hswa_pool_check_error(pool) == 0 and torch.equal(o, good)


def test_a_workspace_serves_every_smaller_call():
    hq, hkv, d, big = 4, 1, 64, 8192
    pool = make_pool(hkv, d, 0, 1, 1, 1, 130)
    pt = torch.arange(130, dtype=torch.int32).view(1, 130).cuda()
    k, v = rows(1, big, hkv, d)[None].cuda(), rows(2, big, hkv, d)[None].cuda()
    hs.kv_pool_append(pool, 0, k, v, torch.tensor([0]).cuda(), page_table=pt)
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 40, 2, hq, big), dtype=torch.uint8, device="cuda")
    want = {}
    for n in (1, 2, 5, 8, 31, 33, 40):
        for L in (1, 700, 5000, big):
            assert hs.hybrid_decode_workspace_size(pool, n, 2, hq, L) <= ws.numel()
            q, kn, vn = (rows(s, 2, h, d)[None].expand(n, 2, h, d).contiguous().cuda() for s, h in ((3, hq), (4, hkv), (5, hkv)))
            ctx = torch.full((n,), L, dtype=torch.int64).cuda()
            o = hs.hybrid_decode_fwd(pool, 0, q, kn, vn, ctx, L, ws, page_table=pt.expand(n, 130).contiguous())
            want.setdefault(L, o[0].float())
            # the same sequence however the batch cuts it into splits: one rounding of the output apart,
            # and the f16 weights' (2^-11 of the weighted codes)
            assert (o.float() - want[L]).abs().max() <= 2.0 ** -7 * want[L].abs().max() + 2.0 ** -9 * 8
    assert hs.hswa_pool_check_error(pool) == 0
