"""GPU: capped scores, distance bias and per-row key ranges (documents, prefixes, padding) in the prefill of
sliding-window and full layers and in decode, over bf16, FP8 and 4-bit pools; prefill over 4-bit pools."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref

pytestmark = pytest.mark.gpu
BF, F8, I4 = hs.HSWA_KV_BF16, hs.HSWA_KV_FP8_E4M3, hs.HSWA_KV_INT4
SCALE8 = 0.0625  # FP8 entries of size up to 28


def randn(seed, *shape, s=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * s).to(torch.bfloat16)


def held(fmt, x, as_bf16=True):
    """The values entries x stand for in a pool, as a prefill (rounded to bf16) or a decode step reads them."""
    if fmt == BF:
        return x.double()
    if fmt == F8:
        y = ((x.float() * (1 / SCALE8)).to(torch.float8_e4m3fn).float() * SCALE8)
    else:
        y = ref.int4_values(x).float()
    return y.to(torch.bfloat16).double() if as_bf16 else y.double()


def make_pool(fmt, hkv, d, n_swa, n_full, W, seqs, pages):
    pool = hs.kv_pool_create(hs.PoolDesc(n_swa, n_full, W, hkv, d, seqs, pages, kv_format=fmt))
    pool.data.fill_(0xFF)  # NaN wherever nothing was committed
    if fmt == F8:
        for layer in range(n_swa + n_full):
            pool.set_scales(layer, [SCALE8] * hkv, [SCALE8] * hkv)
    return pool


def documents(seed, n, mean):
    g = torch.Generator().manual_seed(seed)
    start, at = torch.zeros(n, dtype=torch.int64), 0
    while at < n:
        size = 1 + int(torch.randint(0, 2 * mean, (1,), generator=g))
        start[at: at + size] = at
        at += size
    return start


def key_ranges(mask, seed, B, n_q, starts):
    """(key_begin, key_end) [B, n_q] of a mask kind; padding rows see nothing."""
    if mask == "none":
        return None, None
    begin, end = torch.zeros(B, n_q, dtype=torch.int64), torch.zeros(B, n_q, dtype=torch.int64)
    for b, P in enumerate(starts):
        i = torch.arange(P, P + n_q)
        end[b] = i + 1
        if mask in ("docs", "pad"):
            begin[b] = documents(seed + b, P + n_q, max(1, (P + n_q) // 5))[P:]
        if mask == "prefix":
            end[b] = torch.maximum(i + 1, torch.tensor(P + n_q // 2 + b))
        if mask == "pad":
            end[b, n_q - n_q // 3:] = begin[b, n_q - n_q // 3:] - b  # begin >= end
        if mask == "wild":  # any values are allowed
            begin[b] = torch.where(i % 3 == 0, i - 5, torch.full_like(i, -(1 << 62)))
            end[b] = torch.where(i % 7 == 0, torch.full_like(i, 1 << 62), i - 2)
    return (None if mask == "prefix" else begin), end


def slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32)


def prefill_case(kind, fmt, starts, n_q, hq, hkv, d, W=0, cap=0.0, bias=False, mask="none", q_scale=1.5, seed=5,
                 plain=False, stale=False):
    """stale: entries no query of their sequence sees are not committed or hold NaN."""
    B, swa = len(starts), kind == "swa"
    per = max((P + n_q + 63) // 64 for P in starts)
    pool = make_pool(fmt, hkv, d, 1 if swa else 0, 0 if swa else 1, W or 64, B + 1, B * per + 2)
    pt = torch.randperm(B * per + 2, generator=torch.Generator().manual_seed(3))[: B * per].view(B, per).to(torch.int32)
    ids = torch.arange(B, dtype=torch.int32).flip(0).contiguous()
    begin, end = key_ranges(mask, seed, B, n_q, starts)
    sl = slopes(hq) if bias else None
    q = randn(seed, B, n_q, hq, d, s=q_scale)
    kc, vc, refs = [], [], []
    for b, P in enumerate(starts):
        k, v = randn(seed + 10 + b, P + n_q, hkv, d), randn(seed + 20 + b, P + n_q, hkv, d)
        i = torch.arange(P, P + n_q)
        lo, hi = ref.ranges(n_q, P, P + n_q, W if swa else 0, None if begin is None else begin[b],
                            None if end is None else end[b])
        lo = torch.clamp(lo, min=0)
        some = hi > lo
        first, last = (int(lo[some].min()), int(hi[some].max())) if some.any() else (0, 0)
        if swa:
            pre = max(0, P - W)
            hk = torch.cat([held(fmt, k[:P]), k[P:].double()])
            hv = torch.cat([held(fmt, v[:P]), v[P:].double()])
            if P > pre:
                hs.kv_pool_append(pool, 0, k[None, pre:P].cuda(), v[None, pre:P].cuda(), torch.tensor([pre]).cuda(),
                                  seq_ids=ids[b:b + 1].cuda())
        else:
            hk, hv = held(fmt, k), held(fmt, v)
            a, e = (first, last) if stale else (0, P + n_q)
            if e > a:
                hs.kv_pool_append(pool, 0, k[None, a:e].cuda(), v[None, a:e].cuda(), torch.tensor([a]).cuda(),
                                  page_table=pt[b:b + 1].contiguous().cuda())
            if stale:  # pages wholly unseen need not exist
                pt[b, : first // 64] = -1
                pt[b, (last + 63) // 64:] = 1 << 30
        refs.append(ref.attention(q[b], hk, hv, lo, hi, 0, i, cap, sl))
        kk, vv = k[P:].clone(), v[P:].clone()
        if stale and swa:
            unseen = (i < first) | (i >= last)
            kk[unseen], vv[unseen] = float("nan"), float("nan")
        kc.append(kk); vc.append(vv)
    start = torch.tensor(starts).cuda()
    args = dict(start_pos=start)
    if plain:
        assert mask == "none" and not cap and not bias
    else:
        mod = hs.ScoreMod(cap, sl.cuda() if bias else None, None if begin is None else begin.cuda(),
                          None if end is None else end.cuda())
        ws = torch.empty(hs.prefill_mod_workspace_size(pool, B, n_q), dtype=torch.uint8, device="cuda").fill_(0xCD)
    if swa:
        x = (q.cuda(), torch.stack(kc).cuda(), torch.stack(vc).cuda())
        args["seq_ids"] = ids.cuda()
        o = hs.swa_prefill_fwd(pool, 0, *x, **args) if plain else hs.swa_prefill_mod_fwd(pool, 0, *x, mod, ws, **args)
    elif plain:
        o = hs.full_prefill_fwd(pool, 0, q.cuda(), pt.cuda(), **args)
    else:
        o = hs.full_prefill_mod_fwd(pool, 0, q.cuda(), pt.cuda(), mod, ws, **args)
    assert hs.hswa_pool_check_error(pool) == 0
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"{kind} fmt={fmt} seq {b}")


@pytest.mark.parametrize("starts,n_q,hq,hkv,d", [
    ([0], 1, 1, 1, 64), ([5], 3, 4, 2, 128), ([0, 200], 300, 6, 2, 128), ([129], 130, 4, 4, 64), ([63, 64], 700, 8, 2, 64)])
def test_prefill_over_4bit_pages(starts, n_q, hq, hkv, d):
    prefill_case("full", I4, starts, n_q, hq, hkv, d, plain=True)


@pytest.mark.parametrize("W,starts,n_q,hq,hkv,d", [
    (128, [0], 200, 4, 2, 128), (128, [128, 77], 300, 4, 1, 128), (50, [33], 129, 3, 1, 64), (300, [500], 400, 4, 2, 128),
    (256, [256], 130, 2, 2, 64), (1, [7], 20, 2, 1, 64)])
def test_swa_prefill_over_a_4bit_ring(W, starts, n_q, hq, hkv, d):
    prefill_case("swa", I4, starts, n_q, hq, hkv, d, W=W, plain=True)


@pytest.mark.parametrize("fmt", [BF, F8, I4])
@pytest.mark.parametrize("cap,bias,mask", [(0.0, False, "docs"), (5.0, False, "none"), (0.0, True, "prefix"),
                                           (30.0, True, "pad"), (2.0, False, "wild")])
def test_full_prefill(fmt, cap, bias, mask):
    prefill_case("full", fmt, [0, 100], 333, 8, 2, 128, cap=cap, bias=bias, mask=mask)


@pytest.mark.parametrize("starts,n_q,hq,hkv,d", [([0], 1, 2, 1, 64), ([3], 2, 3, 3, 128), ([64], 64, 5, 1, 64),
                                                 ([511, 0, 1], 129, 6, 2, 128), ([1000], 513, 9, 3, 64)])
@pytest.mark.parametrize("mask", ["docs", "prefix", "wild"])
def test_full_prefill_shapes(starts, n_q, hq, hkv, d, mask):
    prefill_case("full", BF, starts, n_q, hq, hkv, d, cap=20.0, bias=True, mask=mask)


@pytest.mark.parametrize("fmt", [BF, I4])
@pytest.mark.parametrize("mask", ["docs", "pad"])
def test_full_prefill_reads_only_what_is_seen(fmt, mask):
    prefill_case("full", fmt, [300, 77], 200, 4, 2, 128, mask=mask, stale=True)
    prefill_case("full", fmt, [300, 77], 200, 3, 1, 64, mask=mask, stale=True)


@pytest.mark.parametrize("fmt", [BF, F8, I4])
@pytest.mark.parametrize("W,starts", [(1, [9]), (40, [0, 100]), (128, [128, 256]), (129, [33, 0]), (300, [700, 40]),
                                      (512, [512, 1024])])
@pytest.mark.parametrize("cap,bias,mask", [(10.0, False, "none"), (0.0, True, "prefix"), (25.0, True, "docs"),
                                           (0.0, True, "none"), (3.0, True, "none")])
def test_swa_prefill(fmt, W, starts, cap, bias, mask):
    prefill_case("swa", fmt, starts, 270, 4, 2, 128, W=W, cap=cap, bias=bias, mask=mask)


@pytest.mark.parametrize("starts,n_q,hq,hkv,d,W", [([0], 1, 1, 1, 128, 7), ([50], 130, 3, 1, 64, 64), ([0], 400, 5, 5, 64, 200)])
@pytest.mark.parametrize("mask", ["pad", "wild"])
def test_swa_prefill_shapes_and_padding(starts, n_q, hq, hkv, d, W, mask):
    prefill_case("swa", BF, starts, n_q, hq, hkv, d, W=W, cap=50.0, mask=mask, stale=True)


@pytest.mark.parametrize("q_scale,cap", [(0.1, 50.0), (8.0, 3.0), (60.0, 50.0), (2.0, 1000.0), (3.0, 0.05)])
def test_cap_sizes(q_scale, cap):
    # within the cap, far beyond it, and caps whose powers leave the polynomial's range
    prefill_case("full", BF, [40], 200, 4, 2, 128, cap=cap, q_scale=q_scale)
    prefill_case("full", BF, [40], 200, 4, 2, 64, cap=cap, q_scale=q_scale)


def decode_case(fmt, lens, n_qt, hq, hkv, d, W=0, cap=0.0, bias=False, mask="none", seed=9, q_scale=1.5):
    n, swa = len(lens), W > 0
    per = (max(lens) + n_qt + 63) // 64
    pool = make_pool(fmt, hkv, d, 1 if swa else 0, 0 if swa else 1, W or 64, n, n * per + 2)
    pt = torch.randperm(n * per + 2, generator=torch.Generator().manual_seed(3))[: n * per].view(n, per).to(torch.int32)
    ids = torch.arange(n, dtype=torch.int32).flip(0).contiguous().cuda()
    begin, end = key_ranges(mask, seed, n, n_qt, lens)
    sl = slopes(hq) if bias else None
    qs, kn, vn, refs = [], [], [], []
    for b, L in enumerate(lens):
        k, v = randn(seed + 10 + b, L + n_qt, hkv, d), randn(seed + 20 + b, L + n_qt, hkv, d)
        q = randn(seed + b, n_qt, hq, d, s=q_scale)
        lo, hi = ref.ranges(n_qt, L, L + n_qt, W, None if begin is None else begin[b], None if end is None else end[b])
        lo = torch.clamp(lo, min=0)
        some = hi > lo
        first = int(lo[some].min()) if some.any() else L
        a = max(max(0, L - W) if swa else 0, first)  # what no row sees is never committed
        if L > a:
            hs.kv_pool_append(pool, 0, k[None, a:L].cuda(), v[None, a:L].cuda(), torch.tensor([a]).cuda(),
                              seq_ids=ids[b:b + 1] if swa else None,
                              page_table=None if swa else pt[b:b + 1].contiguous().cuda())
        if not swa:
            pt[b, : first // 64] = -1
        hv = held(fmt, v, False)
        i = torch.arange(L, L + n_qt)
        refs.append(ref.attention(q, held(fmt, k, False), hv, lo, hi, 0, i, cap, sl,
                                  weight_eps=ref.F16 if fmt == I4 else ref.BF16,
                                  v_range=hv.amax(-1) - hv.amin(-1) if fmt == I4 else None))
        qs.append(q); kn.append(k[L:]); vn.append(v[L:])
    x = [torch.stack(t).cuda() for t in (qs, kn, vn)]
    mod = hs.ScoreMod(cap, sl.cuda() if bias else None, None if begin is None else begin.cuda(),
                      None if end is None else end.cuda())
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, n, n_qt, hq, max(lens)), dtype=torch.uint8, device="cuda").fill_(0xAB)
    o = hs.hybrid_decode_mod_fwd(pool, 0, *x, torch.tensor(lens).cuda(), max(lens), mod, ws, seq_ids=ids if swa else None,
                                 page_table=None if swa else pt.cuda())
    assert hs.hswa_pool_check_error(pool) == 0
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"decode fmt={fmt} seq {b}")


@pytest.mark.parametrize("fmt", [BF, F8, I4])
@pytest.mark.parametrize("cap,bias,mask", [(20.0, False, "none"), (0.0, True, "none"), (0.0, False, "docs"),
                                           (3.0, True, "wild"), (0.0, False, "pad"), (8.0, False, "prefix")])
@pytest.mark.parametrize("lens,n_qt,hq,hkv,d,W", [
    ([0, 3, 64, 700], 1, 8, 1, 128, 0), ([130, 2500], 4, 16, 2, 128, 0), ([65, 1], 3, 9, 3, 64, 0),
    ([0, 500, 77], 4, 8, 2, 128, 100)])
def test_decode(fmt, cap, bias, mask, lens, n_qt, hq, hkv, d, W):
    decode_case(fmt, lens, n_qt, hq, hkv, d, W, cap, bias, mask)


@pytest.mark.parametrize("cap,bias,mask", [(20.0, True, "none"), (0.0, False, "docs"), (5.0, False, "wild"),
                                           (0.0, True, "pad")])
@pytest.mark.parametrize("n_qt,hq,hkv,d,W", [(4, 64, 8, 128, 100), (2, 16, 8, 64, 0)])
def test_decode_of_many_short_4bit_contexts(cap, bias, mask, n_qt, hq, hkv, d, W):
    decode_case(I4, [0, 1, 400] + [(53 * i * i + 7 * i) % 400 for i in range(75)], n_qt, hq, hkv, d, W, cap, bias, mask)


@pytest.mark.parametrize("fmt", [BF, F8, I4])
def test_padded_new_tokens_may_hold_anything(fmt):
    # rows 2 and 3 of a step are padding: they see nothing, nothing sees them, their k and v are NaN
    hq, hkv, d, L = 4, 2, 64, 100
    pool = make_pool(fmt, hkv, d, 0, 1, 64, 1, 3)
    pt = torch.tensor([[2, 0]], dtype=torch.int32).cuda()
    k, v, q = randn(1, L + 2, hkv, d), randn(2, L + 2, hkv, d), randn(3, 4, hq, d)
    hs.kv_pool_append(pool, 0, k[None, :L].cuda(), v[None, :L].cuda(), torch.tensor([0]).cuda(), page_table=pt)
    nan = torch.full((2, hkv, d), float("nan"), dtype=torch.bfloat16)
    end = torch.tensor([[L + 1, L + 2, 0, 0]])
    ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 1, 4, hq, L), dtype=torch.uint8, device="cuda")
    o = hs.hybrid_decode_mod_fwd(pool, 0, q[None].cuda(), torch.cat([k[L:], nan])[None].cuda(),
                                 torch.cat([v[L:], nan])[None].cuda(), torch.tensor([L]).cuda(), L,
                                 hs.ScoreMod(key_end=end.cuda()), ws, page_table=pt)
    assert hs.hswa_pool_check_error(pool) == 0
    assert (o[0, 2:] == 0).all()
    lo, hi = ref.ranges(2, L, L + 2)
    hv = held(fmt, v, False)
    ref.check(o[0, :2], ref.attention(q[:2], held(fmt, k, False), hv, lo, hi, weight_eps=ref.F16 if fmt == I4 else ref.BF16,
                                      v_range=hv.amax(-1) - hv.amin(-1) if fmt == I4 else None), "real rows")


def test_decode_range_far_into_a_long_context():
    # only the last document of a long context is seen: the splits start at its page
    decode_case(I4, [30000, 9000], 2, 4, 1, 64, mask="docs")
    decode_case(BF, [30000, 9000], 2, 4, 1, 64, mask="docs")


def test_plain_mod_equals_plain_call_within_rounding_and_repeats_bit_for_bit():
    hq, hkv, d, n = 4, 2, 128, 500
    pool = make_pool(BF, hkv, d, 0, 1, 64, 1, 8)
    pt = torch.arange(8, dtype=torch.int32).view(1, 8).cuda()
    k, v, q = randn(1, 1, n, hkv, d).cuda(), randn(2, 1, n, hkv, d).cuda(), randn(3, 1, n, hq, d).cuda()
    hs.kv_pool_append(pool, 0, k, v, torch.tensor([0]).cuda(), page_table=pt)
    a = hs.full_prefill_fwd(pool, 0, q, pt)
    b = hs.full_prefill_mod_fwd(pool, 0, q, pt, hs.ScoreMod())  # no ranges: no workspace
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * a.float().abs().max()
    i = torch.arange(n)
    mod = hs.ScoreMod(key_begin=(i // 100 * 100)[None].cuda(), key_end=(i + 1)[None].cuda())
    ws = torch.empty(hs.prefill_mod_workspace_size(pool, 1, n), dtype=torch.uint8, device="cuda")
    c = [hs.full_prefill_mod_fwd(pool, 0, q, pt, mod, ws) for _ in range(3)]
    assert torch.equal(c[0], c[1]) and torch.equal(c[0], c[2])


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("which", ["tail", "all", "every_other_tile"])
def test_tiles_that_see_nothing(hq, hkv, d, which):
    # many units in a row without a single key
    n, B = 1500, 3
    pool = make_pool(BF, hkv, d, 0, 1, 64, B, 24 * B)
    pt = torch.arange(24 * B, dtype=torch.int32).view(B, 24).cuda()
    k, v, q = randn(1, B, n, hkv, d), randn(2, B, n, hkv, d), randn(3, B, n, hq, d)
    hs.kv_pool_append(pool, 0, k.cuda(), v.cuda(), torch.zeros(B, dtype=torch.int64).cuda(), page_table=pt)
    i = torch.arange(n)
    empty = {"tail": i >= 300, "all": i >= 0, "every_other_tile": (i // 128) % 2 == 0}[which]
    end = torch.where(empty, torch.zeros_like(i), i + 1)[None].expand(B, n).contiguous()
    ws = torch.empty(hs.prefill_mod_workspace_size(pool, B, n), dtype=torch.uint8, device="cuda")
    o = hs.full_prefill_mod_fwd(pool, 0, q.cuda(), pt, hs.ScoreMod(key_end=end.cuda()), ws)
    assert hs.hswa_pool_check_error(pool) == 0
    assert (o[:, empty.cuda()] == 0).all()
    lo, hi = ref.ranges(n, 0, n, 0, None, end[0])
    for b in range(B):
        ref.check(o[b], ref.attention(q[b], k[b], v[b], lo, hi), f"seq {b}")


def test_rows_past_the_chunk_are_left_as_they_were():
    hq, hkv, d, n = 2, 1, 64, 130
    pool = make_pool(BF, hkv, d, 0, 1, 64, 1, 4)
    pt = torch.arange(4, dtype=torch.int32).view(1, 4).cuda()
    hs.kv_pool_append(pool, 0, randn(1, 1, n, hkv, d).cuda(), randn(2, 1, n, hkv, d).cuda(), torch.tensor([0]).cuda(), page_table=pt)
    buf = torch.full((n + 200, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    hs.full_prefill_mod_fwd(pool, 0, randn(3, 1, n, hq, d).cuda(), pt, hs.ScoreMod(softcap=9.0), o=buf[:n].view(1, n, hq, d))
    assert hs.hswa_pool_check_error(pool) == 0
    assert (buf[n:] == 7.0).all() and not (buf[:n] == 7.0).all()


def test_captured_and_replayed_on_new_inputs():
    hq, hkv, d, n = 4, 2, 128, 200
    pool = make_pool(I4, hkv, d, 0, 1, 64, 1, 8)
    pt = torch.arange(8, dtype=torch.int32).view(1, 8).cuda()
    k, v, q = randn(1, 1, n, hkv, d).cuda(), randn(2, 1, n, hkv, d).cuda(), randn(3, 1, n, hq, d).cuda()
    begin = torch.zeros(1, n, dtype=torch.int64, device="cuda")
    mod = hs.ScoreMod(softcap=15.0, key_begin=begin)
    ws = torch.empty(hs.prefill_mod_workspace_size(pool, 1, n), dtype=torch.uint8, device="cuda")
    zero = torch.tensor([0]).cuda()
    q1, kn, vn = randn(4, 1, 1, hq, d).cuda(), randn(5, 1, 1, hkv, d).cuda(), randn(6, 1, 1, hkv, d).cuda()
    b1 = torch.zeros(1, 1, dtype=torch.int64, device="cuda")
    mod1 = hs.ScoreMod(softcap=15.0, key_begin=b1)
    ws1 = torch.empty(hs.hybrid_decode_workspace_size(pool, 1, 1, hq, n), dtype=torch.uint8, device="cuda")
    ctx = torch.tensor([n]).cuda()
    o, o1 = torch.empty_like(q), torch.empty_like(q1)

    def step():
        hs.kv_pool_append(pool, 0, k, v, zero, page_table=pt)
        hs.full_prefill_mod_fwd(pool, 0, q, pt, mod, ws, o=o)
        hs.hybrid_decode_mod_fwd(pool, 0, q1, kn, vn, ctx, n, mod1, ws1, page_table=pt, o=o1)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for s in range(2):
        k.copy_(randn(11 + s, 1, n, hkv, d).cuda()); q.copy_(randn(13 + s, 1, n, hq, d).cuda())
        begin.copy_((torch.arange(n) // (40 + s) * (40 + s))[None].cuda())
        b1.fill_(33 + s)
        g.replay()
        torch.cuda.synchronize()
        a, a1 = o.clone(), o1.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, o) and torch.equal(a1, o1)
    assert hs.hswa_pool_check_error(pool) == 0


def test_pages_out_of_range_are_reported():
    pool = make_pool(I4, 1, 64, 0, 1, 64, 1, 2)
    pool.data.zero_()
    q = randn(1, 1, 100, 1, 64).cuda()
    for fn in (lambda t: hs.full_prefill_fwd(pool, 0, q, t), lambda t: hs.full_prefill_mod_fwd(pool, 0, q, t, hs.ScoreMod(softcap=1.0))):
        fn(torch.tensor([[0, 2]], dtype=torch.int32).cuda())
        assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("fmt", [BF, F8, I4])
def test_a_request_from_prompt_to_tokens(fmt):
    # rotate -> commit -> prefill with an image seen in both directions and capped scores, in two chunks,
    # on a sliding-window and a full layer; then decode steps with drafts, committed token by token
    hq, hkv, d, W, P, C = 8, 2, 128, 100, 150, 130
    total = P + C + 4
    pool = make_pool(fmt, hkv, d, 1, 1, W, 1, 6)
    pt = torch.tensor([[4, 1, 5, 0, 2]], dtype=torch.int32).cuda()
    sid = torch.zeros(1, dtype=torch.int32).cuda()
    inv = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    axis = [i % 3 for i in range(d // 2)]
    rope = hs.RopeDesc(inv, axis, 3)
    pos = torch.stack([torch.arange(total), torch.arange(total) // 3, torch.arange(total) % 50])
    raw = {layer: [randn(40 + 3 * layer + i, total, h, d) for i, h in enumerate((hq, hkv, hkv))] for layer in (0, 1)}
    turned = {}
    for layer in (0, 1):
        q, k, v = raw[layer]
        a, b = hs.rope_fwd(rope, q.cuda(), k.cuda(), pos.cuda())
        turned[layer] = (a.cpu(), b.cpu(), v)
    end_all = torch.arange(total) + 1
    end_all[20:90] = 90  # the image
    for c0, c1 in ((0, P), (P, P + C)):
        end = end_all[None, c0:c1].contiguous().cuda()
        mod = hs.ScoreMod(softcap=30.0, key_end=end)
        ws = torch.empty(hs.prefill_mod_workspace_size(pool, 1, c1 - c0), dtype=torch.uint8, device="cuda")
        start = torch.tensor([c0]).cuda()
        px = pos[:, c0:c1].contiguous().cuda()
        for layer in (0, 1):
            q, k, v = (x[None, c0:c1].contiguous().cuda() for x in raw[layer])
            if layer == 0:
                q, k = hs.rope_fwd(rope, q, k, px)
                o = hs.swa_prefill_mod_fwd(pool, 0, q, k, v, mod, ws, start_pos=start, seq_ids=sid)
                hs.kv_pool_append(pool, 0, k, v, start, seq_ids=sid)
            else:
                q, _ = hs.kv_pool_append_rope(pool, 1, rope, q, k, v, px, start, page_table=pt, keys_out=False)
                o = hs.full_prefill_mod_fwd(pool, 1, q, pt, mod, ws, start_pos=start)
            tq, tk, tv = turned[layer]
            lo, hi = ref.ranges(c1 - c0, c0, c1, W if layer == 0 else 0, None, end_all[c0:c1])
            hk = torch.cat([held(fmt, tk[:c0]), tk[c0:c1].double() if layer == 0 else held(fmt, tk[c0:c1])])
            hv = torch.cat([held(fmt, tv[:c0]), tv[c0:c1].double() if layer == 0 else held(fmt, tv[c0:c1])])
            ref.check(o[0], ref.attention(tq[c0:c1], hk, hv, lo, hi, 0, None, 30.0), f"layer {layer} chunk {c0}")
    for L, n in ((P + C, 3), (P + C + 1, 1)):
        ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 1, n, hq, L), dtype=torch.uint8, device="cuda")
        for layer in (0, 1):
            tq, tk, tv = turned[layer]
            q, k, v = (x[None, L:L + n].contiguous().cuda() for x in (tq, tk, tv))
            kw = dict(seq_ids=sid) if layer == 0 else dict(page_table=pt)
            ctx = torch.tensor([L]).cuda()
            o = hs.hybrid_decode_mod_fwd(pool, layer, q, k, v, ctx, L, hs.ScoreMod(softcap=30.0), ws, **kw)
            lo, hi = ref.ranges(n, L, L + n, W if layer == 0 else 0)
            hv = held(fmt, tv[:L + n], False)
            r = ref.attention(tq[L:L + n], held(fmt, tk[:L + n], False), hv, lo, hi, 0, None, 30.0,
                              weight_eps=ref.F16 if fmt == I4 else ref.BF16,
                              v_range=hv.amax(-1) - hv.amin(-1) if fmt == I4 else None)
            ref.check(o[0], r, f"layer {layer} decode at {L}")
            hs.kv_pool_append(pool, layer, k[:, :1].contiguous(), v[:, :1].contiguous(), ctx, **kw)
    assert hs.hswa_pool_check_error(pool) == 0


def test_calls_in_a_row_share_a_workspace_and_feed_each_other():
    """Each call's output is the next one's queries; sizes on both sides of the one-launch key ranges."""
    hq, hkv, d = 4, 2, 64
    sizes = [150, 4500, 130, 900]
    n = max(sizes)
    per = (n + 63) // 64
    pool = make_pool(BF, hkv, d, 0, 1, 64, 1, per)
    pt = torch.arange(per, dtype=torch.int32).view(1, per).cuda()
    zero = torch.tensor([0]).cuda()
    hs.kv_pool_append(pool, 0, randn(1, 1, n, hkv, d).cuda(), randn(2, 1, n, hkv, d).cuda(), zero, page_table=pt)
    q = randn(3, 1, n, hq, d).cuda()
    mods = [hs.ScoreMod(key_begin=(torch.arange(m) // (20 + m // 7) * (20 + m // 7))[None].cuda()) for m in sizes]
    ws = torch.empty(hs.prefill_mod_workspace_size(pool, 1, n), dtype=torch.uint8, device="cuda")

    def chain(wait):
        x = q.clone()
        for _ in range(3):
            for m, mod in zip(sizes, mods):
                y = x.clone()
                y[:, :m] = hs.full_prefill_mod_fwd(pool, 0, x[:, :m].contiguous(), pt, mod, ws, start_pos=zero)
                x = y
                if wait:
                    torch.cuda.synchronize()
        return x

    assert torch.equal(chain(False), chain(True))
    assert hs.hswa_pool_check_error(pool) == 0
