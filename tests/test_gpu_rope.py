"""GPU: rotary positions over several axes, alone and with the commit into each kind of pool."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref

pytestmark = pytest.mark.gpu


def x_rows(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def plan(rot, n_axes, base=10000.0):
    half = rot // 2
    return [base ** (-2.0 * i / rot) for i in range(half)], [(i * n_axes // half) for i in range(half)]


def positions(seed, n_axes, n, far):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (n_axes, n), generator=g)


def check(got, want, what):
    y, tol = want
    g = got.cpu().double()
    assert ((g - y).abs() <= tol).all(), f"{what}: worst {float(((g - y).abs() / (tol + 1e-30)).max()):.2f} tolerances"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,rot,n_axes,far", [
    (1, 1, 1, 64, 64, 1, 10),
    (1, 32, 8, 128, 128, 3, 1 << 20),
    (7, 5, 1, 128, 32, 2, 5000),
    (1333, 8, 2, 64, 48, 4, 1 << 31),      # four tokens per block, a ragged last block
    (2500, 3, 3, 128, 128, 3, 1 << 20),
])
def test_rope(n, hq, hkv, d, rot, n_axes, far, interleaved):
    inv, axis = plan(rot, n_axes)
    q, k, pos = x_rows(1, n, hq, d), x_rows(2, n, hkv, d), positions(3, n_axes, n, far)
    desc = hs.RopeDesc(inv, axis, n_axes, interleaved)
    qc, kc = q.cuda(), k.cuda()
    qo, ko = hs.rope_fwd(desc, qc, kc, pos.cuda())
    check(qo, ref.rope(q, pos, inv, axis, interleaved), "q")
    check(ko, ref.rope(k, pos, inv, axis, interleaved), "k")
    assert torch.equal(qc.cpu(), q) and torch.equal(kc.cpu(), k)
    assert torch.equal(qo.cpu()[..., rot:], q[..., rot:])  # entries past rot_dim pass
    # in place gives the same bits
    hs.rope_fwd(desc, qc, kc, pos.cuda(), q_out=qc, k_out=kc)
    assert torch.equal(qc, qo) and torch.equal(kc, ko)


def test_position_zero_and_negative_positions():
    inv, axis = plan(64, 1)
    q, k = x_rows(4, 3, 2, 64), x_rows(5, 3, 2, 64)
    pos = torch.tensor([[0, -5, -(1 << 31)]])
    qo, ko = hs.rope_fwd(hs.RopeDesc(inv, axis), q.cuda(), k.cuda(), pos.cuda())
    assert torch.equal(qo[0].cpu(), q[0])
    check(qo, ref.rope(q, pos, inv, axis, False), "q")
    check(ko, ref.rope(k, pos, inv, axis, False), "k")


@pytest.mark.parametrize("fmt", [hs.HSWA_KV_BF16, hs.HSWA_KV_FP8_E4M3, hs.HSWA_KV_INT4])
@pytest.mark.parametrize("swa", [False, True])
@pytest.mark.parametrize("n_seqs,n_tok,hq,hkv,d,interleaved", [(1, 1, 4, 4, 128, False), (3, 77, 6, 2, 64, True),
                                                               (2, 700, 8, 1, 128, False)])
def test_commit_equals_rope_then_append(fmt, swa, n_seqs, n_tok, hq, hkv, d, interleaved):
    inv, axis = plan(d, 3)
    desc = hs.RopeDesc(inv, axis, 3, interleaved)
    per = (n_tok + 30 + 63) // 64
    pools = []
    for _ in range(2):
        p = hs.kv_pool_create(hs.PoolDesc(1, 1, 100, hkv, d, n_seqs, n_seqs * per + 1, kv_format=fmt))
        p.data.fill_(0x11)
        if fmt == hs.HSWA_KV_FP8_E4M3:
            for layer in range(2):
                p.set_scales(layer, [0.01 * (g + 1) for g in range(hkv)], [0.02] * hkv)
        pools.append(p)
    q, k, v = x_rows(6, n_seqs, n_tok, hq, d).cuda(), x_rows(7, n_seqs, n_tok, hkv, d).cuda(), x_rows(8, n_seqs, n_tok, hkv, d).cuda()
    pos = positions(9, 3, n_seqs * n_tok, 100000).cuda()
    start = torch.tensor([30, 0, 5][:n_seqs]).cuda()
    kw = dict(seq_ids=torch.arange(n_seqs, dtype=torch.int32).flip(0).contiguous().cuda()) if swa else dict(
        page_table=torch.randperm(n_seqs * per + 1, generator=torch.Generator().manual_seed(1))[: n_seqs * per]
        .view(n_seqs, per).to(torch.int32).cuda())
    layer = 0 if swa else 1
    q1, k1 = hs.rope_fwd(desc, q, k, pos)
    hs.kv_pool_append(pools[0], layer, k1, v, start, **kw)
    q2, k2 = hs.kv_pool_append_rope(pools[1], layer, desc, q, k, v, pos, start, **kw)
    assert torch.equal(q1, q2) and torch.equal(k1, k2)
    assert torch.equal(pools[0].data, pools[1].data)
    pools[1].data.fill_(0x11)
    q3, k3 = hs.kv_pool_append_rope(pools[1], layer, desc, q, k, v, pos, start, keys_out=False, **kw)
    assert k3 is None and torch.equal(q1, q3) and torch.equal(pools[0].data, pools[1].data)
    for p in pools:
        assert hs.hswa_pool_check_error(p) == 0


def test_append_rope_bounds_are_reported():
    pool = hs.kv_pool_create(hs.PoolDesc(1, 1, 4, 1, 64, 1, 2))
    pool.data.zero_()
    inv, axis = plan(64, 1)
    x = x_rows(1, 1, 2, 1, 64).cuda()
    pos = torch.zeros(1, 2, dtype=torch.int64, device="cuda")
    for bad in ([[5, 5]], [[-1, 0]]):
        hs.kv_pool_append_rope(pool, 1, hs.RopeDesc(inv, axis), x, x, x, pos, torch.tensor([0]).cuda(),
                               page_table=torch.tensor(bad, dtype=torch.int32).cuda())
        assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS
    hs.kv_pool_append_rope(pool, 0, hs.RopeDesc(inv, axis), x, x, x, pos, torch.tensor([0]).cuda(),
                           seq_ids=torch.tensor([3], dtype=torch.int32).cuda())
    assert hs.hswa_pool_check_error(pool) == hs.HSWA_ERR_DEVICE_BOUNDS
    assert (pool.data == 0).all()


def test_rope_on_a_side_stream_and_in_a_graph():
    inv, axis = plan(128, 2)
    desc = hs.RopeDesc(inv, axis, 2)
    q, k, pos = x_rows(1, 40, 4, 128).cuda(), x_rows(2, 40, 2, 128).cuda(), positions(3, 2, 40, 9999).cuda()
    want = hs.rope_fwd(desc, q, k, pos)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hs.rope_fwd(desc, q, k, pos, qo, ko, stream=s)
    s.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hs.rope_fwd(desc, q, k, pos, qo, ko)
    q.copy_(x_rows(9, 40, 4, 128).cuda())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, hs.rope_fwd(desc, q, k, pos)[0])
