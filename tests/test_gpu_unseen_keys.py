"""GPU: keys that other rows see, and a query does not, add nothing to its row, however large they are. What they may
change is rounding: the order of its sums and, with a cap, the formula of tanh that its warp uses."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref
from test_gpu_score_mod import BF, F8, I4, held, make_pool, randn, slopes

pytestmark = pytest.mark.gpu


def run(fmt, kind, size, cap, bias, d, hq, hkv, n, cut, W):
    """Two documents, [0, cut) and [cut, n): the first one's keys `size` times larger. Outputs and their references."""
    swa = kind == "swa"
    pool = make_pool(fmt, hkv, d, 1 if swa else 0, 0 if swa else 1, W or 64, 1, -(-n // 64))
    pt = torch.arange(-(-n // 64), dtype=torch.int32).view(1, -1).cuda()
    k, v, q = randn(1, n, hkv, d), randn(2, n, hkv, d), randn(3, n, hq, d, s=1.5)
    k[:cut] = (k[:cut].float() * size).to(torch.bfloat16)
    i = torch.arange(n)
    begin = torch.where(i < cut, 0, cut)
    sl = slopes(hq) if bias else None
    if kind == "decode":  # the last tokens of the second document, one of the first among them
        n_q = 4
        q, i = q[n - n_q:], i[n - n_q:]
        begin, end = begin[n - n_q:].clone(), i + 1
        begin[1], end[1] = 0, cut
        hs.kv_pool_append(pool, 0, k[None, : n - n_q].cuda(), v[None, : n - n_q].cuda(), torch.tensor([0]).cuda(),
                          page_table=pt)
        ws = torch.empty(hs.hybrid_decode_workspace_size(pool, 1, n_q, hq, n), dtype=torch.uint8, device="cuda")
        mod = hs.ScoreMod(cap, sl.cuda() if bias else None, begin[None].cuda(), end[None].cuda())
        o = hs.hybrid_decode_mod_fwd(pool, 0, *[x[None].contiguous().cuda() for x in (q, k[n - n_q:], v[n - n_q:])],
                                     torch.tensor([n - n_q]).cuda(), n - n_q, mod, ws, page_table=pt)
    else:
        mod = hs.ScoreMod(cap, sl.cuda() if bias else None, begin[None].cuda())
        ws = torch.empty(hs.prefill_mod_workspace_size(pool, 1, n), dtype=torch.uint8, device="cuda")
        if swa:
            o = hs.swa_prefill_mod_fwd(pool, 0, q[None].cuda(), k[None].cuda(), v[None].cuda(), mod, ws)
        else:
            hs.kv_pool_append(pool, 0, k[None].cuda(), v[None].cuda(), torch.tensor([0]).cuda(), page_table=pt)
            o = hs.full_prefill_mod_fwd(pool, 0, q[None].cuda(), pt, mod, ws)
        end = i + 1
    assert hs.hswa_pool_check_error(pool) == 0
    lo, hi = ref.ranges(len(i), int(i[0]), n, W, begin, end)
    as_bf16 = kind != "decode"
    hk, hv = (x.double() if swa else held(fmt, x, as_bf16) for x in (k, v))
    i4 = fmt == I4 and kind == "decode"
    r = ref.attention(q, hk, hv, lo, hi, 0, i, cap, sl, weight_eps=ref.F16 if i4 else ref.BF16,
                      v_range=hv.amax(-1) - hv.amin(-1) if i4 else None)
    small = begin == cut  # the rows that do not see the large keys
    return o[0][small.cuda()], ref.Attention(r.o[small], r.tol[small])


@pytest.mark.parametrize("kind", ["full", "swa", "decode"])
@pytest.mark.parametrize("fmt", [BF, F8, I4])
@pytest.mark.parametrize("size", [30.0, 1e3, 1e30])
@pytest.mark.parametrize("cap,bias", [(50.0, False), (50.0, True), (1e6, False), (0.0, True)])
def test_rows_do_not_feel_keys_they_do_not_see(kind, fmt, size, cap, bias):
    if fmt == F8 and size > 1e3:
        size = 25.0  # the format's range
    o, r = run(fmt, kind, size, cap, bias, 128, 8, 2, 333, 150, 200 if kind == "swa" else 0)
    ref.check(o, r, f"{kind} fmt={fmt} size={size}")
