"""GPU: caps far above the scores. tanh of a small argument keeps its relative accuracy, so a cap of any size leaves
the scores what they are, up to the rounding that every fp32 score has."""
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref
from test_gpu_score_mod import BF, F8, I4, decode_case, make_pool, prefill_case, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [150.0, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("fmt", [BF, F8, I4])
@pytest.mark.parametrize("bias,mask", [(False, "none"), (True, "docs")])
def test_prefill(cap, fmt, bias, mask):
    prefill_case("full", fmt, [40], 200, 4, 2, 128, cap=cap, bias=bias, mask=mask, q_scale=3.0)
    prefill_case("swa", fmt, [40], 200, 4, 2, 64, W=70, cap=cap, bias=bias, mask=mask, q_scale=3.0)


@pytest.mark.parametrize("cap", [150.0, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("fmt", [BF, F8, I4])
@pytest.mark.parametrize("bias,mask", [(False, "none"), (True, "docs")])
def test_decode(cap, fmt, bias, mask):
    decode_case(fmt, [3, 64, 700], 2, 8, 2, 128, cap=cap, bias=bias, mask=mask, q_scale=3.0)
    decode_case(fmt, [2, 300], 1, 4, 4, 64, W=100, cap=cap, bias=bias, mask=mask, q_scale=3.0)


@pytest.mark.parametrize("fmt", [BF, I4])
@pytest.mark.parametrize("bias,mask", [(False, "none"), (True, "docs")])
def test_scores_around_an_eighth_of_the_cap_and_far_above(fmt, bias, mask):
    prefill_case("full", fmt, [40], 200, 4, 2, 128, cap=200.0, bias=bias, mask=mask, q_scale=12.0)
    prefill_case("swa", fmt, [40], 200, 4, 2, 64, W=70, cap=300.0, bias=bias, mask=mask, q_scale=15.0)
    decode_case(fmt, [3, 64, 700], 2, 8, 2, 128, cap=200.0, bias=bias, mask=mask, q_scale=12.0)
    decode_case(fmt, [2, 300], 1, 4, 4, 64, W=100, cap=300.0, bias=bias, mask=mask, q_scale=15.0)


# Two keys whose values are +1 and -1: the output is tanh of half the difference of their scores, w1 - w2, in which
# an error of the scores is not averaged away. The weights are rounded to bf16 and the output once more: at most
# 2^-8 (w1 + w2) + 2^-8 |o| <= 2 x 2^-8. Over many rows, roundings that are uniform in their half steps and
# independent have a root mean square of at most 2^-8 sqrt((w1^2 + w2^2 + o^2) / 3) <= 2^-8 sqrt(2 / 3).
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [1e4, 1e5, 1e6])
def test_two_keys(d, cap):
    n, hq = 512, 8
    pool = make_pool(BF, 1, d, 0, 1, 64, 1, 8)
    pt = torch.arange(8, dtype=torch.int32).view(1, 8).cuda()
    k, v, q = randn(1, n, 1, d), torch.ones(n, 1, d, dtype=torch.bfloat16), randn(2, n, hq, d, s=2.0)
    v[1::2] = -1
    hs.kv_pool_append(pool, 0, k[None].cuda(), v[None].cuda(), torch.tensor([0]).cuda(), page_table=pt)
    i = torch.arange(n)
    begin = torch.clamp(i - 1, min=0)
    ws = torch.empty(hs.prefill_mod_workspace_size(pool, 1, n), dtype=torch.uint8, device="cuda")
    o = hs.full_prefill_mod_fwd(pool, 0, q[None].cuda(), pt, hs.ScoreMod(cap, key_begin=begin[None].cuda()), ws)
    z = torch.einsum("ihd,jd->ihj", q.double(), k[:, 0].double()) / d ** 0.5
    z = cap * torch.tanh(z / cap)
    own, before = z[i, :, i], z[i, :, torch.clamp(i - 1, min=0)]
    sign = torch.where(i % 2 == 0, 1.0, -1.0).double()[:, None]
    want = torch.where(i[:, None] > 0, sign * torch.tanh((own - before) / 2), torch.ones_like(own))
    off = o[0, :, :, 0].cpu().double() - want
    assert float(off.abs().max()) <= 2 * 2.0 ** -8 + 1e-4
    assert float(off.square().mean().sqrt()) <= 2.0 ** -8
