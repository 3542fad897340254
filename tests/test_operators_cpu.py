"""Without a GPU: layout of 4-bit pools, the refusals of the rotary, 4-bit and modified-score calls, and the
plain forms the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_sliding_window_swa_b200 as hs
import operators_ref as ref
from hybrid_sliding_window_swa_b200 import _build

INVALID, SHAPE = hs.HSWA_ERR_INVALID_ARG, hs.HSWA_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return hs.load_library()


@pytest.mark.parametrize("args", [(60, 10, 128, 8, 128, 1, 1 << 14), (6, 1, 128, 8, 128, 256, 200_000), (1, 1, 1, 1, 64, 3, 7),
                                  (2, 1, 5, 3, 64, 2, 9)])
def test_layout_of_a_4bit_pool(lib, args):
    n_swa, n_full, W, hkv, d, seqs, pages = args
    total, swa, full = hs.kv_pool_layout(hs.PoolDesc(*args, kv_format=hs.HSWA_KV_INT4))
    block = lambda rows: rows * d // 2 + -(-rows * 4 // 16) * 16
    assert swa == -(-2 * seqs * n_swa * hkv * block(W) // 256) * 256
    assert full == -(-2 * n_full * pages * hkv * block(64) // 256) * 256
    assert total == swa + full + 256
    if d == 128:  # 68 bytes a row against 256
        assert block(64) * 256 == 64 * 68 * 256
        assert full * 256 // 68 <= hs.kv_pool_layout(hs.PoolDesc(*args))[2] + 4 * 256


def rope_desc(**kw):
    c = hs.RopeDesc([1.0 / (i + 1) for i in range(32)], [i % 3 for i in range(32)], 3).c().contents
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(c, k)[v[0]] = v[1]
        else:
            setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), SHAPE), (dict(rot_dim=24), SHAPE), (dict(rot_dim=-16), SHAPE), (dict(rot_dim=128), SHAPE),
    (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE), (dict(axis=(5, 3)), INVALID),
    (dict(inv_freq=(3, float("nan"))), INVALID), (dict(inv_freq=(31, float("inf"))), INVALID)])
def test_rope_descriptors_are_checked(lib, kw, code):
    x = ctypes.c_void_p(0x1000)
    assert lib.rope_fwd(rope_desc(**kw), 64, 1, x, x, x, 1, x, x, 1, None) == code
    assert b"rope_fwd" in lib.hswa_last_error()


def test_rope_arguments_are_checked(lib):
    r, x = rope_desc(), ctypes.c_void_p(0x1000)
    assert lib.rope_fwd(None, 64, 1, x, x, x, 1, x, x, 1, None) == INVALID
    assert lib.rope_fwd(r, 96, 1, x, x, x, 1, x, x, 1, None) == SHAPE
    assert lib.rope_fwd(r, 64, -1, x, x, x, 1, x, x, 1, None) == INVALID
    assert lib.rope_fwd(r, 64, 1, x, x, x, -1, x, x, 1, None) == INVALID
    assert lib.rope_fwd(r, 64, 1, x, x, x, 65536, x, x, 1, None) == SHAPE
    assert lib.rope_fwd(r, 64, 1, None, x, x, 1, x, x, 1, None) == INVALID
    assert lib.rope_fwd(r, 64, 1, x, None, x, 1, x, x, 1, None) == INVALID
    assert lib.rope_fwd(r, 64, 1, x, x, ctypes.c_void_p(0x1008), 1, x, x, 1, None) == INVALID
    assert lib.rope_fwd(r, 64, 1, x, x, x, 1, x, None, 1, None) == INVALID
    assert lib.rope_fwd(r, 64, 0, None, None, None, 1, None, None, 1, None) == hs.HSWA_OK
    assert lib.rope_fwd(r, 64, 9, None, None, None, 0, None, None, 0, None) == hs.HSWA_OK
    assert lib.kv_pool_append_rope(None, 0, r, x, 1, x, x, 1, x, x, 1, x, x, x, x, 1, None) == INVALID


def test_modified_scores_are_checked(lib):
    x = ctypes.c_void_p(0x1000)
    for cap in (float("nan"), float("inf"), -1.0, 1e-7, 1e7):
        m = ctypes.byref(hs.ScoreModC(cap, None, None, None))
        assert lib.swa_prefill_mod_fwd(None, 0, x, x, x, x, 1, 1, None, None, 1, m, None, 0, None) == INVALID
        assert lib.full_prefill_mod_fwd(None, 0, x, x, 1, 1, None, x, 1, 1, m, None, 0, None) == INVALID
        assert lib.hybrid_decode_mod_fwd(None, 0, x, x, x, x, 1, 1, x, 1, x, x, 1, 1, m, x, 0, None) == INVALID
        assert b"softcap" in lib.hswa_last_error()
    m = ctypes.byref(hs.ScoreModC(1.0, None, None, None))
    assert lib.swa_prefill_mod_fwd(None, 0, x, x, x, x, 1, 1, None, None, 1, m, None, 0, None) == INVALID
    assert lib.full_prefill_mod_fwd(None, 0, x, x, 1, 1, None, x, 1, 1, None, None, 0, None) == INVALID
    assert lib.hybrid_decode_mod_fwd(None, 0, x, x, x, x, 1, 1, x, 1, x, x, 1, 1, m, x, 0, None) == INVALID
    n = ctypes.c_size_t()
    assert lib.prefill_mod_workspace_size(None, 1, 1, ctypes.byref(n)) == INVALID


def test_python_side_checks():
    with pytest.raises(ValueError):
        hs.RopeDesc([1.0] * 65).c()
    with pytest.raises(ValueError):
        hs.RopeDesc([1.0] * 8, [0] * 7).c()
    with pytest.raises(ValueError):
        hs.ScoreMod(key_begin=torch.zeros(2, 3, dtype=torch.int64)).c((2, 4), 8)
    with pytest.raises(ValueError):
        hs.ScoreMod(dist_slope=torch.zeros(7)).c((2, 3), 8)


def test_outputs_of_a_rotating_commit_have_the_shapes_of_their_inputs():
    class Pool:
        desc = hs.PoolDesc(1, 1, 128, 2, 64, 1, 1)
        handle = None
    rope, q, k = hs.RopeDesc((1.0,) * 8), torch.zeros(1, 3, 4, 64), torch.zeros(1, 3, 2, 64)
    pos, start = torch.zeros(1, 3, dtype=torch.int64), torch.zeros(1, dtype=torch.int64)
    for bad in (dict(q_out=torch.zeros(1, 3, 2, 64)), dict(k_out=torch.zeros(1, 2, 2, 64)),
                dict(k_out=torch.zeros(1, 2, 2, 64), keys_out=False), dict(k_out=torch.zeros(1, 3, 2, 64, device="meta"))):
        with pytest.raises(ValueError, match="shape and device"):
            hs.kv_pool_append_rope(Pool, 1, rope, q, k, k, pos, start, **bad)


def test_plain_attention_equals_torch():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 4, 64), (9, 2, 64), (9, 2, 64)))
    lo, hi = ref.ranges(5, 4, 9, window=3)
    i, j = torch.arange(4, 9)[:, None], torch.arange(9)[None]
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(2, 1).transpose(0, 1), v.repeat_interleave(2, 1).transpose(0, 1),
        attn_mask=(j <= i) & (j > i - 3)).transpose(0, 1)
    assert (ref.attention(q, k, v, lo, hi).o - want).abs().max() < 1e-12
    none = ref.attention(q, k, v, hi, lo)
    assert (none.o == 0).all()


def test_plain_4bit_rows():
    x = torch.tensor([[0.0, 1.5, -1.5, 0.75] * 16, [2.0] * 64]).to(torch.bfloat16)
    codes, step, low = ref.int4_rows(x)
    assert step[0, 0].float() == torch.tensor(0.2).to(torch.bfloat16).float() and low[0, 0] == -1.5
    assert codes[0, :4].tolist() == [7, 15, 0, 11]  # 7.49 -> 7 (step is a little above 0.2), 14.99, 0, 11.2
    assert step[1, 0] == 0 and (ref.int4_values(x)[1] == 2.0).all()
    y = torch.randn(200, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    span = (y.float().amax(-1) - y.float().amin(-1))[:, None].double()
    assert ((ref.int4_values(y) - y.double()).abs() <= span / 30 * (1 + 2.0 ** -7) + span * 2.0 ** -8).all()
    bad = y.clone()
    bad[3, 5], bad[4, 6], bad[5, 0], bad[5, 1] = float("nan"), float("inf"), 3e38, -3e38
    assert torch.isnan(ref.int4_values(bad)[3:6]).all() and not torch.isnan(ref.int4_values(bad)[:3]).any()


def test_plain_rope_against_differences():
    # d/d(theta) of the turned pair is the pair turned by a quarter: checked by central differences
    x = torch.randn(2, 1, 32, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    inv, axis, h = [0.3] * 16, [0] * 16, 1e-6
    at = lambda t: ref.rope(x, torch.full((1, 2), float(t), dtype=torch.float64), inv, axis, False)[0]
    diff = (at(1 + h) - at(1 - h)) / (2 * h * 0.3)
    quarter = at(1 + np.pi / 2 / 0.3)
    assert (diff - quarter).abs().max() < 1e-6
