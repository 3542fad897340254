"""GPU: decode over 4-bit rings whose full window is as long as the longest context that is not split."""
import pytest

import operators_ref as ref
from test_gpu_int4 import decode_case

pytestmark = pytest.mark.gpu


# 512 cached keys and the token itself; sequences x KV heads between one and one and a half of what the CTAs hold
@pytest.mark.parametrize("W", [512, 513, 514])
@pytest.mark.parametrize("n,n_qt,hq,hkv,d", [(33, 1, 16, 4, 64), (36, 2, 8, 4, 128), (65, 1, 4, 2, 64), (131, 4, 2, 1, 64),
                                             (36, 3, 16, 4, 64)])
def test_full_rings_of_about_512_slots(W, n, n_qt, hq, hkv, d):
    lens = [W + 17 * i for i in range(n - 3)] + [W - 1, W, 40]
    o, refs = decode_case(41, lens, n_qt, hq, hkv, d, W)
    for b, r in enumerate(refs):
        ref.check(o[b], r, f"W={W} seq {b} L={lens[b]}")
