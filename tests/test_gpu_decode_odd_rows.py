"""GPU: decode with an odd number of query rows per KV head over several splits (each split's partial
result must start on a 16-byte boundary)."""
import pytest

from hswa_testlib import compare
from test_gpu_decode import run_decode_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_qt,hq,hkv,d", [(1, 1, 1, 64), (1, 6, 2, 128), (3, 15, 3, 128)])
def test_odd_rows_over_several_splits(n_qt, hq, hkv, d):
    got, ref, _ = run_decode_case(301, [8193, 20000, 100], n_qt, hq, hkv, d, 128, "full")
    compare(got, ref, f"{n_qt * hq // hkv} rows")
