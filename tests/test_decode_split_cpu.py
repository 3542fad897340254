"""Without a GPU: how decode calls cut their keys (csrc/decode_split.h)."""
import ctypes
import subprocess

import pytest

from hybrid_sliding_window_swa_b200 import _build


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    # sweep: the first (n_seqs, Hkv, rows, window, max_ctx_len) of a range of sizes that goes to teams of warps with
    # more than one split, or whose splits are not whole pages; 0 when there is none
    (d / "split.cpp").write_text('''
#include <initializer_list>
#include "decode_split.h"
using namespace hswa;
extern "C" int ext_split_c(int n, int h, int w, long long L) { return ext_split(n, h, w, L); }
extern "C" int teams_c(int n, int h, int r, int w, long long L) { return i4_teams(n, h, r, w, L); }
extern "C" long long splits_c(int w, long long L, int split) { return max_splits(w, L, split); }
// the first smaller call (m sequences, up to `length` keys) with more items than the size query has room for
extern "C" int uncovered(int n, int h, long long ctx, int* where) {
  const int64_t room = ext_items_bound(n, h, ctx);
  for (int m = 1; m <= n; ++m)
    for (long long length = 0; length <= ctx; length += length < 1200 ? 61 : 1013)
      for (int w : {0, 128, 513, 4096}) {
        const int64_t items = (int64_t)m * h * max_splits(w, length, ext_split(m, h, w, length));
        if (items > room) { where[0] = m; where[1] = (int)length; where[2] = w; return 1; }
      }
  return 0;
}
extern "C" int sweep(int w, long long L, int* where) {
  for (int n = 1; n <= 700; ++n)
    for (int h = 1; h <= 32; h = h < 8 ? h + 1 : h * 2)
      for (int r : {1, 8, 9, 32}) {
        const int split = ext_split(n, h, w, L);
        const bool bad = split < 256 || split > SPLIT || split % 64 || (i4_teams(n, h, r, w, L) && max_splits(w, L, split) != 1);
        if (bad) { where[0] = n; where[1] = h; where[2] = r; return 1; }
      }
  return 0;
}
''')
    so = str(d / "split.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", _build.CSRC, "-o", so, str(d / "split.cpp")],
                   check=True)
    out = ctypes.CDLL(so)
    out.splits_c.restype = ctypes.c_longlong
    return out


@pytest.mark.parametrize("first,last,step", [(1, 80, 1), (370, 400, 1), (505, 600, 1), (640, 4200, 97)])
def test_teams_of_warps_take_contexts_of_one_split(lib, first, last, step):
    where = (ctypes.c_int * 3)()
    for size in range(first, last, step):
        for window, ctx in ((size, 100000), (size, size), (size, size - 1), (0, size)):
            assert not lib.sweep(window, ctypes.c_longlong(ctx), where), (window, ctx, list(where))


@pytest.mark.parametrize("n_seqs,hkv", [(33, 4), (36, 4), (65, 2), (129, 1), (148, 1)])
def test_a_full_ring_of_513_slots_is_one_split(lib, n_seqs, hkv):
    # 512 cached keys and the token itself
    split = lib.ext_split_c(n_seqs, hkv, 513, ctypes.c_longlong(100000))
    assert split >= 512 and lib.splits_c(513, ctypes.c_longlong(100000), split) == 1


def test_a_ring_counts_the_keys_its_rows_see(lib):
    for w, ctx, keys in ((1, 9, 0), (2, 9, 1), (128, 127, 127), (128, 128, 127), (128, 5000, 127), (0, 5000, 5000)):
        assert lib.splits_c(w, ctypes.c_longlong(ctx), 64) == max(1, -(-keys // 64))


@pytest.mark.parametrize("hkv", [1, 4, 32])
def test_the_size_query_covers_every_smaller_call(lib, hkv):
    where = (ctypes.c_int * 3)()
    for n, ctx in ((1, 600), (1, 262144), (7, 5000), (40, 700), (150, 9000), (300, 70000)):
        assert not lib.uncovered(n, hkv, ctypes.c_longlong(ctx), where), (n, ctx, list(where))
