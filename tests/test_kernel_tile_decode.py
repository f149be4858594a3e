"""The tile decode of the grouped pair kernel, compiled from its own source text for the CPU:
the division by multiplication (Divider), WGrad's decode with the dividers that the launch
fills in, and the forward's walk over an expert's row blocks. Every tile of every expert has
to come exactly once, whatever the number of column panels and row blocks."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_block_scaled_08_b200", "csrc")

SHIM = r"""
#include <cstdint>
#include <algorithm>
using std::max; using std::min;
#define __device__
#define __forceinline__ inline
#define __restrict__
static inline uint32_t __umulhi(uint32_t a, uint32_t b) { return (uint32_t)(((uint64_t)a * b) >> 32); }
"""

MAIN = r"""
extern "C" int64_t divider(int32_t d, const int32_t* n, int64_t count) {
  const Divider by(d);
  for (int64_t i = 0; i < count; ++i)
    if (by(n[i]) != n[i] / d) return i;
  return -1;
}
static GemmParams params(int E, int mblocks, int nblocks, int M, int limit) {
  GemmParams p = {};
  p.M = M; p.mblocks = mblocks; p.nblocks = nblocks; p.experts = E; p.limit = limit;
  p.kblocks = 7; p.bx_step = 0; p.by_step = 1000; p.sb_se = 10;
  p.group = min(8, nblocks);
  return p;
}
// out[t] = expert, row block, panel, slices, first slice
extern "C" void wgrad(int E, int mblocks, int nblocks, int limit, const int* first, int* out) {
  GemmParams p = params(E, mblocks, nblocks, mblocks * kPairM, limit);
  WIRING
  for (int t = 0; t < E * mblocks * nblocks; ++t, out += 5) {
    const GroupTile g = grouped_tile<true>(t, p, nullptr, first);
    out[0] = g.out_row0 / p.M; out[1] = g.row0 / kPairM; out[2] = g.nb; out[3] = g.kblocks; out[4] = g.slice0;
  }
}
extern "C" int row_blocks(int lo, int hi) { return grouped_row_blocks<false>(lo, hi); }
// out[t] = first row, rows of the expert, panel, expert
extern "C" void rows(int E, int nblocks, const int* off, const int* first, int* out) {
  GemmParams p = params(E, 0, nblocks, 0, off[E]);
  for (int t = 0; t < first[E] * nblocks; ++t, out += 5) {
    const GroupTile g = grouped_tile<false>(t, p, off, first);
    out[0] = g.row0; out[1] = g.lo; out[2] = g.hi; out[3] = g.nb; out[4] = g.by / 1000;
  }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    with open(os.path.join(CSRC, "fp8q_gemm.cu")) as f:
        gemm = f.read()
    with open(os.path.join(CSRC, "fp8q_grouped.cuh")) as f:
        grouped = f.read()
    consts = "".join(re.search(r"constexpr int %s = [^;]*;" % n, gemm).group(0) + "\n"
                     for n in ("BM", "BN", "BK", "kPairM"))
    find = re.search(r"__device__ __forceinline__ int group_find\(.*?\n}\n", grouped, re.S).group(0)
    decode = gemm[gemm.index("struct Divider {"):gemm.index("// Wait used while winding down")]
    wiring = re.search(r"const int32_t last = .*?p\.by_last = [^;]*;", gemm, re.S).group(0)
    at = tmp_path_factory.mktemp("decode")
    src, so = at / "decode.cc", at / "decode.so"
    src.write_text(SHIM + consts + find + decode + MAIN.replace("WIRING", wiring))
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", str(src), "-o", str(so)])
    return ctypes.CDLL(str(so))


def ints(a):
    a = np.ascontiguousarray(a, np.int32)
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


@pytest.mark.parametrize("divisors", [range(1, 2049), [2**k + j for k in range(12, 31) for j in (-1, 0, 1)],
                                      [2**31 - 1, 2**31 - 2, 3**19, 10**9 + 7]])
def test_divider_source(lib, divisors):
    rng = np.random.RandomState(12)
    top = 2**31 - 1
    lib.divider.restype = ctypes.c_int64
    for d in divisors:
        near = np.array([1, 2, 3, 1000, top // d], np.int64) * d
        n = np.concatenate([[0, 1, 2, top - 1, top], near - 1, near, near + d - 1,
                            rng.randint(0, top, 300)])
        n, at = ints(n[n <= top])
        assert lib.divider(d, at, ctypes.c_int64(n.size)) == -1, d


@pytest.mark.parametrize("E", [1, 3, 64])
@pytest.mark.parametrize("mblocks", [1, 2, 5])
@pytest.mark.parametrize("nblocks", [1, 2, 7, 8, 9, 11, 16, 20, 40])
def test_wgrad_tiles_come_once(lib, E, mblocks, nblocks):
    rng = np.random.RandomState(E + mblocks + nblocks)
    groups = rng.randint(0, 4, E)
    first = np.concatenate([[0], np.cumsum(groups)])
    limit = int(first[-1]) - (1 if E > 1 else 0)      # the last group may be dropped
    f, at = ints(first)
    out = np.zeros((E * mblocks * nblocks, 5), np.int32)
    lib.wgrad(E, mblocks, nblocks, limit, at, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    want = {(e, m, n) for e in range(E) for m in range(mblocks) for n in range(nblocks)}
    assert {tuple(r[:3]) for r in out} == want
    assert np.array_equal(out[:, 4], np.minimum(first[out[:, 0]], limit))
    assert np.array_equal(out[:, 3], np.minimum(first[out[:, 0] + 1], limit) - out[:, 4])


@pytest.mark.parametrize("counts", [[1], [0, 5, 0, 600, 255, 257, 1, 0], [256, 256, 0, 512], [1] * 40])
@pytest.mark.parametrize("lead", [0, 1, 2, 3, 255])
@pytest.mark.parametrize("nblocks", [1, 8, 9, 21])
def test_row_blocks_cover_every_row_once(lib, counts, lead, nblocks):
    off = np.concatenate([[0], np.cumsum(counts)]) + lead
    E = len(counts)
    first = np.concatenate([[0], np.cumsum([lib.row_blocks(int(off[e]), int(off[e + 1]))
                                            for e in range(E)])])
    (o, oat), (f, fat) = ints(off), ints(first)
    out = np.zeros((int(first[-1]) * nblocks, 5), np.int32)
    lib.rows(E, nblocks, oat, fat, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    seen = np.zeros((int(off[-1]), nblocks), np.int32)
    for row0, lo, hi, nb, e in out:
        assert (lo, hi) == (off[e], off[e + 1]) and row0 % 4 == 0
        seen[max(row0, lo):min(row0 + 256, hi), nb] += 1
    assert np.all(seen[lead:] == 1) and np.all(seen[:lead] == 0)
