"""The rules by which the gated block's and the orthogonalised update's products choose their kernels, compiled for the
host from the headers that the launches use."""
import ctypes
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sharded_mixed_precision_rank_amd", "csrc")
SOURCE = """
#include "zs_glu_choice.h"
#include "zs_muon_choice.h"
extern "C" int glu(int op, int64_t M, int64_t N, int64_t K, int direct) {
  return (int)zs::glu::choose((zs::GluOp)op, M, N, K, direct != 0);
}
extern "C" int ns(int64_t m, int64_t n, int64_t k, int64_t batch, int triangle) {
  const zs::ns::Choice c = zs::ns::choose(m, n, k, batch, triangle != 0);
  return (int)c.tile * 100 + c.splits;
}
extern "C" int64_t small_side() { return zs::ns::kSmallSide; }
extern "C" int64_t slab_side() { return zs::ns::kSlabSide; }
"""
GLU = ("any", "through", "few", "split", "64x32", "32", "64", "64x128", "128", "128 near", "192", "256")
OPS = ("forward", "input", "weight")
SIDES = (32, 64, 128, 192, 256)


class Choices:
    def __init__(self, to):
        out = os.path.join(to, "choices.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-x", "c++", "-", "-o", out], input=SOURCE, text=True,
                       check=True)
        self.lib = ctypes.CDLL(out)
        i64 = ctypes.c_int64
        self.lib.glu.argtypes = [ctypes.c_int, i64, i64, i64, ctypes.c_int]
        self.lib.ns.argtypes = [i64, i64, i64, i64, ctypes.c_int]
        self.lib.small_side.restype = self.lib.slab_side.restype = i64

    def glu(self, op, M, N, K, direct=True):
        """The kernel of M x N outputs over a summed axis of K; `direct`: rows on 4-byte boundaries."""
        return GLU[self.lib.glu(OPS.index(op), M, N, K, int(direct))]

    def orthogonalize(self, rows, cols, batch=1):
        """{product: (tile's side, splits)} of a matrix of a stack: none where one workgroup does all of it."""
        if max(rows, cols) <= self.lib.small_side():
            return {}
        m, n = (-(-v // 32) * 32 for v in sorted((rows, cols)))
        products = {"gram": (m, m, n, batch, 1), "poly": (m, m, m, batch, 1), "apply": (m, n, m, batch, 0)}
        if m <= self.lib.slab_side():
            del products["poly"], products["apply"]
        return {k: (SIDES[c // 100], c % 100) for k, c in ((k, self.lib.ns(*v)) for k, v in products.items())}
