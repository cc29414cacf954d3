"""The rule that picks a kernel shape for products with packed 4-bit weights,
compiled from its own header, and sizes that reach every shape."""
import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "matvec_shape.hpp"
extern "C" void shape(int routed, int64_t rows, int N, int K, int group, int* out) {
  const moe::MatvecShape c = moe::matvec_shape(routed != 0, rows, N, K, group);
  out[0] = c.chunk, out[1] = c.rows, out[2] = c.share, out[3] = c.splits, out[4] = c.flush;
}
"""


def compile_rule(folder):
    """shape(routed, rows, N, K, group) -> (chunk, rows, share, splits, flush)."""
    src, lib = os.path.join(folder, "shape.cpp"), os.path.join(folder, "libshape.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "mixture_experts_ffn_align_amd", "csrc"), src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).shape
    fn.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]

    def shape(routed, rows, N, K, group):
        out = (ctypes.c_int * 5)()
        fn(int(routed), rows, N, K, group, out)
        return tuple(out)

    return shape


# What the kernel is built for: chunk, rows, share, each with scalings after 1, 2 and 4 products, and the
# splits each is started with.
BUILT = {(256, 4, 1): {2}, (128, 4, 1): {2, 4, 8}, (128, 16, 1): {4}, (128, 16, 2): {2, 4}, (128, 16, 4): {2},
         (128, 32, 2): {2, 4}, (128, 32, 4): {1, 2}, (128, 48, 2): {2, 4}, (128, 48, 4): {1, 2},
         (128, 64, 2): {2, 4}, (128, 64, 4): {1, 2}}

# Sums of one batch of scales and of several, with a tail in a chunk or in a split, or whole (then neighbouring
# tiles start at other places); groups scaled after 1, 2 and 4 products, some of odd multiples.
SHORT = [(544, 32), (672, 96), (1024, 32), (576, 64), (960, 192), (2048, 64), (640, 128), (768, 384), (2048, 128)]
LONG = [(4128, 32), (4160, 160), (8192, 32), (4160, 64), (4224, 192), (8192, 64), (4224, 128), (6144, 256), (8192, 128)]
DEEP = [(8224, 32), (8256, 64), (8320, 128)]


def cases():
    """(M, k, N, K, group), k = 0 for one matrix; N is odd, its last tile and its last workgroup end inside."""
    for K, group in SHORT:
        yield from ((3, 0, 101, K, group), (2, 0, 16389, K, group), (1, 0, 32773, K, group))
        yield from ((5, 0, 8197, K, group), (16, 0, 8197, K, group), (9, 0, 101, K, group))
        yield from ((16, 0, 16389, K, group), (7, 0, 16389, K, group))
        for M in (17, 48, 64):
            yield from ((M, 0, 101, K, group), (M, 0, 16389, K, group), (M, 0, 32773, K, group))
        yield from ((130, 0, 16389, K, group), (3, 2, 2741, K, group), (2, 3, 101, K, group), (1, 8, 2053, K, group))
    for K, group in LONG:
        yield from ((1, 0, 101, K, group), (4, 0, 4101, K, group), (1, 0, 16389, K, group), (4, 0, 16389, K, group))
        yield from ((2, 2, 101, K, group), (1, 8, 2053, K, group), (32, 0, 101, K, group), (33, 0, 101, K, group))
        yield from ((63, 0, 101, K, group), (20, 0, 16389, K, group), (16, 0, 16389, K, group))
    for K, group in DEEP:
        yield from ((12, 0, 8197, K, group), (1, 0, 16389, K, group), (1, 0, 101, K, group))


CASES = list(dict.fromkeys(cases()))
