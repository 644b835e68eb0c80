"""Which kernels a dense block's products run in, asked of the library's own rules
(csrc/ffn_plan.h, plain C++) without a GPU."""
import ctypes
import functools
import os
import subprocess
import tempfile

from mixture_experts_layer_deterministic_amd import build

BIG, TALL, WIDE, SMALL, SHARES = range(5)  # 256 x 256, 256 x 128, 128 x 256, 128 x 128, shares of K
FEW = 5  # the kernels for a handful of tokens
# ffn.hip's products: rows x columns, steps of K
_SOURCE = """
#include "ffn_plan.h"
using namespace moe::ffn;
extern "C" void plan(int T, int d, int I, int* out) {
  const int few = 5;
  out[0] = few_gate_up(T, d, I) ? few : plan_of({T, 2LL * I, d / 64}).shape;
  out[1] = few_down(T, d, I) ? few : plan_of({T, d, I / 64}).shape;
  const PairPlan a = plan_of_pair({T, I, d / 64}, {d, I, (T + 63) / 64});
  const PairPlan b = plan_of_pair({T, d, 2 * I / 64}, {2LL * I, d, (T + 63) / 64});
  out[2] = a.rows.shape;
  out[3] = a.dw.shape;
  out[4] = b.rows.shape;
  out[5] = b.dw.shape;
}
"""
PRODUCTS = ("gate_up", "down", "dh", "dw2", "dx", "dw1")


@functools.lru_cache(maxsize=1)
def _lib():
    with tempfile.TemporaryDirectory() as tmp:
        src, so = os.path.join(tmp, "plan.cpp"), os.path.join(tmp, "plan.so")
        with open(src, "w") as f:
            f.write(_SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC",
                        f"-I{build.CSRC}", src, "-o", so], check=True)
        return ctypes.CDLL(so)


def plan(T, d, I):
    """{product: the kernel it takes} of a block of T tokens."""
    out = (ctypes.c_int * 6)()
    _lib().plan(T, d, I, out)
    return dict(zip(PRODUCTS, out))
