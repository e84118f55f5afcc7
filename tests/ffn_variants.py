"""The kernels that the feed-forward calls choose between, as csrc/ffn_choice.h chooses them (compiled for the host)."""
import ctypes
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_rank_matmul_amd", "csrc")
SOURCE = """
#include "ffn_choice.h"
using namespace dyra;
typedef long long ll;
extern "C" {
int narrow(int elem, int gated, ll M, ll N) { return takes_narrow(elem, gated, M, N); }
int few(int gated, ll M, ll N, ll bytes) { const FewTokens f = few_tokens(gated, M, N, bytes); return f.slabs * 4 + f.blocks; }
int tile(int elem, int gated, ll M, ll N, ll bytes) { return pick_tile(elem, gated, M, N, bytes); }
int up(ll bytes) { return up_slabs(bytes); }
int down(int T, int k, int E, ll c) { const Down d = down_kernel(T, k, E, c); return d.rows * 32 + d.slot; }
int splits(int elem, int T, int k, int E, ll c, ll f, int parts, int rest) {
    return down_splits(down_kernel(T, k, E, c), elem, T, k, E, c, f, parts, rest);
}
int skinny_tokens() { return kSkinnyTokens; }
}
"""
ELEM = {"bf16": 2, "f32": 4}


class Choice:
    def __init__(self, folder):
        src, so = os.path.join(folder, "choice.cpp"), os.path.join(folder, "choice.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", so, src], check=True)
        self.lib = ctypes.CDLL(so)
        i, ll = ctypes.c_int, ctypes.c_longlong
        for name, args in dict(narrow=[i, i, ll, ll], few=[i, ll, ll, ll], tile=[i, i, ll, ll, ll], up=[ll], down=[i, i, i, ll],
                               splits=[i, i, i, i, ll, ll, i, i], skinny_tokens=[]).items():
            getattr(self.lib, name).argtypes = args

    def linear(self, gated, dtype, N, c1, c2):
        """The kernel of dyra_linear or dyra_gated."""
        elem = ELEM[dtype]
        if N <= self.lib.skinny_tokens():
            slabs, blocks = divmod(self.lib.few(gated, N, c2, c1 * elem), 4)
            return ("registers", slabs, blocks) if slabs else ("ring", (N + 15) // 16)
        if self.lib.narrow(elem, gated, N, c2):
            return ("narrow", 2 if gated or c2 > 16 else 1)
        return ("tile", self.lib.tile(elem, gated, N, c2, c1 * elem))

    def moe_up(self, dtype, c):
        return self.lib.up(c * ELEM[dtype])

    def moe_down(self, dtype, T, k, E, c, f, parts, rest):
        """(features, pairs of a slot, H in two parts, shared slabs)."""
        rows, slot = divmod(self.lib.down(T, k, E, c), 32)
        return rows, slot, rest, self.lib.splits(ELEM[dtype], T, k, E, c, f, parts, rest) > 1
