"""The kernels that the products of 8-bit integers choose between, as csrc/ffn_choice.h chooses them (compiled for the host)."""
import ctypes
import os
import subprocess

from ffn_variants import CSRC

SOURCE = """
#include "ffn_choice.h"
using namespace dyra;
typedef long long ll;
extern "C" {
int narrow(int gated, ll M, ll N) { return takes_narrow(1, gated, M, N); }
int few(int gated, ll M, ll N, ll bytes) { const FewTokens f = few_tokens(gated, M, N, bytes); return f.slabs * 4 + f.blocks; }
int tile(int gated, ll M, ll N, ll bytes) { return pick_tile(1, gated, M, N, bytes); }
int split(int gated, ll M, ll N, ll bytes) { const Split s = pick_split(gated, M, N, bytes); return s.parts * 16 + s.tile; }
ll split_size(int gated, ll M, ll N, int parts) { return split_bytes(gated, M, N, parts); }
int skinny_tokens() { return kSkinnyTokens; }
}
"""


class Choice:
    def __init__(self, folder):
        src, so = os.path.join(folder, "choice.cpp"), os.path.join(folder, "choice.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", so, src], check=True)
        self.lib = ctypes.CDLL(so)
        i, ll = ctypes.c_int, ctypes.c_longlong
        for name, args in dict(narrow=[i, ll, ll], few=[i, ll, ll, ll], tile=[i, ll, ll, ll], split=[i, ll, ll, ll],
                               split_size=[i, ll, ll, i], skinny_tokens=[]).items():
            getattr(self.lib, name).argtypes = args
        self.lib.split_size.restype = ll

    def whole(self, gated, N, c1, c2):
        """The kernel of a call without a workspace."""
        if N <= self.lib.skinny_tokens():
            slabs, blocks = divmod(self.lib.few(gated, N, c2, c1), 4)
            return ("registers", slabs, blocks) if slabs else ("ring", (N + 15) // 16)
        if self.lib.narrow(gated, N, c2):
            return ("narrow", 2 if gated or c2 > 16 else 1)
        return ("tile", self.lib.tile(gated, N, c2, c1))

    def parts(self, gated, N, c1, c2):
        """(parts of K, tile) of a call with a workspace; parts 1: as without."""
        if self.whole(gated, N, c1, c2)[0] != "tile":
            return 1, None
        parts, tile = divmod(self.lib.split(gated, N, c2, c1), 16)
        return parts, tile
