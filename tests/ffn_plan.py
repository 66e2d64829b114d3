"""The feed-forward block's choice of kernels (csrc/ss_ffn_plan.h), compiled by
the host's C++ compiler, and the sizes that the tests reach its forms with."""
from __future__ import annotations

import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sampled_softmax_output_gb300", "csrc")
SMS = 152

# 17 to 32 tokens (the tiles of 32 tokens, by themselves in that range), and the
# forms that the sizes of test_ffn_gpu.py do not reach
FORM_SIZES = [(17, 72, 136), (24, 264, 520), (31, 520, 1032), (32, 1096, 392), (17, 1096, 2056),
              (32, 2048, 5504), (2, 200, 208), (1772, 1288, 8), (608, 976, 4832), (902, 8, 8),
              (33, 8, 336), (971, 8, 72), (33, 8, 7704), (1273, 8512, 392), (1255, 15552, 144),
              (3435, 272, 664), (885, 264, 4248), (3, 9856, 648), (24, 9856, 712),
              (19545, 14608, 24), (111, 12080, 7480), (88, 9408, 15016)]
# gate/up and dA on CTA pairs, stored from registers and through shared memory,
# with tiles of 256 and 192 columns: for every activation
ACT_SIZES = [(2187, 240, 792), (2574, 248, 1176), (1944, 968, 528), (2080, 968, 1552)]

SOURCE = r"""
#include "ss_ffn_plan.h"
using namespace ss;
extern "C" void forward(long T, long D, long F, int sms, int* o) {
  const ForwardPlan p = forward_plan(T, D, F, sms);
  const int v[] = {p.up_on_pairs, p.up_pair.bn, p.up.bn, p.up.cluster,
                   p.down_on_pairs, p.down.bn, p.down.cluster};
  for (int x : v) *o++ = x;
}
extern "C" void backward(long T, long D, long F, int sms, int* o) {
  const BackwardPlan p = backward_plan(T, D, F, sms);
  const int v[] = {p.act_on_pairs, p.act_pair.bn, p.act.bn, p.act.cluster, p.grads_together,
                   p.x_on_pairs, p.x.bn, p.x.cluster, p.w_on_pairs, p.w.bn, p.w.cluster};
  for (int x : v) *o++ = x;
}
// the units of all pairs, one pair after the other; ends[p]: where pair p's end
extern "C" long deal(int n_a, long kb_a, int n_b, long kb_b, int pairs, int* units, int* ends) {
  const UnitDeal d = deal_units(n_a, kb_a, n_b, kb_b);
  int n = 0;
  for (int p = 0; p < pairs; ++p) {
    const PairShare s = share_of(d, p, pairs);
    for (int k = 0; k < s.count(); ++k) units[n++] = s.unit(k);
    ends[p] = n;
  }
  return busiest_pair(d, std::max(kb_a, kb_b), std::min(kb_a, kb_b), pairs);
}
"""


def compile_plan(folder: str) -> ctypes.CDLL:
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "libplan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                    "-I" + CSRC, src, "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    for f in (L.forward, L.backward):
        f.restype = None
        f.argtypes = [ctypes.c_long] * 3 + [ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.deal.restype = ctypes.c_long
    L.deal.argtypes = [ctypes.c_int, ctypes.c_long, ctypes.c_int, ctypes.c_long, ctypes.c_int,
                       ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
    return L


def deal(L: ctypes.CDLL, n_a: int, kb_a: int, n_b: int, kb_b: int, pairs: int):
    """(units of each pair, the busiest pair's k-blocks)."""
    units, ends = (ctypes.c_int * (n_a + n_b))(), (ctypes.c_int * pairs)()
    most = L.deal(n_a, kb_a, n_b, kb_b, pairs, units, ends)
    out, at = [], 0
    for p in range(pairs):
        out.append(list(units[at:ends[p]]))
        at = ends[p]
    return out, most


def forms(L: ctypes.CDLL, T: int, D: int, F: int) -> set:
    """What one forward and one backward of this size run, with G, U and A kept
    and every tensor on a 32-byte boundary."""
    o = (ctypes.c_int * 11)()
    L.forward(T, D, F, SMS, o)
    up = ("up pair", "registers" if F % 16 == 0 else "staged", o[1]) if o[0] else (
        "up split", o[2], o[3])
    down = ("down pair",) if o[4] else ("down split", o[5], o[6])
    L.backward(T, D, F, SMS, o)
    act = ("act pair", "registers" if D > 960 else "staged", o[1]) if o[0] else (
        "act split", o[2], o[3])
    if o[4]:
        return {up, down, act, ("grads pair",)}
    x = ("x pair",) if o[5] else ("x split", o[6], o[7])
    w = ("w pair",) if o[8] else ("w split", o[9], o[10])
    return {up, down, act, x, w}
