"""The products' schedule (csrc/hc_plan.h) compiled for the host, and which of
its plans the products of a call take."""
from __future__ import annotations

import ctypes
import math
import os
import random
import subprocess

from hyper_connection_rank_amd import build

SOURCE = """
#include "hc_plan.h"
// [n][9]: dtype, M, N, K, p_trans, dual, segments, batch, aligned -> [n][8]: tile rows and columns, whole and split
// tiles, parts of a split one, contraction step, scratch that is asked for, scratch that the plan uses
extern "C" void plans(const long long* q, long long* r, long long n) {
  for (long long i = 0; i < n; ++i, q += 9, r += 8) {
    const hc::Plan p = hc::make_plan((int)q[0], q[1], q[2], q[3], q[4], q[5], (int)q[6], (int)q[7], q[8]);
    r[0] = p.shape->bm; r[1] = p.shape->bn; r[2] = p.whole; r[3] = p.rest; r[4] = p.splits; r[5] = p.shape->bk;
    r[6] = (long long)hc::product_scratch((int)q[0], q[1], q[2], q[3], q[4], q[5], (int)q[6], (int)q[7]);
    r[7] = p.rest * p.splits * hc::part_size(*p.shape, q[1]) * 4;
  }
}
"""


def compile_plan(folder):
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", lib], check=True)
    return ctypes.CDLL(lib)


CODES = {"f32": 1, "f16": 10, "bf16": 16}


def products(rows, k, n, dtype):
    """{product: query} of linear, glu and their gradients on contiguous 16-byte aligned tensors."""
    a16 = 4 if dtype == "f32" else 8
    code = CODES[dtype]
    # aligned: both operands' rows are whole 16-byte chunks; dx reads dz and the weight, whose rows are both n long
    aln, dx = int(k % a16 == 0 and n % a16 == 0), int(n % a16 == 0)
    return {"linear": (code, rows, n, k, 0, 0, 1, 1, aln), "glu": (code, rows, n, k, 0, 1, 1, 1, aln),
            "dx": (code, rows, k, n, 0, 0, 1, 1, dx), "dx of glu": (code, rows, k, n, 0, 0, 2, 1, dx),
            "dw": (code, k, n, rows, 1, 0, 1, 1, aln), "dw of glu": (code, k, n, rows, 1, 0, 1, 2, aln)}


def ask(lib, queries):
    q = (ctypes.c_longlong * (9 * len(queries)))(*[v for t in queries for v in t])
    r = (ctypes.c_longlong * (8 * len(queries)))()
    lib.plans(q, r, ctypes.c_longlong(len(queries)))
    return [tuple(r[8 * i:8 * i + 8]) for i in range(len(queries))]


def kind(plan):
    return "whole" if plan[3] == 0 else "split" if plan[2] == 0 else "mixed"


def keys(lib, calls):
    """{(bits of T, product, rows x columns of a tile, aligned, whole/split/mixed)} that the calls
    (rows, in, out, dtype) take, with how often."""
    names, queries = [], []
    for rows, k, n, dtype in calls:
        for name, q in products(rows, k, n, dtype).items():
            names.append((32 if dtype == "f32" else 16, name, q[8]))
            queries.append(q)
    found = {}
    for (b, name, aln), p in zip(names, ask(lib, queries)):
        key = (b, name, f"{p[0]}x{p[1]}", "aligned" if aln else "unaligned", kind(p))
        found[key] = found.get(key, 0) + 1
    return found


def sample(count, seed=7):
    """Calls of the operators' range: rows 1 to 8192 and widths 64 to 12288 over their logarithms, a third of
    the widths odd, at most 2^37.6 multiplications."""
    rng = random.Random(seed)

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width():
        v = log_int(64, 12288)
        return v | 1 if rng.random() < 1 / 3 else max(8, v & ~7)

    calls = []
    for _ in range(count):
        dtype = rng.choice(["bf16", "f32"])
        k, n = width(), width()
        most = 8192 * 2560 * 10240 // (8 if dtype == "f32" else 1)
        calls.append((max(1, min(log_int(1, 8192), most // (k * n))), k, n, dtype))
    return calls
