"""The attention calls' launch plans (csrc/attention_plan.h) built for the host, and the shapes whose kernel the tests rely
on.  Tests only."""
import ctypes
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
sys.path.insert(0, ROOT)


class Forward:
    def __init__(self, few, pack, splits, blocks, threads, join_blocks):
        self.few, self.pack, self.splits, self.blocks, self.threads, self.join_blocks = few, pack, splits, blocks, threads, join_blocks


class Backward:
    def __init__(self, pack, parts, far_blocks, dq_blocks, dk_blocks, join_blocks):
        self.pack, self.parts, self.far_blocks = pack, parts, far_blocks
        self.dq_blocks, self.dk_blocks, self.join_blocks = dq_blocks, dk_blocks, join_blocks


class Plans:
    def __init__(self, folder):
        lib = os.path.join(str(folder), "attention_plan.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wno-attributes", "-D__HIP_PLATFORM_AMD__", "-I",
                        "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(ROOT, "blockwise_fp8_gemm_act_amd", "csrc"),
                        os.path.join(HERE, "csrc", "attention_plan_probe.cpp"), "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)

    def _ask(self, call, shape):
        out = (ctypes.c_int64 * 6)()
        call(ctypes.byref(shape), out)
        return list(out)

    def forward(self, shape):
        return Forward(*self._ask(self.lib.forward, shape))

    def backward(self, shape):
        return Backward(*self._ask(self.lib.backward, shape))

    def rope(self, tokens, heads, head_dim):
        out = (ctypes.c_int64 * 3)()
        self.lib.rope(ctypes.c_int64(tokens), ctypes.c_int64(heads), ctypes.c_int64(head_dim), out)
        return list(out)


def shape(qh, kh, hd, q_tokens, k_tokens, sequences=1, window=0, sinks=0, max_k=0):
    import blockwise_fp8_gemm_act_amd as puro
    if window >= k_tokens:
        window = 0
    s = min(sinks, k_tokens) if window else 0
    return puro.AttentionShape(q_tokens, k_tokens, sequences, qh, kh, hd, qh * hd, kh * hd, kh * hd, qh * hd, qh * hd, kh * hd,
                               kh * hd, max_k, window, s, hd ** -0.5)


# Calls that take the kernel for many queries: (query heads, key heads, head_dim, heads of a workgroup, queries of each
# sequence, keys, window, first keys)
MANY = [(16, 8, 128, 2, [2100], [2100], 0, 0), (16, 8, 128, 2, [2100], [2100], 300, 5), (16, 8, 128, 2, [1301, 700], [1301, 1400], 0, 0),
        (24, 24, 128, 1, [2049], [2049], 0, 0), (24, 24, 128, 1, [1999], [1999], 130, 0),
        (24, 8, 128, 1, [1100, 0, 900], [1100, 70, 900], 200, 70), (16, 4, 128, 4, [2111], [2111], 0, 0), (16, 4, 128, 4, [2111], [2111], 64, 1),
        (16, 8, 128, 2, [1500, 900], [1000, 0], 0, 0), (16, 4, 64, 4, [2000, 700], [1400, 9], 300, 2),
        (32, 32, 64, 1, [2100], [2100], 0, 0), (16, 4, 64, 4, [1027, 1500], [1027, 1500], 500, 3), (32, 16, 64, 2, [2300], [2300], 0, 0)]

# The same over a cache with room left: (query heads, key heads, head_dim, heads of a workgroup, queries, keys in use, room,
# window, first keys)
MANY_CACHED = [(16, 8, 128, 2, [700, 800, 900], [900, 800, 1000], 1300, 0, 0), (16, 8, 128, 2, [700, 800, 900], [900, 800, 1000], 1300, 100, 3),
               (16, 4, 64, 4, [1000, 1200], [1100, 1201], 1500, 64, 0), (32, 32, 64, 1, [512, 700, 400], [600, 700, 401], 750, 0, 0)]

# Single tokens and few: (query heads, key heads, head_dim, queries, sequences, keys of each)
FEW = [(16, 8, 128, 1, 1, 4000), (16, 8, 128, 1, 64, 500), (16, 4, 64, 1, 1, 4000), (16, 4, 64, 3, 16, 700)]


if __name__ == "__main__":
    with tempfile.TemporaryDirectory() as d:
        p = Plans(d)
        for qh, kh, hd, _, ql, kl, w, s in MANY:
            print(vars(p.forward(shape(qh, kh, hd, sum(ql), sum(kl), len(ql), w, s))))
        for qh, kh, hd, _, ql, kl, room, w, s in MANY_CACHED:
            print(vars(p.forward(shape(qh, kh, hd, sum(ql), room * len(ql), len(ql), w, s, max(kl)))))
        for qh, kh, hd, q, n, kl in FEW:
            print(vars(p.forward(shape(qh, kh, hd, q * n, kl * n, n))))
