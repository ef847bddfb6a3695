"""The kernels that a call of attention over the paged cache goes to, asked of the library's own plans (on the host: tests
that are meant for one kernel say so, and a border that moves past them is noticed)."""
import functools
import os
import subprocess
import tempfile

from stochastic_sparse_decode_split_gb300 import build as santa_build

HERE = os.path.dirname(os.path.abspath(__file__))


@functools.lru_cache(maxsize=None)
def _program():
    exe = os.path.join(tempfile.mkdtemp(), "join_route")
    subprocess.run([santa_build.nvcc(), "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", santa_build.CSRC, "-o", exe,
                    os.path.join(HERE, "join_route.cu")], check=True, capture_output=True)
    return exe


def route(kv, n, H, Hkv, D, e4m3=False, page=16, diff=False, causal=True, window=0, prefix=None, first=None, pad=0):
    """``Batch(kv, n, ...)``'s call, or with prefix and first that of ``Shared(prefix, first, kv, n, ...)``'s (whose kv are
    the keys behind the prefixes): a list such as ["prefix:chunk", "own:tokens"]."""
    groups, most, own, size = 0, 1, 1, 1
    nk = max(max(kv), 1)
    if prefix is not None:
        groups, most, own = len(prefix), max(max(prefix), 1), max(max(kv), 1)
        size = max(b - a for a, b in zip(first, first[1:]))
        nk = max(p + max(kv[a:b], default=0) for p, a, b in zip(prefix, first, first[1:]))
    line = [int(diff), int(e4m3), D, H, Hkv, page, int(causal), window, nk, max(n), sum(n) + pad, len(kv), groups, most, own, size]
    out = subprocess.run([_program()], input=" ".join(str(x) for x in line), capture_output=True, text=True, check=True).stdout
    status, *kernels = out.split()
    assert status == "0", (status, line)
    return kernels
