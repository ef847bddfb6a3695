"""The host side of attention over shared prefixes and of differential attention, without a GPU: every refusal of the C
entry points comes before any CUDA call, the workspace's size follows the bounds, the structures match the header."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from stochastic_sparse_decode_split_gb300 import build as santa_build
from stochastic_sparse_decode_split_gb300 import paged
from test_paged_host import A, BAD, INVALID, UNSUPPORTED, WORKSPACE, params


@pytest.fixture(scope="module")
def lib():
    santa_build.build()
    return santa.library()


def prefix(**kw):
    x = paged.PrefixParams()
    x.n_groups, x.group_offsets, x.prefix_lens, x.max_prefix, x.max_own, x.max_group = 1, None, A, 900, 100, 2
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def shared(lib, p, x, q=A, K=A, V=A, ks=None, vs=None, out=A, lse=None, ws=A, n=1 << 42):
    return lib.santa_shared_attention(ctypes.byref(p), None if x is None else ctypes.byref(x), q, K, V, ks, vs, out, lse, ws, n, None)


def diff(lib, p, x=None, q=A, K=A, V=A, ks=None, vs=None, out=A, lse=None, ws=A, n=1 << 42, none=False, **kw):
    d = paged.DiffParams()
    d.lambda_, d.lambda_stride, d.norm, d.eps, d.gain = A, 0, A, 1e-5, 0.8
    for k, v in kw.items():
        setattr(d, k, v)
    return lib.santa_diff_attention(ctypes.byref(p), None if x is None else ctypes.byref(x), None if none else ctypes.byref(d), q,
                                    K, V, ks, vs, out, lse, ws, n, None)


def sizes(lib, p, x):
    ref = None if x is None else ctypes.byref(x)
    return lib.santa_shared_workspace_size(ctypes.byref(p), ref), lib.santa_diff_workspace_size(ctypes.byref(p), ref)


@pytest.mark.parametrize("kw,status", BAD)
def test_parameters_refused(lib, kw, status):
    p = params(**kw)
    assert shared(lib, p, prefix()) == diff(lib, p) == diff(lib, p, prefix()) == status
    assert sizes(lib, p, prefix()) == (0, 0) and sizes(lib, p, None)[1] == 0


def test_prefixes_refused(lib):
    good = params()
    for kw in (dict(n_groups=0), dict(n_groups=3), dict(max_prefix=0), dict(max_own=0), dict(max_group=0)):
        assert shared(lib, good, prefix(**kw)) == diff(lib, good, prefix(**kw)) == INVALID, kw
        assert sizes(lib, good, prefix(**kw)) == (0, 0)
    for kw in (dict(n_groups=2), dict(prefix_lens=None), dict(prefix_lens=A + 2), dict(group_offsets=A + 2)):
        assert shared(lib, good, prefix(**kw)) == diff(lib, good, prefix(**kw)) == INVALID, kw
    assert shared(lib, good, None) == INVALID and sizes(lib, good, None)[0] == 0
    windowed = params(window=100)
    assert shared(lib, windowed, prefix()) == diff(lib, windowed, prefix()) == UNSUPPORTED
    assert sizes(lib, windowed, prefix()) == (0, 0) and sizes(lib, windowed, None)[1] > 0
    # one that no key is outside of is none
    assert sizes(lib, params(window=1000), prefix()) == sizes(lib, good, prefix())
    # bounds above what there can be are what there can be
    assert sizes(lib, good, prefix(max_prefix=1 << 40, max_own=1 << 40, max_group=1 << 30)) == sizes(lib, good, prefix(
        max_prefix=1000, max_own=1000))


def test_buffers_refused(lib):
    good, e4m3 = params(), params(cache_dtype=3)
    for call, need in ((lambda p, **kw: shared(lib, p, prefix(), **kw), sizes(lib, good, prefix())[0]),
                       (lambda p, **kw: diff(lib, p, prefix(), **kw), sizes(lib, good, prefix())[1]),
                       (lambda p, **kw: diff(lib, p, **kw), sizes(lib, good, None)[1])):
        assert need > 256 and need % 256 == 0
        assert call(good, q=0) == call(good, out=A + 8) == call(good, lse=A + 2) == call(good, K=0) == call(good, V=A + 8) == INVALID
        assert call(params(page_table=0)) == call(params(kv_lens=A + 2)) == call(good, ks=A, vs=A) == call(e4m3) == INVALID
        assert call(good, ws=0) == call(good, ws=A + 16) == call(good, n=need - 1) == WORKSPACE
        assert call(params(dtype=2, cache_dtype=2)) == UNSUPPORTED


def test_differential_heads_refused(lib):
    assert diff(lib, params(), none=True) == INVALID
    assert diff(lib, params(n_q_heads=15, n_kv_heads=3)) == INVALID and sizes(lib, params(n_q_heads=15, n_kv_heads=3), None)[1] == 0
    for kw in (dict(lambda_=0), dict(lambda_=A + 2), dict(lambda_stride=15), dict(lambda_stride=-16), dict(norm=A + 8), dict(eps=-1.0),
               dict(eps=math.nan), dict(eps=math.inf), dict(gain=math.nan), dict(gain=math.inf)):
        assert diff(lib, params(), **kw) == INVALID, kw
    assert diff(lib, params(), n=0, norm=None, eps=math.nan) == WORKSPACE   # eps is the norm's


def test_structures_and_constants_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "santa.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %d\\n", sizeof(santa_prefix_t), offsetof(santa_prefix_t, max_group),'
                   ' sizeof(santa_diff_t), offsetof(santa_diff_t, gain), SANTA_CACHE_DEVERR_PREFIX);\nreturn 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(santa_build.ROOT, "include"), str(src), "-o",
                    str(tmp_path / "sizes")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(paged.PrefixParams), paged.PrefixParams.max_group.offset, ctypes.sizeof(paged.DiffParams),
                   paged.DiffParams.gain.offset, santa.CACHE_DEVERR_PREFIX]


def test_the_packed_diff_parameters_are_the_structure():
    values = dict(lambda_=1 << 40, lambda_stride=16, norm=3 << 40, eps=0.125, gain=0.5)
    packed = paged._DIFF.pack(*values.values())
    back = paged.DiffParams.from_buffer_copy(packed + bytes(ctypes.sizeof(paged.DiffParams) - len(packed)))
    assert all(getattr(back, k) == v for k, v in values.items())


def test_weights_from_their_vectors():
    v = [torch.tensor([[0.1 * i, 0.2], [0.3, -0.1 * i]], dtype=torch.bfloat16) for i in range(1, 5)]
    got = santa.diff_weights(*v, init=0.2)
    want = [math.exp(sum(float(a) * float(b) for a, b in zip(v[0][h], v[1][h]))) -
            math.exp(sum(float(a) * float(b) for a, b in zip(v[2][h], v[3][h]))) + 0.2 for h in range(2)]
    assert got.dtype == torch.float32 and got.shape == (2,)
    assert all(abs(float(g) - w) < 2.0 ** -20 for g, w in zip(got, want))   # a few roundings of values near 1
