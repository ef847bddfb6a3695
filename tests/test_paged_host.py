"""The paged cache's host side, without a GPU: every refusal of the C entry
points comes before any CUDA call, the binding refuses what it can see, the
structures match the header, and the rotation table is what it says."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import stochastic_sparse_decode_split_gb300 as santa
from stochastic_sparse_decode_split_gb300 import build as santa_build
from stochastic_sparse_decode_split_gb300 import paged

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 1 << 12   # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    santa_build.build()
    return santa.library()


def params(**kw):
    p = paged.PagedParams()
    p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim, p.dtype, p.cache_dtype = 2, 32, 8, 128, 0, 0
    p.page_size, p.n_pages, p.page_table, p.max_pages, p.kv_lens, p.nk = 16, 512, A, 64, A, 1000
    p.q_offsets, p.max_q, p.total_q, p.causal, p.window, p.scale = None, 3, 6, 1, 0, 0.0
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD = [
    (dict(batch=0), INVALID), (dict(batch=65536, q_offsets=A), INVALID), (dict(n_kv_heads=5), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=72), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(cache_dtype=1), UNSUPPORTED),
    (dict(cache_dtype=4), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(n_pages=1 << 27), INVALID),
    (dict(max_pages=62), INVALID), (dict(max_pages=0), INVALID), (dict(nk=0), INVALID),
    (dict(nk=(1 << 21) + 1, max_pages=1 << 20), INVALID), (dict(max_q=0), INVALID), (dict(max_q=7), INVALID),
    (dict(total_q=5), INVALID), (dict(total_q=0), INVALID), (dict(total_q=1 << 31, q_offsets=A), INVALID),
    (dict(causal=2), INVALID), (dict(window=-1), INVALID), (dict(causal=0, window=4), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
]


def attention(lib, p, q=A, K=A, V=A, ks=None, vs=None, out=A, lse=None, ws=A, n=1 << 40):
    return lib.santa_paged_attention(ctypes.byref(p), q, K, V, ks, vs, out, lse, ws, n, None)


def read(lib, p, K=A, V=A, ks=None, vs=None, off=A, rows=2000, ko=A, vo=A, ws=A, n=256):
    return lib.santa_kv_read(ctypes.byref(p), K, V, ks, vs, off, rows, ko, vo, ws, n, None)


def append(lib, p, K=A, V=A, ks=None, vs=None, ws=A, n=256, **kw):
    a = paged.AppendParams()
    a.q, a.k, a.v, a.q_stride, a.k_stride, a.v_stride, a.q_out = A, A, A, 4096, 1024, 1024, 2 * A
    a.eps, a.rope, a.rope_positions, a.rotated = 1e-6, A, 1000, 128
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.santa_kv_append(ctypes.byref(p), ctypes.byref(a), K, V, ks, vs, ws, n, None)


@pytest.mark.parametrize("kw,status", BAD)
def test_parameters_refused_by_all_three(lib, kw, status):
    p = params(**kw)
    assert attention(lib, p) == read(lib, p) == append(lib, p) == status
    assert lib.santa_paged_workspace_size(ctypes.byref(p)) == 0
    assert lib.santa_paged_workspace_size(None) == 0


def test_buffers_refused(lib):
    good, e4m3 = params(), params(cache_dtype=3)
    need = lib.santa_paged_workspace_size(ctypes.byref(good))
    assert need >= 256 and need % 256 == 0
    for call in (attention, read, append):
        assert call(lib, good, K=0) == call(lib, good, V=A + 8) == INVALID
        assert call(lib, params(page_table=0)) == call(lib, params(kv_lens=A + 2)) == INVALID
        assert call(lib, good, ks=A, vs=A) == INVALID                   # scales without an e4m3 cache
        assert call(lib, e4m3) == call(lib, e4m3, ks=A) == call(lib, e4m3, ks=A + 4, vs=A) == INVALID
        assert call(lib, good, ws=0) == call(lib, good, ws=A + 16) == call(lib, good, n=0) == WORKSPACE
    assert attention(lib, params(dtype=2, cache_dtype=2)) == UNSUPPORTED
    assert attention(lib, good, q=0) == attention(lib, good, out=A + 8) == attention(lib, good, lse=A + 2) == INVALID
    if need > 256:
        assert attention(lib, good, n=need - 1) == WORKSPACE
    assert read(lib, good, ko=0) == read(lib, good, vo=A + 8) == read(lib, good, off=A + 4) == INVALID
    assert read(lib, good, rows=-1) == read(lib, good, off=None, rows=1999) == INVALID
    for kw in (dict(k=0), dict(v=A + 8), dict(q_out=0), dict(k_stride=1023), dict(k_stride=1028), dict(q_stride=4088),
               dict(q_out=A, q_stride=4104), dict(q=0), dict(q_norm=A + 2), dict(k_norm=A, eps=-1.0),
               dict(k_norm=A, eps=math.nan), dict(rope_positions=0), dict(rotated=0), dict(rotated=144),
               dict(interleaved=2), dict(rope=A + 4), dict(rope=0)):
        assert append(lib, good, **kw) == INVALID, kw
    assert append(lib, good, rotated=24) == UNSUPPORTED
    assert lib.santa_kv_append(ctypes.byref(good), None, A, A, None, None, A, 256, None) == INVALID


def test_structures_and_constants_match_the_header(lib, tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "santa.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %d %d %d %d\\n", sizeof(santa_paged_t), offsetof(santa_paged_t, scale),'
                   ' sizeof(santa_append_t), offsetof(santa_append_t, interleaved), SANTA_E4M3, SANTA_CACHE_DEVERR_PAGE,'
                   ' SANTA_CACHE_DEVERR_CHUNK, SANTA_CACHE_DEVERR_POSITION);\nreturn 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(santa_build.ROOT, "include"), str(src), "-o",
                    str(tmp_path / "sizes")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(paged.PagedParams), paged.PagedParams.scale.offset, ctypes.sizeof(paged.AppendParams),
                   paged.AppendParams.interleaved.offset, paged.E4M3, santa.CACHE_DEVERR_PAGE, santa.CACHE_DEVERR_CHUNK,
                   santa.CACHE_DEVERR_POSITION]


def test_the_binding_refuses_cpu_tensors_and_wrong_pools():
    K = torch.zeros(4, 16, 2, 64)
    with pytest.raises(ValueError):
        santa.PagedCache.of(K, K)
    with pytest.raises(ValueError):
        santa.PagedCache.of(K, K[:3])
    with pytest.raises(ValueError):
        santa.PagedCache.of(K, K, torch.ones(4, 2, 16), torch.ones(4, 2, 16))


def test_rope_table():
    """Angles against Python's own 64-bit arithmetic; cos and sin rounded once to float32 (half a step, 2^-24 of 1)."""
    t = santa.rope_table(3000, 64, base=500000.0, device="cpu")
    assert t.shape == (3000, 32, 2) and t.dtype == torch.float32
    for p, i in ((0, 0), (1, 0), (2999, 0), (2999, 31), (777, 13)):
        a = p * 500000.0 ** (-2 * i / 64)
        assert abs(float(t[p, i, 0]) - math.cos(a)) <= 2.0 ** -24 and abs(float(t[p, i, 1]) - math.sin(a)) <= 2.0 ** -24
    half = santa.rope_table(3000, 64, base=500000.0, linear=2.0, device="cpu")
    assert torch.equal(half[::2], t[:1500])
    ntk = santa.rope_table(100, 64, ntk=8.0, device="cpu")
    a = 99 * 10000.0 ** (-62 / 64) / 8   # the lowest frequency is divided by 8, the highest stays
    assert abs(float(ntk[99, 31, 0]) - math.cos(a)) <= 2.0 ** -23
    assert torch.equal(ntk[:, 0], santa.rope_table(100, 64, device="cpu")[:, 0])
    parts = santa.rope_table(100, 64, by_parts=(4.0, 1.0, 4.0, 1000), attention_factor=1.5, device="cpu")
    plain = santa.rope_table(100, 64, device="cpu")
    assert abs(float(parts[99, 0, 0]) - 1.5 * float(plain[99, 0, 0])) <= 2.0 ** -22   # 159 turns: as it is
    slow = santa.rope_table(100, 64, linear=4.0, device="cpu")
    assert abs(float(parts[99, 31, 0]) - 1.5 * float(slow[99, 31, 0])) <= 2.0 ** -22  # 0.02 turns: divided by 4
    for kw in (dict(linear=0.0), dict(ntk=-1.0), dict(base=0.0), dict(by_parts=(4.0, 4.0, 1.0, 1000))):
        with pytest.raises(ValueError):
            santa.rope_table(10, 64, device="cpu", **kw)
    for bad in ((0, 64), (10, 0), (10, 7)):
        with pytest.raises(ValueError):
            santa.rope_table(*bad, device="cpu")


def test_the_packed_append_parameters_are_the_structure():
    a = paged.AppendParams()
    values = dict(q=1 << 40, k=2 << 40, v=3 << 40, q_stride=4, k_stride=-5, v_stride=6, q_out=7 << 33, q_norm=8, k_norm=9,
                  eps=0.125, rope=10, rope_positions=1 << 35, rotated=12, interleaved=1)
    for k, v in values.items():
        setattr(a, k, v)
    packed = paged._APPEND.pack(*values.values())
    size = ctypes.sizeof(a)
    assert paged._APPEND.size <= size <= paged._APPEND.size + 7      # the structure's end is padded
    back = paged.AppendParams.from_buffer_copy(packed + bytes(8))
    assert all(getattr(back, k) == v for k, v in values.items())


def test_more_output_rows_than_a_launch_has_blocks_are_refused(lib):
    p = params(total_q=1 << 28, q_offsets=A)
    assert attention(lib, p) == read(lib, p) == append(lib, p) == UNSUPPORTED
    assert lib.santa_paged_workspace_size(ctypes.byref(p)) == 0


def test_a_window_past_every_key_needs_the_workspace_of_none(lib):
    sizes = {lib.santa_paged_workspace_size(ctypes.byref(params(window=w))) for w in (0, 1000, (1 << 31) - 1)}
    assert len(sizes) == 1 and sizes.pop() > 0
