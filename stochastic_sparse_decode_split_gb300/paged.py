"""The paged cache: new tokens written into it, exact attention over it (also
over prefixes that sequences share, and of differential heads), and its rows
back in the packed layout that ``santa_decode`` reads.

Binding of ``santa_kv_append``, ``santa_paged_attention``,
``santa_shared_attention``, ``santa_diff_attention`` and ``santa_kv_read``
(``include/santa.h`` states the layouts, the mask and the device-side checks).
``PagedCache`` holds the pool, ``PagedStep`` a batch's description and the
workspace, so that each operator of a step is one C-ABI call.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional

import torch

CACHE_DEVERR_PAGE, CACHE_DEVERR_CHUNK, CACHE_DEVERR_POSITION, CACHE_DEVERR_PREFIX = 16, 32, 64, 128   # SANTA_CACHE_DEVERR_* in santa.h
E4M3 = 3                                                                   # SANTA_E4M3
PAGE_SIZES = (16, 32, 64, 128, 256)
KEPT_ROWS_BYTES = 1 << 24   # packed rows up to this are the step's own: made anew they cost 3 us, as much as writing this many


class PagedParams(ctypes.Structure):
    """Mirror of santa_paged_t."""
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("cache_dtype", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("page_table", ctypes.c_void_p),
        ("max_pages", ctypes.c_int32),
        ("kv_lens", ctypes.c_void_p),
        ("nk", ctypes.c_int64),
        ("q_offsets", ctypes.c_void_p),
        ("max_q", ctypes.c_int32),
        ("total_q", ctypes.c_int64),
        ("causal", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class PrefixParams(ctypes.Structure):
    """Mirror of santa_prefix_t."""
    _fields_ = [
        ("n_groups", ctypes.c_int32),
        ("group_offsets", ctypes.c_void_p),
        ("prefix_lens", ctypes.c_void_p),
        ("max_prefix", ctypes.c_int64),
        ("max_own", ctypes.c_int64),
        ("max_group", ctypes.c_int32),
    ]


class DiffParams(ctypes.Structure):
    """Mirror of santa_diff_t (calls pack it with _DIFF)."""
    _fields_ = [
        ("lambda_", ctypes.c_void_p),
        ("lambda_stride", ctypes.c_int64),
        ("norm", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("gain", ctypes.c_float),
    ]


class AppendParams(ctypes.Structure):
    """Mirror of santa_append_t (calls pack it with _APPEND, in a quarter of the time)."""
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("q_out", ctypes.c_void_p),
        ("q_norm", ctypes.c_void_p),
        ("k_norm", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("rope", ctypes.c_void_p),
        ("rope_positions", ctypes.c_int64),
        ("rotated", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
    ]


_APPEND = struct.Struct("@PPPqqqPPPfPqii")   # AppendParams' fields in their order, natively aligned
_DIFF = struct.Struct("@PqPff")              # DiffParams'
_current_device, _capturing = torch.cuda.current_device, torch.cuda.is_current_stream_capturing


def _captures(stream) -> bool:
    """Whether calls on that stream (None: the current one) go into a graph."""
    if stream is None:
        return _capturing()
    with torch.cuda.stream(stream):
        return _capturing()


def declare(lib) -> None:
    """Argument types of the paged entry points."""
    vp, sz, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
    P, A = ctypes.POINTER(PagedParams), vp   # a packed santa_append_t
    lib.santa_paged_workspace_size.argtypes = [P]
    lib.santa_paged_workspace_size.restype = sz
    lib.santa_kv_append.argtypes = [P, A, vp, vp, vp, vp, vp, sz, vp]
    lib.santa_paged_attention.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.santa_kv_read.argtypes = [P, vp, vp, vp, vp, vp, i64, vp, vp, vp, sz, vp]
    X, d = ctypes.POINTER(PrefixParams), vp   # a packed santa_diff_t
    for fn in ("santa_shared_workspace_size", "santa_diff_workspace_size"):
        getattr(lib, fn).argtypes, getattr(lib, fn).restype = [P, X], sz
    lib.santa_shared_attention.argtypes = [P, X, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.santa_diff_attention.argtypes = [P, X, d, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for fn in ("santa_kv_append", "santa_paged_attention", "santa_kv_read", "santa_shared_attention", "santa_diff_attention"):
        getattr(lib, fn).restype = ctypes.c_int32


def rope_table(positions: int, rotated: int, base: float = 10000.0, *, linear: float = 1.0, ntk: float = 1.0,
               by_parts: Optional[tuple] = None, attention_factor: float = 1.0, device="cuda") -> torch.Tensor:
    """cos and sin of every position's angles, float32 [positions, rotated / 2, 2], for ``PagedStep.append``.

    The angle of pair i at position p is p * base^(-2 i / rotated), computed in float64.  For contexts longer than the
    model was trained on: ``linear`` divides every frequency; ``ntk`` raises the base to base * ntk^(rotated / (rotated
    - 2)), which divides the lowest frequency by ntk and leaves the highest; ``by_parts = (factor, low, high,
    original)`` divides by factor the frequencies that turn less than ``low`` times in ``original`` positions, leaves
    those that turn more than ``high`` times, and blends in between.  ``attention_factor`` multiplies cos and sin."""
    if positions < 1 or rotated < 2 or rotated % 2:
        raise ValueError("positions must be positive and rotated a positive even number")
    if not (base > 0 and linear > 0 and ntk > 0):
        raise ValueError("base, linear and ntk must be positive")
    if ntk != 1.0:
        if rotated == 2:
            raise ValueError("ntk needs more than one pair")
        base = base * ntk ** (rotated / (rotated - 2))
    pair = torch.arange(rotated // 2, dtype=torch.float64, device=device)
    freq = base ** (-2.0 * pair / rotated) / linear
    if by_parts is not None:
        factor, low, high, original = by_parts
        if not (factor > 0 and 0 <= low < high and original > 0):
            raise ValueError("by_parts is (factor > 0, low, high > low, original > 0)")
        turns = original * freq / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return (torch.stack((angle.cos(), angle.sin()), -1) * attention_factor).to(torch.float32)


def diff_weights(q1, k1, q2, k2, init: float) -> torch.Tensor:
    """The weights of differential heads from their learned vectors, float32: exp(q1 . k1) - exp(q2 . k2) + init over the
    last dimension, [H / 2, d] to the [H / 2] that ``PagedStep.attend_diff`` takes.  (One weight for all heads, from
    vectors [d], becomes that by ``.expand(H // 2).contiguous()``, once per layer.)"""
    q1, k1, q2, k2 = (x.float() for x in (q1, k1, q2, k2))
    return (q1 * k1).sum(-1).exp() - (q2 * k2).sum(-1).exp() + init


class PagedCache:
    """A pool of pages: K and V [n_pages, page_size, n_kv_heads, head_dim] in bf16, fp16, fp32 or e4m3 and, for an e4m3
    cache, the rows' scales k_scale and v_scale [n_pages, n_kv_heads, page_size].  Attention takes bf16 and fp16 tokens;
    an fp32 cache is written, read back and sampled from."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                 device="cuda"):
        shape = (n_pages, page_size, n_kv_heads, head_dim)
        stored = torch.uint8 if dtype == torch.float8_e4m3fn else dtype   # code 0 is the value 0
        K, V = (torch.zeros(shape, dtype=stored, device=device).view(dtype) for _ in range(2))
        ks = vs = None
        if dtype == torch.float8_e4m3fn:
            ks, vs = (torch.ones((n_pages, n_kv_heads, page_size), dtype=torch.float32, device=device)
                      for _ in range(2))
        self._take(K, V, ks, vs)

    @classmethod
    def of(cls, K, V, k_scale=None, v_scale=None) -> "PagedCache":
        """A cache of tensors that are there already (nothing is copied)."""
        self = cls.__new__(cls)
        self._take(K, V, k_scale, v_scale)
        return self

    def _take(self, K, V, ks, vs):
        from . import DTYPES
        if K.dim() != 4 or K.shape != V.shape or K.dtype != V.dtype:
            raise ValueError("K and V must both be [n_pages, page_size, n_kv_heads, head_dim] of one type")
        self.quantized = K.dtype == torch.float8_e4m3fn
        if not self.quantized and K.dtype not in DTYPES:
            raise ValueError("the cache must be bf16, fp16, fp32 or e4m3")
        if self.quantized != (ks is not None) or self.quantized != (vs is not None):
            raise ValueError("k_scale and v_scale belong to an e4m3 cache, and to no other")
        tensors = [K, V] + ([ks, vs] if self.quantized else [])
        if any(not t.is_cuda or not t.is_contiguous() or t.device != K.device for t in tensors):
            raise ValueError("the cache's tensors must be contiguous CUDA tensors of one device")
        if self.quantized:
            want = (K.shape[0], K.shape[2], K.shape[1])
            if any(t.shape != want or t.dtype != torch.float32 for t in (ks, vs)):
                raise ValueError("k_scale and v_scale must be float32 [n_pages, n_kv_heads, page_size]")
        self.K, self.V, self.k_scale, self.v_scale = K, V, ks, vs
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = K.shape
        if self.page_size not in PAGE_SIZES:
            raise ValueError(f"page_size must be one of {PAGE_SIZES}")


class PagedStep:
    """A batch over a paged cache: its page table, lengths and workspace.

    page_table int32 [B, max_pages], kv_lens int32 [B] (the new tokens among them; None: nk each), q_offsets int64
    [B + 1] (None: max_q new tokens each).  All three are read by the GPU when a call runs and may be changed in place
    between calls; nk and max_q bound what they may hold.  Calls of one step share its workspace: order them on one
    stream.  Outputs that a call is not given are the step's own, as ``Decoder``'s: its next such call on that stream
    overwrites them (packed rows of more than 16 MiB are made anew by each ``read`` outside a capture, and not kept).
    Keep the step while graphs that captured its calls are used; otherwise it may go while its calls still run, on
    whichever streams (tensors given to a call with ``stream=`` are the caller's to keep until it has run).  ``error()``
    reports what the device refused.

    Sequences that have their first keys in common: ``prefix_lens`` int32 [groups] and, with more than one group,
    ``group_offsets`` int32 [groups + 1], group g being the sequences group_offsets[g] .. group_offsets[g + 1] (also read
    by the GPU when a call runs).  Attention then reads a group's prefix once, through its first sequence's row of the
    table; the new tokens stand behind it, and there is no window.  ``max_prefix`` bounds the prefixes, ``max_own`` the
    keys that a sequence has behind its own, ``max_group`` the sequences of a group: the closer, the better the work is
    divided.  ``append``, ``read`` and ``sample`` look every key up in its own sequence's row.  ``diff``: the
    step's heads are differential (``attend_diff``, whose workspace it then holds)."""

    def __init__(self, cache: PagedCache, page_table, kv_lens=None, *, n_q_heads: int, dtype=None,
                 nk: Optional[int] = None, max_q: int = 1, total_q: Optional[int] = None, q_offsets=None,
                 causal: bool = True, window: int = 0, scale: float = 0.0, prefix_lens=None, group_offsets=None,
                 max_prefix: Optional[int] = None, max_own: Optional[int] = None, max_group: Optional[int] = None,
                 diff: bool = False):
        from . import DTYPES, alloc_workspace, library
        dtype = dtype if dtype is not None else (torch.bfloat16 if cache.quantized else cache.K.dtype)
        if dtype not in DTYPES:
            raise ValueError("dtype must be bf16, fp16 or fp32")
        if not cache.quantized and cache.K.dtype != dtype:
            raise ValueError("a cache that is not e4m3 has the tokens' type")
        self.device = cache.K.device
        self._tensor(page_table, torch.int32, "page_table", 2)
        B = page_table.shape[0]
        if kv_lens is not None:
            self._tensor(kv_lens, torch.int32, "kv_lens", 1, B)
        if q_offsets is not None:
            self._tensor(q_offsets, torch.int64, "q_offsets", 1, B + 1)
            if total_q is None:
                raise ValueError("give total_q (the rows of the token arrays) with q_offsets")
        self.cache, self.page_table, self.kv_lens, self.q_offsets = cache, page_table, kv_lens, q_offsets
        self.dtype, self.batch, self.n_q_heads = dtype, B, n_q_heads
        self.nk = int(nk) if nk is not None else page_table.shape[1] * cache.page_size
        self.total_q = int(total_q) if total_q is not None else B * max_q
        for name, x in (("n_q_heads", n_q_heads), ("max_q", max_q), ("window", window), ("nk", self.nk), ("total_q", self.total_q)):
            if not 0 <= x < 1 << 31:   # ctypes would cut it off
                raise ValueError(f"{name} = {x} is out of range")
        p = PagedParams()
        p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim = B, n_q_heads, cache.n_kv_heads, cache.head_dim
        p.dtype = DTYPES[dtype]
        p.cache_dtype = E4M3 if cache.quantized else p.dtype
        p.page_size, p.n_pages, p.max_pages = cache.page_size, cache.n_pages, page_table.shape[1]
        p.page_table = page_table.data_ptr()
        p.kv_lens = None if kv_lens is None else kv_lens.data_ptr()
        p.q_offsets = None if q_offsets is None else q_offsets.data_ptr()
        p.nk, p.max_q, p.total_q = self.nk, int(max_q), self.total_q
        p.causal, p.window, p.scale = int(bool(causal)), int(window), float(scale)
        self.p, self._ref = p, ctypes.byref(p)
        self.prefix_lens, self.group_offsets, self.diff = prefix_lens, group_offsets, bool(diff)
        self._prefix = self._prefix_ref = None
        if prefix_lens is not None:
            self._groups(max_prefix, max_own, max_group)
        elif any(x is not None for x in (group_offsets, max_prefix, max_own, max_group)):
            raise ValueError("group_offsets, max_prefix, max_own and max_group go with prefix_lens")
        with torch.cuda.device(self.device):
            sizes = [library().santa_paged_workspace_size(self._ref) if self._prefix is None
                     else library().santa_shared_workspace_size(self._ref, self._prefix_ref)]
            if self.diff:
                sizes.append(library().santa_diff_workspace_size(self._ref, self._prefix_ref))
            n = max(sizes)
            if min(sizes) == 0:
                raise ValueError("invalid paged parameters")
            self.workspace = alloc_workspace(n, self.device)
            # the stream that clears the workspace's error word, and when it has
            self._streams = {torch._C._cuda_getCurrentRawStream(self.device.index)}
            self._cleared = None if _capturing() else torch.cuda.current_stream().record_event()
        # what every call checks and passes again: shapes, the pool (whose tensors the cache keeps), the workspace
        self._index = self.device.index
        self._outputs, self._captured = {}, []
        self._shape = torch.Size((self.total_q, n_q_heads, cache.head_dim))
        self._kv_shape = torch.Size((self.total_q, cache.n_kv_heads, cache.head_dim))
        self._lse_shape, self._weight_shape = self._shape[:2], self._shape[2:]
        self._diff_shape = torch.Size((self.total_q, n_q_heads // 2, 2 * cache.head_dim))
        self._pairs, self._norm_shape = self._diff_shape[1:2], self._diff_shape[2:]
        self._kept = (cache.K, cache.V, cache.k_scale, cache.v_scale)
        self._pool = tuple(ctypes.c_void_p(None if t is None else t.data_ptr()) for t in self._kept)
        self._ws = (ctypes.c_void_p(self.workspace.data_ptr()), ctypes.c_size_t(n))
        lib = library()
        self._append_fn, self._attend_fn, self._read_fn = lib.santa_kv_append, lib.santa_paged_attention, lib.santa_kv_read
        self._shared_fn, self._diff_fn = lib.santa_shared_attention, lib.santa_diff_attention

    def _groups(self, max_prefix, max_own, max_group):
        """The santa_prefix_t of prefix_lens and group_offsets."""
        n = self.prefix_lens.shape[0] if self.prefix_lens.dim() == 1 else 0
        self._tensor(self.prefix_lens, torch.int32, "prefix_lens", 1, n)
        if self.group_offsets is not None:
            self._tensor(self.group_offsets, torch.int32, "group_offsets", 1, n + 1)
        elif n != 1:
            raise ValueError("give group_offsets with more than one group")
        bounds = (self.nk if max_prefix is None else max_prefix, self.nk if max_own is None else max_own,
                  self.batch if max_group is None else max_group)
        for name, x in zip(("max_prefix", "max_own", "max_group"), bounds):
            if not 1 <= x < 1 << 31:
                raise ValueError(f"{name} = {x} is out of range")
        x = self._prefix = PrefixParams()
        x.n_groups, x.prefix_lens = n, self.prefix_lens.data_ptr()
        x.group_offsets = None if self.group_offsets is None else self.group_offsets.data_ptr()
        x.max_prefix, x.max_own, x.max_group = (int(b) for b in bounds)
        self._prefix_ref = ctypes.byref(x)

    def _tensor(self, t, dtype, name, dim, size=None):
        if t.dtype != dtype or t.dim() != dim or (size is not None and t.shape[0] != size):
            raise ValueError(f"{name} must be {dtype} with {dim} dimension(s)" + (f" and {size} entries" if size else ""))
        if t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous and on the cache's device")

    def _heads(self, x, shape, name):
        """Token rows of heads: any row stride, each row dense.  Returns the stride in elements."""
        row, head, one = x.stride() if x.dim() == 3 else (0, 0, 0)
        if x.dtype is not self.dtype or x.shape != shape or x.get_device() != self._index:   # -1: not on a GPU
            raise ValueError(f"{name} must be {self.dtype} {list(shape)} on the cache's device")
        if one != 1 or (head != shape[2] and shape[1] > 1):
            raise ValueError(f"the rows of {name} must be dense")
        return row if shape[0] > 1 else shape[1] * shape[2]

    def _dense(self, x, shape, dtype, name):
        if x.dtype is not dtype or x.shape != shape or x.get_device() != self._index or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on the cache's device")
        return x.data_ptr()

    def _on(self, stream):
        """The raw stream of a call: the given one, or the device's current one."""
        if _current_device() != self._index:
            raise ValueError("make the cache's device the current one for its calls")
        raw = torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream
        if raw not in self._streams:
            self._meet(raw, stream)
        return raw

    def _meet(self, raw, stream):
        """The first call on a stream other than the step's own: behind the clearing of the error word, and what the step
        holds goes back to the allocator, when it is dropped, only after what that stream does with it."""
        with torch.cuda.stream(stream):
            on = torch.cuda.current_stream()
            for t in (self.workspace, self.page_table, self.kv_lens, self.q_offsets, self.prefix_lens, self.group_offsets,
                      *self._kept):
                if t is not None:
                    t.record_stream(on)
            if not _capturing():   # a capture takes no event from outside; it begins with a synchronisation
                if self._cleared is not None:
                    on.wait_event(self._cleared)
                self._streams.add(raw)

    def _own(self, name, raw, shape, dtype, stream, most=None):
        """The step's own output of that name for calls on that stream (making one anew costs as much as a call).  One
        of more than ``most`` bytes is not kept, and takes the place of the one that was."""
        x = self._outputs.get((name, raw))
        if x is None or x.shape != shape:
            with torch.cuda.stream(stream):
                x = self._outputs[name, raw] = torch.empty(shape, dtype=dtype, device=self.device)
            if most is not None and x.nbytes > most:
                del self._outputs[name, raw]
        return x

    @staticmethod
    def _check(status, fn):
        if status:
            from . import SantaError
            raise SantaError(status, fn)

    def append(self, q, k, v, *, rope=None, interleaved: bool = False, q_norm=None, k_norm=None, eps: float = 1e-6,
               q_out=None, stream=None):
        """New tokens into the cache; returns the rotated and normalised queries [total_q, n_q_heads, head_dim] (None
        with q None).  q, k and v may be slices of one row-major projection.  Token rows past q_offsets[-1] of q_out
        are left as they were."""
        raw = self._on(stream)
        k_stride, v_stride = self._heads(k, self._kv_shape, "k"), self._heads(v, self._kv_shape, "v")
        q_ptr = q_stride = q_out_ptr = qw = kw = rope_ptr = positions = rotated = 0
        if q is not None:
            q_stride, q_ptr = self._heads(q, self._shape, "q"), q.data_ptr()
            if q_out is None:
                q_out = self._own("q", raw, self._shape, self.dtype, stream)
                q_out_ptr = q_out.data_ptr()
            else:
                q_out_ptr = self._dense(q_out, self._shape, self.dtype, "q_out")
        elif q_out is not None or q_norm is not None:
            raise ValueError("q_out and q_norm go with q")
        if q_norm is not None:
            qw = self._dense(q_norm, self._weight_shape, self.dtype, "q_norm")
        if k_norm is not None:
            kw = self._dense(k_norm, self._weight_shape, self.dtype, "k_norm")
        if rope is not None:
            shape = rope.shape
            if len(shape) != 3 or shape[2] != 2:
                raise ValueError("rope must be [positions, rotated / 2, 2]")
            rope_ptr = self._dense(rope, shape, torch.float32, "rope")
            positions, rotated = shape[0], 2 * shape[1]
        a = _APPEND.pack(q_ptr, k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, q_out_ptr, qw, kw, eps, rope_ptr,
                         positions, rotated, 1 if interleaved and rotated else 0)
        self._check(self._append_fn(self._ref, a, *self._pool, *self._ws, raw), "santa_kv_append")
        return q_out

    def attend(self, q, *, out=None, lse=None, return_lse: bool = False, stream=None):
        """softmax(scale q K^T + mask) V over the pages, [total_q, n_q_heads, head_dim] in q's type, bf16 or fp16 (out may
        be q); with return_lse (or an lse to fill) also the float32 [total_q, n_q_heads] logarithms of the softmax sums."""
        raw = self._on(stream)
        q_ptr = self._dense(q, self._shape, self.dtype, "q")
        if out is not None:
            out_ptr = self._dense(out, self._shape, self.dtype, "out")
        else:
            out = self._own("out", raw, self._shape, self.dtype, stream)
            out_ptr = out.data_ptr()
        lse_ptr = None
        if lse is not None:
            lse_ptr = self._dense(lse, self._lse_shape, torch.float32, "lse")
        elif return_lse:
            lse = self._own("lse", raw, self._lse_shape, torch.float32, stream)
            lse_ptr = lse.data_ptr()
        if self._prefix is None:
            self._check(self._attend_fn(self._ref, q_ptr, *self._pool, out_ptr, lse_ptr, *self._ws, raw), "santa_paged_attention")
        else:
            self._check(self._shared_fn(self._ref, self._prefix_ref, q_ptr, *self._pool, out_ptr, lse_ptr, *self._ws, raw),
                        "santa_shared_attention")
        return out if lse is None else (out, lse)

    def attend_diff(self, q, weights, *, norm=None, eps: float = 1e-5, gain: float = 1.0, out=None, lse=None,
                    return_lse: bool = False, stream=None):
        """Differential attention, [total_q, n_q_heads / 2, 2 head_dim] in q's type: query heads 2h and 2h + 1 against key
        heads 2j and 2j + 1 (j = h / (n_q_heads / n_kv_heads)), the first map less ``weights`` times the second over the
        values of both, divided by the root of its mean square (+ eps) and multiplied by ``norm`` [2 head_dim] where that
        is given, and by ``gain``.  weights: float32 [n_q_heads / 2], or [total_q, n_q_heads / 2] with dense rows.  out may
        lie over q; with return_lse (or an lse to fill) also the float32 [total_q, n_q_heads] logarithms of the maps' sums."""
        raw = self._on(stream)
        if not self.diff:
            raise ValueError("make the step with diff=True")
        q_ptr = self._dense(q, self._shape, self.dtype, "q")
        stride = 0
        if weights.shape != self._pairs or not weights.is_contiguous():   # not the same for all tokens
            pairs = self._pairs[0]
            if weights.shape != self._diff_shape[:2] or (pairs > 1 and weights.stride(1) != 1):
                raise ValueError("weights must be [n_q_heads / 2] or [total_q, n_q_heads / 2] with dense rows")
            stride = weights.stride(0) if self.total_q > 1 else 0
            if 0 < stride < pairs:
                raise ValueError("the rows of weights overlap")
        if weights.dtype is not torch.float32 or weights.get_device() != self._index:
            raise ValueError("weights must be float32 on the cache's device")
        if out is not None:
            out_ptr = self._dense(out, self._diff_shape, self.dtype, "out")
        else:
            out = self._own("diff", raw, self._diff_shape, self.dtype, stream)
            out_ptr = out.data_ptr()
        lse_ptr = None
        if lse is not None:
            lse_ptr = self._dense(lse, self._lse_shape, torch.float32, "lse")
        elif return_lse:
            lse = self._own("lse", raw, self._lse_shape, torch.float32, stream)
            lse_ptr = lse.data_ptr()
        norm_ptr = 0 if norm is None else self._dense(norm, self._norm_shape, self.dtype, "norm")
        d = _DIFF.pack(weights.data_ptr(), stride, norm_ptr, eps, gain)
        self._check(self._diff_fn(self._ref, self._prefix_ref, d, q_ptr, *self._pool, out_ptr, lse_ptr, *self._ws, raw),
                    "santa_diff_attention")
        return out if lse is None else (out, lse)

    def read(self, kv_offsets=None, rows: Optional[int] = None, *, K_out=None, V_out=None, stream=None):
        """The sequences' keys and values as packed rows [rows, n_kv_heads, head_dim] in the tokens' type: key n of
        sequence b in row kv_offsets[b] + n (int64 [B + 1]; None: b * nk).  Rows that no key falls on keep what they
        held."""
        raw = self._on(stream)
        off_ptr = None
        if kv_offsets is not None:
            if rows is None:
                raise ValueError("give rows (of the packed arrays) with kv_offsets")
            off_ptr = self._dense(kv_offsets, (self.batch + 1,), torch.int64, "kv_offsets")
        elif rows is None:
            rows = self.batch * self.nk
        shape = (rows, self._kv_shape[1], self._kv_shape[2])
        if K_out is None or V_out is None:
            # what a graph writes to is kept, and the next capture's; a later call with other rows replaces it as the
            # step's own, but the graph still writes there
            captured = _captures(stream)
            most = None if captured else KEPT_ROWS_BYTES
            if K_out is None:
                K_out = self._own("K", raw, shape, self.dtype, stream, most)
            if V_out is None:
                V_out = self._own("V", raw, shape, self.dtype, stream, most)
            if captured and not any(K is K_out and V is V_out for K, V in self._captured):
                self._captured.append((K_out, V_out))
        self._check(self._read_fn(self._ref, *self._pool, off_ptr, rows, self._dense(K_out, shape, self.dtype, "K_out"),
                                  self._dense(V_out, shape, self.dtype, "V_out"), *self._ws, raw), "santa_kv_read")
        return K_out, V_out

    def sample(self, q, S: int, kv_offsets, rows: int, *, variant: str = "systematic", seed: int = 0, step: int = 0,
               sample_idx=None, stream=None):
        """One S2ANTA / SANTA decode step over the paged cache: its rows read back packed (kv_offsets the exclusive
        sums of kv_lens), then santa_decode on them, for steps of one token per sequence that sees all of its keys.
        q [B, n_q_heads, head_dim]; the result is float32.  The packed copy costs twice the cache's bytes: ``attend`` is
        exact and moves them once, so this is for what wants the estimator's draws."""
        from . import santa_decode
        if self.total_q != self.batch:
            raise ValueError("sample takes steps of one token per sequence")
        if 0 < self.p.window < self.nk:
            raise ValueError("sample knows no window: it would draw from keys that the token does not see")
        with torch.cuda.device(self.device), torch.cuda.stream(stream):
            K, V = self.read(kv_offsets, rows)
            return santa_decode(q, K, V, S, variant=variant, seed=seed, step=step, nk=self.nk, kv_offsets=kv_offsets,
                                scale=self.p.scale, sample_idx=sample_idx)

    def error(self, stream=None) -> int:
        """Synchronises and returns (then clears) the device error bits."""
        from . import get_error
        with torch.cuda.device(self.device):
            return get_error(self.workspace, stream)
