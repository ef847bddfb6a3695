"""Batches over a paged cache for the tests, and the operators' definitions in
64 bits, one sequence and one head at a time."""
import random

import torch

F8 = torch.float8_e4m3fn
FLOOR = 2.0 ** -60


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def quantised(x):
    """float32 rows [..., D] as (codes, scales), as include/santa.h states it."""
    amax = x.abs().amax(-1, keepdim=True).clamp(min=FLOOR)
    code = (x * torch.div(torch.full_like(amax, 448.0), amax)).clamp(-448, 448).to(F8)
    return code, torch.div(amax, torch.full_like(amax, 448.0)).squeeze(-1)


class Batch:
    """Lengths, pages and a cache full of values; what no key owns holds NaN."""

    def __init__(self, kv, n, H, Hkv, D, dtype=torch.bfloat16, e4m3=False, page=16, seed=0, device="cuda", pad=0,
                 shared_n=False, planted=True):
        self.kv, self.n, self.H, self.Hkv, self.D, self.dtype, self.e4m3, self.page = kv, n, H, Hkv, D, dtype, e4m3, page
        self.B = len(kv)
        gen = torch.Generator(device="cpu").manual_seed(seed)
        rng = random.Random(seed)
        self.used = [-(-k // page) for k in kv]
        self.max_pages = max(max(self.used), 1) + 1
        self.n_pages = sum(self.used) + 3
        order = list(range(self.n_pages))
        rng.shuffle(order)
        table = torch.full((self.B, self.max_pages), -7, dtype=torch.int32)
        for b in range(self.B):
            for i in range(self.used[b]):
                table[b, i] = order.pop()
        self.table = table.to(device)
        self.tokens, self.pad = sum(n), pad
        self.total_q = self.tokens + pad
        self.offsets = torch.tensor([sum(n[:b]) for b in range(self.B + 1)], device=device)
        self.uniform = shared_n
        self.kv_t = torch.tensor(kv, dtype=torch.int32, device=device)
        self.q = torch.randn(self.total_q, H, D, generator=gen).to(dtype).to(device)
        self.K_rows, self.V_rows = [], []   # float32 [kv, Hkv, D]: what the cache stands for
        K = torch.full((self.n_pages, page, Hkv, D), float("nan"), device=device)
        V = K.clone()
        for b in range(self.B):
            k, v = (torch.randn(kv[b], Hkv, D, generator=gen).to(device) for _ in range(2))
            if planted and self.tokens and kv[b]:
                at = torch.randperm(kv[b], generator=gen)[:max(1, kv[b] // 60)].to(device)
                k[at] += 1.5 * self.q[0].float().view(Hkv, H // Hkv, D).mean(1)
            k, v = k.to(dtype).float(), v.to(dtype).float()
            for pool, x in ((K, k), (V, v)):
                for i in range(self.used[b]):
                    part = x[i * page:(i + 1) * page]
                    pool[int(table[b, i]), :part.shape[0]] = part
        if e4m3:
            self.K, ks = quantised(K)
            self.V, vs = quantised(V)
            self.ks, self.vs = (s.transpose(1, 2).contiguous() for s in (ks, vs))
        else:
            self.K, self.V, self.ks, self.vs = K.to(dtype), V.to(dtype), None, None
        self.device = device

    def cache(self):
        import stochastic_sparse_decode_split_gb300 as santa
        return santa.PagedCache.of(self.K, self.V, self.ks, self.vs)

    def step(self, **kw):
        import stochastic_sparse_decode_split_gb300 as santa
        kw.setdefault("nk", max(max(self.kv), 1))
        return santa.PagedStep(self.cache(), self.table, self.kv_t, n_q_heads=self.H, dtype=self.dtype,
                               max_q=max(self.n), total_q=self.total_q,
                               q_offsets=None if self.uniform else self.offsets, **kw)

    def rows(self, b, which):
        """float64 [kv, Hkv, D] of what the cache holds for sequence b."""
        pool, scale = (self.K, self.ks) if which == "K" else (self.V, self.vs)
        at = self.table[b, :self.used[b]].long()
        x = pool[at].to(torch.float64)
        if scale is not None:
            x = x * scale[at].to(torch.float64).transpose(1, 2)[..., None]
        return x.reshape(-1, self.Hkv, self.D)[:self.kv[b]]


def attention(batch, causal=True, window=0, scale=None):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits, padding rows zero.

    The tolerance counts: the rounding of the output to its type (half a step of it) and of every probability to 16
    bits (half a step of it, so at most that share of sum p |v|); the 32-bit sums of the scores (D products, each
    rounding at most 2^-23 of the sum of magnitudes, twice for the maximum's own error) and the exponential's 2^-21."""
    H, Hkv, D = batch.H, batch.Hkv, batch.D
    scale = D ** -0.5 if scale is None else scale
    dev, d = batch.q.device, torch.float64
    out = torch.zeros(batch.total_q, H, D, dtype=d, device=dev)
    lse = torch.full((batch.total_q, H), float("-inf"), dtype=d, device=dev)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = half_step(batch.dtype)
    first = 0
    for b in range(batch.B):
        n, kv = batch.n[b], batch.kv[b]
        K, V = batch.rows(b, "K"), batch.rows(b, "V")
        pos = torch.arange(kv - n, kv, device=dev)[:, None]
        key = torch.arange(kv, device=dev)
        keep = torch.ones(n, kv, dtype=torch.bool, device=dev)
        if causal:
            keep = key <= pos
            if window:
                keep = keep & (key > pos - window)
        any_key = keep.any(1)
        for h in range(H):
            if not kv:
                continue
            q, k, v = batch.q[first:first + n, h].to(d), K[:, h * Hkv // H], V[:, h * Hkv // H]
            x = torch.where(keep, torch.nan_to_num(q @ k.T, nan=float("nan")) * scale, float("-inf"))
            size = torch.where(keep, q.abs() @ k.abs().T * scale, 0.0).amax(1)
            row = torch.logsumexp(x, 1)
            p = torch.where(keep, torch.exp(x - row[:, None]), 0.0)
            clean = torch.where(torch.isfinite(v), v, 0.0)
            o = p @ clean
            if not bool(torch.isfinite(v).all()):   # odd values reach the rows that see their key, and no other
                for j in (~torch.isfinite(v).all(1)).nonzero().flatten().tolist():
                    odd = torch.where(torch.isfinite(v[j]), 0.0, v[j])
                    o = torch.where(keep[:, j, None], o + odd, o)
            err = 2 * (D + 8) * 2.0 ** -23 * size + 2.0 ** -20
            out[first:first + n, h] = torch.where(any_key[:, None], o, 0.0)
            lse[first:first + n, h] = torch.where(any_key, row, float("-inf"))
            tol[first:first + n, h] = u * o.abs() * (1 + 2 * u) + (u + err[:, None]) * (1 + u) * (p @ clean.abs())
            tol_lse[first:first + n, h] = err + 2.0 ** -20 * row.abs()
        first += n
    return out, lse, tol, tol_lse


def check_attention(batch, got, lse, **kw):
    want, want_lse, tol, tol_lse = attention(batch, **kw)
    t = batch.tokens
    got, lse = got[:t].double(), lse[:t].double()
    fine = torch.isfinite(want[:t])
    assert torch.equal(torch.isfinite(got), fine), "finite where the definition is not, or the other way round"
    off = ((got - want[:t]).abs() - tol[:t])[fine]
    assert not off.numel() or float(off.max()) <= 0, f"out is {float(off.max()):.3g} over its tolerance"
    seen = torch.isfinite(want_lse[:t])
    assert torch.equal(lse == float("-inf"), want_lse[:t] == float("-inf"))
    off = ((lse - want_lse[:t]).abs() - tol_lse[:t])[seen]
    assert not off.numel() or float(off.max()) <= 0, f"lse is {float(off.max()):.3g} over its tolerance"
