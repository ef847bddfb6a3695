"""Batches whose sequences share prefixes, and differential attention's definition in 64 bits."""
import random

import torch

from paged_reference import Batch, half_step, quantised

NAN = float("nan")


class Shared(Batch):
    """Groups of sequences: own[b] keys behind the prefix of b's group, n[b] of them new.  Of a prefix only the pages that
    its group's first sequence names hold it: the other rows of the table say -7 there, and their own copies of the page
    that it ends in hold NaN in its place.  (A run of the plain attention wants ``whole``: tables and copies filled in.)"""

    def __init__(self, prefix, first, own, n, H, Hkv, D, dtype=torch.bfloat16, e4m3=False, page=16, seed=0, pad=0,
                 shared_n=False, whole=False, device="cuda", pairs=False):
        of = [g for g in range(len(prefix)) for _ in range(first[g], first[g + 1])]
        self.prefix, self.first, self.own, self.group = prefix, first, own, of
        self.kv, self.n, self.H, self.Hkv, self.D, self.dtype, self.e4m3, self.page = (
            [prefix[g] + k for g, k in zip(of, own)], n, H, Hkv, D, dtype, e4m3, page)
        self.B = len(own)
        gen = torch.Generator(device="cpu").manual_seed(seed)
        rng = random.Random(seed)
        self.max_pages = max(-(-k // page) for k in self.kv) + 1
        shared = [p // page for p in prefix]                     # pages that lie wholly inside a prefix
        mine = [-(-self.kv[b] // page) - shared[of[b]] for b in range(self.B)]
        for g, p in enumerate(prefix):                           # the first sequence's row holds the whole prefix
            if first[g] < first[g + 1]:
                mine[first[g]] = max(mine[first[g]], -(-p // page) - shared[g])
        self.n_pages = sum(shared) + sum(mine) + 3
        order = list(range(self.n_pages))
        rng.shuffle(order)
        K = torch.full((self.n_pages, page, Hkv, D), NAN)
        V = K.clone()
        table = torch.full((self.B, self.max_pages), -7, dtype=torch.int32)
        self.full = []                                           # page lists with the prefix's in them
        self.tokens, self.pad = sum(n), pad
        self.total_q = self.tokens + pad
        self.q = torch.randn(self.total_q, H, D, generator=gen).to(dtype)
        G = H // Hkv
        lean = 0.0
        if self.tokens:
            q0 = self.q[0].float()
            lean = 1.5 * (q0.view(Hkv // 2, G, 2, D).mean(1).reshape(Hkv, D) if pairs else q0.view(Hkv, G, D).mean(1))

        def rows(keys):
            k, v = (torch.randn(keys, Hkv, D, generator=gen) for _ in range(2))
            if keys:
                at = torch.randperm(keys, generator=gen)[:max(1, keys // 60)]
                k[at] += lean
            return k.to(dtype).float(), v.to(dtype).float()

        common = [rows(p) for p in prefix]
        pages = [[order.pop() for _ in range(s)] for s in shared]
        for b in range(self.B):
            g = of[b]
            k, v = (torch.cat((c, x)) for c, x in zip(common[g], rows(own[b])))
            list_b = pages[g] + [order.pop() for _ in range(mine[b])]
            self.full.append(list_b)
            leads = b == first[g]
            table[b, :len(list_b)] = torch.tensor(list_b, dtype=torch.int32)
            if not leads and not whole:
                table[b, :shared[g]] = -7
            for pool, x in ((K, k), (V, v)):
                for i, pg in enumerate(list_b):
                    part = x[i * page:(i + 1) * page].clone()
                    if i < shared[g] and not leads:
                        continue
                    if not leads and not whole and i == shared[g]:
                        part[:prefix[g] % page] = NAN
                    pool[pg, :part.shape[0]] = part
        K, V = K.to(device), V.to(device)
        if e4m3:
            (self.K, ks), (self.V, vs) = quantised(K), quantised(V)
            self.ks, self.vs = (s.transpose(1, 2).contiguous() for s in (ks, vs))
        else:
            self.K, self.V, self.ks, self.vs = K.to(dtype), V.to(dtype), None, None
        self.q, self.table = self.q.to(device), table.to(device)
        self.offsets = torch.tensor([sum(n[:b]) for b in range(self.B + 1)], device=device)
        self.uniform = shared_n
        self.kv_t = torch.tensor(self.kv, dtype=torch.int32, device=device)
        self.prefix_t = torch.tensor(prefix, dtype=torch.int32, device=device)
        self.first_t = torch.tensor(first, dtype=torch.int32, device=device)
        self.device = device

    def shared_step(self, **kw):
        kw.setdefault("max_prefix", max(max(self.prefix), 1))
        kw.setdefault("max_own", max(max(self.own), 1))
        kw.setdefault("max_group", max(b - a for a, b in zip(self.first, self.first[1:])))
        kw.setdefault("group_offsets", self.first_t if len(self.prefix) > 1 else None)
        return self.step(prefix_lens=self.prefix_t, **kw)

    def rows(self, b, which):
        pool, scale = (self.K, self.ks) if which == "K" else (self.V, self.vs)

        def read(pages):
            at = torch.tensor(pages, device=pool.device, dtype=torch.long)
            x = pool[at].to(torch.float64)
            if scale is not None:
                x = x * scale[at].to(torch.float64).transpose(1, 2)[..., None]
            return x.reshape(-1, self.Hkv, self.D)

        p = self.prefix[self.group[b]]
        lead = read(self.full[self.first[self.group[b]]])[:p]
        return torch.cat((lead, read(self.full[b])[p:self.kv[b]]))


def diff_attention(batch, weights, norm=None, eps=1e-5, gain=1.0, causal=True, window=0, scale=None):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits; padding rows zero.

    Each map's output a_e may be off by T_e as in ``paged_reference.attention`` (16-bit probabilities, 32-bit scores), but
    for the rounding of the result; the difference x = a_0 - w a_1 by T = T_0 + |w| T_1 and 2^-22 of its terms.  Its root
    mean square r (with eps) may be off by t = rms(T), since r is a norm of (x, sqrt(eps)), so x / r by (T + |x / r| t) /
    (r - t).  The result is rounded once (half a step), the factors before it cost 2^-20 of it."""
    H, Hkv, D = batch.H, batch.Hkv, batch.D
    G, scale = H // Hkv, D ** -0.5 if scale is None else scale
    dev, d = batch.q.device, torch.float64
    out = torch.zeros(batch.total_q, H // 2, 2 * D, dtype=d, device=dev)
    lse = torch.full((batch.total_q, H), float("-inf"), dtype=d, device=dev)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = half_step(batch.dtype)
    weights = weights.to(d).expand(batch.total_q, H // 2) if weights.dim() == 1 else weights.to(d)
    first = 0
    for b in range(batch.B):
        n, kv = batch.n[b], batch.kv[b]
        rows = slice(first, first + n)
        first += n
        if not kv or not n:
            continue
        K, V = batch.rows(b, "K"), batch.rows(b, "V")
        pos = torch.arange(kv - n, kv, device=dev)[:, None]
        key = torch.arange(kv, device=dev)
        keep = torch.ones(n, kv, dtype=torch.bool, device=dev)
        if causal:
            keep = key <= pos
            if window:
                keep = keep & (key > pos - window)
        any_key = keep.any(1)
        for h in range(H // 2):
            j = 2 * (h // G)
            v = torch.cat((V[:, j], V[:, j + 1]), -1)
            clean = torch.where(torch.isfinite(v), v, 0.0)
            a, T = [], []
            for e in range(2):
                q, k = batch.q[rows, 2 * h + e].to(d), K[:, j + e]
                x = torch.where(keep, q @ k.T * scale, float("-inf"))
                size = torch.where(keep, q.abs() @ k.abs().T * scale, 0.0).amax(1)
                row = torch.logsumexp(x, 1)
                p = torch.where(keep, torch.exp(x - row[:, None]), 0.0)
                o = p @ clean
                for i in (~torch.isfinite(v).all(1)).nonzero().flatten().tolist():
                    o = torch.where(keep[:, i, None], o + torch.where(torch.isfinite(v[i]), 0.0, v[i]), o)
                err = 2 * (D + 8) * 2.0 ** -23 * size + 2.0 ** -20
                a.append(o)
                T.append((u + err[:, None]) * (1 + u) * (p @ clean.abs()))
                lse[rows, 2 * h + e] = torch.where(any_key, row, float("-inf"))
                tol_lse[rows, 2 * h + e] = err + 2.0 ** -20 * row.abs()
            w = weights[rows, h, None]
            y = a[0] - w * a[1]
            t = T[0] + w.abs() * T[1] + 2.0 ** -22 * (a[0].abs() + (w * a[1]).abs())
            if norm is not None:
                r, tr = (y.square().mean(-1, keepdim=True) + eps).sqrt(), t.square().mean(-1, keepdim=True).sqrt()
                y = y / r
                t = (t + y.abs() * tr) / (r - tr)
                ok = (r > 2 * tr) | ~torch.isfinite(r) | ~any_key[:, None]
                assert bool(ok.all()), "a row whose difference is mostly rounding: not an input to compare by"
                y, t = y * norm.to(d), t * norm.to(d).abs()
            y, t = gain * y, abs(gain) * t
            out[rows, h] = torch.where(any_key[:, None], y, 0.0)
            tol[rows, h] = t * (1 + u) + (u + 2.0 ** -20) * y.abs() * (1 + 2 * u)
    return out, lse, tol, tol_lse


def check_diff(batch, got, lse, weights, **kw):
    want, want_lse, tol, tol_lse = diff_attention(batch, weights, **kw)
    t = batch.tokens
    got, lse = got[:t].double(), lse[:t].double()
    fine = torch.isfinite(want[:t])
    assert torch.equal(torch.isfinite(got), fine), "finite where the definition is not, or the other way round"
    off = ((got - want[:t]).abs() - tol[:t])[fine]
    assert not off.numel() or float(off.max()) <= 0, f"out is {float(off.max()):.3g} over its tolerance"
    assert torch.equal(lse == float("-inf"), want_lse[:t] == float("-inf"))
    off = ((lse - want_lse[:t]).abs() - tol_lse[:t])[torch.isfinite(want_lse[:t])]
    assert not off.numel() or float(off.max()) <= 0, f"lse is {float(off.max()):.3g} over its tolerance"
