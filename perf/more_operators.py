"""Attention over a shared prefix and differential attention, in a plain form and through the library.

Both read the paged cache.  A step that knows what its sequences have in common (``prefix_lens``, ``group_offsets``)
attends to a group's prefix once for all of its sequences; ``attend_diff`` is the difference of two softmax maps, of
neighbouring heads, over the values of both, with learned weights and a norm of each pair of heads.  The two go together
where a batch of a model with such heads shares its prompt.

``own`` false: elementary torch operations in 32 bits, rounded once at the end.  ``own`` true: the library's calls.
"""
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0

# (query heads, KV heads, head dim, type): the decode geometries of this repository's workloads and tests
HEADS = ((32, 8, 128, "bf16"), (28, 4, 128, "fp16"), (16, 2, 64, "fp16"), (8, 2, 128, "bf16"), (14, 2, 128, "fp16"),
         (6, 2, 128, "bf16"), (16, 16, 64, "fp16"), (32, 8, 64, "bf16"))


def _case(name, batch, tokens, keys, heads, page, prefix=(0, 0), groups=0, e4m3=False, diff=False, norm=True,
          per_token=False, causal=True, window=0):
    """tokens, keys and prefix are ranges: new tokens of a sequence, keys of its own (those tokens among them), keys
    that a group's sequences share."""
    return {"name": name, "batch": batch, "tokens_lo": tokens[0], "tokens": tokens[1], "keys_lo": keys[0], "keys": keys[1],
            "prefix_lo": prefix[0], "prefix": prefix[1], "groups": groups, "H": heads[0], "Hkv": heads[1], "D": heads[2],
            "type": heads[3], "page": page, "e4m3": e4m3, "diff": diff, "norm": norm, "per_token": per_token,
            "causal": causal, "window": window}


def listed():
    return [
        # a few users behind a short common instruction: latency
        _case("shared_tokens_4x600", 4, (1, 1), (5, 60), HEADS[0], 16, prefix=(600, 600), groups=1),
        # several answers to one question sampled at once
        _case("shared_tokens_16x8192", 16, (1, 1), (1, 700), HEADS[1], 64, prefix=(8192, 8192), groups=1),
        # a serving batch behind one long document
        _case("shared_tokens_64x32768", 64, (1, 1), (100, 2000), HEADS[0], 64, prefix=(32768, 32768), groups=1),
        # users of three instructions, an 8-bit cache
        _case("shared_tokens_96_3groups_e4m3", 96, (1, 1), (20, 1500), HEADS[0], 128, prefix=(5000, 20001), groups=3,
              e4m3=True),
        # proposed tokens of each sequence checked at once, behind a common prefix
        _case("shared_verify_24x5_16384", 24, (2, 5), (10, 900), HEADS[2], 32, prefix=(16381, 16381), groups=1),
        # different questions read in, behind one document
        _case("shared_chunks_8x600_20000", 8, (70, 600), (70, 700), HEADS[0], 64, prefix=(20000, 20000), groups=1),
        # differential heads, one user's next token: latency
        _case("diff_token_1x1000", 1, (1, 1), (1000, 1000), HEADS[0], 16, diff=True),
        # a serving batch's next tokens, contexts of all lengths
        _case("diff_tokens_16x32768_ragged", 16, (1, 1), (1024, 32768), HEADS[1], 64, diff=True),
        # two very long contexts in an 8-bit cache
        _case("diff_tokens_2x131072_e4m3", 2, (1, 1), (100000, 131072), HEADS[0], 128, e4m3=True, diff=True),
        # a chunk of a long prompt behind what is already cached
        _case("diff_chunk_2048_in_16384", 1, (2048, 2048), (16384, 16384), HEADS[0], 64, diff=True),
        # prompts and single tokens of several users in one call, narrow heads, weights from the tokens, a sliding window
        _case("diff_mixed_6x700_window", 6, (1, 700), (900, 6001), HEADS[7], 16, diff=True, per_token=True, window=4096),
        # differential heads behind a common prefix
        _case("diff_shared_32x16384", 32, (1, 1), (50, 1000), HEADS[0], 64, prefix=(16384, 16384), groups=1, diff=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    heads = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128))
    e4m3 = rng.random() < 0.35
    norm, per_token = rng.random() < 0.7, rng.random() < 0.3
    op = rng.choice(("shared", "shared", "shared_verify", "shared_chunk", "diff", "diff", "diff_chunk", "diff_cross",
                     "diff_shared"))
    if op in ("shared", "shared_verify", "diff_shared"):
        most = _log(rng, 1, 2000)
        batch = max(2, min(_log(rng, 2, 128), 150000 // most))
        tokens = (1, 1) if op != "shared_verify" else (rng.randint(1, 3), rng.randint(3, 8))
        most += tokens[1]
        prefix = _log(rng, 100, 33000)
        groups = rng.choice((1, 1, 1, rng.randint(1, max(1, min(6, batch // 2)))))
        case = _case("", batch, tokens, (tokens[1], most), heads, page, groups=groups,
                     prefix=(max(1, prefix // rng.randint(1, 3)), prefix), e4m3=e4m3, diff=op == "diff_shared", norm=norm,
                     per_token=per_token)
    elif op == "shared_chunk":
        chunk = _log(rng, 17, 600)
        batch = rng.randint(2, 8)
        prefix = _log(rng, 200, 20000)
        case = _case("", batch, (rng.randint(1, chunk), chunk), (chunk, chunk + rng.randint(0, 600)), heads, page,
                     groups=rng.choice((1, 1, 2)), prefix=(max(1, prefix // 2), prefix), e4m3=e4m3)
    elif op == "diff":
        keys = _log(rng, 200, 100000)
        batch = max(1, min(_log(rng, 1, 64), 400000 // keys))
        tokens = rng.choice(((1, 1), (1, 1), (1, 6)))
        case = _case("", batch, tokens, (max(10, keys // rng.randint(1, 12)), keys), heads, page, e4m3=e4m3, diff=True,
                     norm=norm, per_token=per_token, window=rng.choice((0, 0, _log(rng, 50, keys))))
    elif op == "diff_chunk":
        keys = _log(rng, 300, 16000)
        chunk = min(keys, _log(rng, 17, 1500))
        batch = max(1, min(rng.randint(1, 6), 40000 // keys, 20000000 // (keys * chunk)))
        case = _case("", batch, (rng.randint(1, chunk), chunk), (max(chunk, keys // rng.randint(1, 5)), keys), heads, page,
                     e4m3=e4m3, diff=True, norm=norm, per_token=per_token, window=rng.choice((0, 0, _log(rng, 100, keys))))
    else:
        keys, chunk = _log(rng, 60, 3000), _log(rng, 1, 600)
        case = _case("", rng.randint(1, 8), (rng.randint(1, chunk), chunk), (max(1, keys // 3), keys), heads, page,
                     e4m3=e4m3, diff=True, norm=norm, per_token=per_token, causal=False)
    del case["name"]
    return case


def _sizes(case):
    """New tokens and keys of its own of each sequence, first sequences and prefixes of the groups: the case's ranges,
    the first of each at their ends."""
    B, groups = case["batch"], case["groups"]
    rng = random.Random("%d %d %d %d %d" % (B, case["tokens_lo"], case["tokens"], case["keys"], case["prefix"]))
    n = [case["tokens"]] + [rng.randint(case["tokens_lo"], case["tokens"]) for _ in range(B - 1)]
    kv = [case["keys"]] + [rng.randint(case["keys_lo"], case["keys"]) for _ in range(B - 1)]
    if case["causal"]:
        kv = [max(a, b) for a, b in zip(n, kv)]
    if not groups:
        return n, kv, [0, B], [0]
    first = [0] + sorted(rng.sample(range(1, B), groups - 1)) + [B]
    prefix = [case["prefix"]] + [rng.randint(case["prefix_lo"], case["prefix"]) for _ in range(groups - 1)]
    return n, kv, first, prefix


def work(case):
    n, kv, first, prefix = _sizes(case)
    H, D, tokens = case["H"], case["D"], sum(n)
    row = case["Hkv"] * (D + 4 if case["e4m3"] else 2 * D)   # one row of K or of V in the cache
    pairs, seen = 0, sum(prefix)
    for a, b in zip(n, kv):
        if case["causal"]:
            w = case["window"] or b
            pairs += sum(min(b - a + i + 1, w) for i in range(a))
            seen += b - max(0, b - a - w + 1)
        else:
            pairs, seen = pairs + a * b, seen + b
    for g in range(len(prefix)):
        pairs += prefix[g] * sum(n[first[g]:first[g + 1]])
    weights = (4 * tokens * H // 2 if case["per_token"] else 2 * H) + 4 * D if case["diff"] else 0
    return {"bytes": 2 * seen * row + tokens * H * (4 * D + 4) + weights,
            "flops": (6 if case["diff"] else 4) * pairs * H * D}


def _quantised(x):
    """e4m3 values and the scale of each row: x is their product, but for the rounding."""
    amax = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -60)
    code = (x * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return code, (amax / E4M3_MAX).squeeze(-1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    n, kv, first, prefix = _sizes(case)
    B, H, Hkv, D, page, t = case["batch"], case["H"], case["Hkv"], case["D"], case["page"], TYPES[case["type"]]
    G = H // Hkv
    group = [g for g in range(len(prefix)) for _ in range(first[g], first[g + 1])]
    whole = [prefix[g] // page for g in group]                       # pages that a sequence shares
    most = max(-(-(prefix[g] + k) // page) for g, k in zip(group, kv))
    table = torch.full((B, most), -1, dtype=torch.int32)
    perm = torch.randperm(sum(p // page for p in prefix) + sum(-(-(p + max(kv)) // page) * B for p in prefix) + 3,
                          generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    used, shared = 0, {}
    for b, g in enumerate(group):
        if g not in shared:
            shared[g] = perm[used:used + whole[b]]
            used += whole[b]
        mine = -(-(prefix[g] + kv[b]) // page) - whole[b]
        table[b, :whole[b]] = shared[g]
        table[b, whole[b]:whole[b] + mine] = perm[used:used + mine]
        used += mine
    pages = used + 3
    rank = torch.empty_like(perm)
    rank[perm[:used].sort().values.long()] = torch.arange(used, dtype=torch.int32)   # the pool holds what is used, in no order
    table = torch.where(table >= 0, rank[table.clamp(min=0).long()], -1)
    s = {"case": case, "t": t, "table": table.to(dev), "first": first, "prefix": prefix, "n": n, "kv": kv,
         "lens": torch.tensor([prefix[g] + k for g, k in zip(group, kv)], dtype=torch.int32, device=dev),
         "offsets": torch.tensor([sum(n[:b]) for b in range(B + 1)], device=dev), "tokens": sum(n)}
    s["q"] = torch.randn(s["tokens"], H, D, generator=gen, device=dev).to(t)
    q0 = s["q"][0].float()
    lean = q0.view(Hkv // 2, G, 2, D).mean(1).reshape(Hkv, D) if case["diff"] else q0.view(Hkv, G, D).mean(1)

    def pool(planted):
        x = torch.randn(pages * page, Hkv, D, generator=gen, device=dev)
        if planted:   # one key in fifty leans towards a query, as in attention that has learned
            x = x + torch.where(torch.rand(pages * page, 1, 1, generator=gen, device=dev) < 0.02, 1.2 * lean, 0.0)
        x = x.to(t).view(pages, page, Hkv, D)
        for g, p in enumerate(prefix):   # a page that the prefix ends in is each sequence's own copy
            if p % page:
                at = s["table"][first[g]:first[g + 1], p // page].long()
                x[at, :p % page] = x[at[0], :p % page].clone()
        if not case["e4m3"]:
            return x, None
        code, scale = _quantised(x.float())
        return code, scale.transpose(1, 2).contiguous()

    (s["K"], s["ks"]), (s["V"], s["vs"]) = pool(True), pool(False)
    if case["diff"]:
        shape = (s["tokens"], H // 2) if case["per_token"] else (H // 2,)
        s["lam"] = 0.1 + 0.8 * torch.rand(shape, generator=gen, device=dev)
        s["w"] = (1 + 0.2 * torch.randn(2 * D, generator=gen, device=dev)).to(t) if case["norm"] else None
    if own:
        import stochastic_sparse_decode_split_gb300 as santa
        more = {}
        if case["groups"]:
            more = {"prefix_lens": torch.tensor(prefix, dtype=torch.int32, device=dev), "max_prefix": max(prefix),
                    "max_own": max(kv), "max_group": max(b - a for a, b in zip(first, first[1:]))}
            if case["groups"] > 1:
                more["group_offsets"] = torch.tensor(first, dtype=torch.int32, device=dev)
        cache = santa.PagedCache.of(s["K"], s["V"], s["ks"], s["vs"])
        s["step"] = santa.PagedStep(cache, s["table"], s["lens"], n_q_heads=H, dtype=t, nk=most_keys(s), max_q=max(n),
                                    total_q=s["tokens"], q_offsets=None if min(n) == max(n) else s["offsets"],
                                    causal=case["causal"], window=case["window"], diff=case["diff"], **more)
    return s


def most_keys(s):
    return max(p + max(s["kv"][a:b]) for p, a, b in zip(s["prefix"], s["first"], s["first"][1:]))


def _rows(s, at, keys):
    """K and V, float32 [.., keys, Hkv, D], of the pages `at` [.., pages]."""
    got = []
    for pool, scale in ((s["K"], s["ks"]), (s["V"], s["vs"])):
        x = pool[at.clamp(min=0).long()].float()
        if scale is not None:
            x = x * scale[at.clamp(min=0).long()].transpose(-1, -2).unsqueeze(-1)
        got.append(x.flatten(-4, -3)[..., keys, :, :])
    return got


def _plain(s):
    """One group after another: scores over the prefix for all of its sequences, over each one's own keys, one softmax."""
    case = s["case"]
    H, Hkv, D, page = case["H"], case["Hkv"], case["D"], case["page"]
    G, diff, dev = H // Hkv, case["diff"], s["q"].device
    outs, lses = [], []
    for g, P in enumerate(s["prefix"]):
        b0, b1 = s["first"][g], s["first"][g + 1]
        n = torch.tensor(s["n"][b0:b1], device=dev)
        kv = torch.tensor(s["kv"][b0:b1], device=dev)
        N, K0, nb = max(s["n"][b0:b1]), max(s["kv"][b0:b1]), b1 - b0
        i = torch.arange(N, device=dev)
        live = i < n[:, None]
        q = torch.zeros(nb, N, H, D, device=dev)
        q[live] = s["q"][sum(s["n"][:b0]):sum(s["n"][:b1])].float()
        # query heads by the key head that they meet: [nb, Hkv, G, N, D]
        q = q.view(nb, N, Hkv // 2, G, 2, D).permute(0, 2, 4, 3, 1, 5) if diff else q.view(nb, N, Hkv, G, D).permute(0, 2, 3, 1, 4)
        q = q.reshape(nb, Hkv, G, N, D).contiguous()
        lo = P // page
        K, V = _rows(s, s["table"][b0:b1, lo:-(-(P + K0) // page)], slice(P - lo * page, P - lo * page + K0))
        key = torch.arange(K0, device=dev)
        K, V = (torch.where((key < kv[:, None])[..., None, None], x, 0.0).transpose(1, 2) for x in (K, V))
        x = (q.view(nb, Hkv, G * N, D) @ K.transpose(2, 3)).mul_(D ** -0.5).view(nb, Hkv, G, N, K0)
        pos = (kv - n)[:, None] + i
        hidden = (key >= kv[:, None])[:, None].expand(nb, N, K0)
        if case["causal"]:
            hidden = hidden | (key > pos[..., None])
            if case["window"]:
                hidden = hidden | (key <= pos[..., None] - case["window"])
        x.masked_fill_(hidden[:, None, None], float("-inf"))
        if P:
            Kp, Vp = _rows(s, s["table"][b0, :-(-P // page)], slice(0, P))
            y = q.transpose(0, 1).reshape(Hkv, nb * G * N, D) @ Kp.permute(1, 2, 0)
            x = torch.cat((y.mul_(D ** -0.5).view(Hkv, nb, G, N, P).transpose(0, 1), x), -1)
        top = x.amax(-1, keepdim=True)
        x.sub_(top.clamp(min=-1e30)).exp_()
        total = x.sum(-1, keepdim=True)
        lse = (top + total.log()).squeeze(-1)
        x.div_(total.clamp(min=1e-30))
        if diff:
            x = x.view(nb, Hkv // 2, 2, G, N, -1)
            lam = s["lam"].view(-1, Hkv // 2, G)
            if case["per_token"]:
                full = torch.zeros(nb, N, Hkv // 2, G, device=dev)
                full[live] = lam[sum(s["n"][:b0]):sum(s["n"][:b1])]
                lam = full.permute(0, 2, 3, 1)[..., None]
            else:
                lam = lam[:, :, :, None, None]
            x = x[:, :, 0] - lam * x[:, :, 1]
            V = V.transpose(1, 2).reshape(nb, K0, Hkv // 2, 2 * D).transpose(1, 2)
            if P:
                Vp = Vp.view(P, Hkv // 2, 2 * D)
        heads, wide = V.shape[1], V.shape[3]
        out = (x[..., P:].reshape(nb, heads, G * N, K0) @ V).view(nb, heads, G, N, wide)
        if P:
            z = x[..., :P].transpose(0, 1).reshape(heads, nb * G * N, P) @ Vp.transpose(0, 1)
            out = out + z.view(heads, nb, G, N, wide).transpose(0, 1)
        out = out.permute(0, 3, 1, 2, 4).reshape(nb, N, heads * G, wide)[live]
        if diff:
            if s["w"] is not None:
                out = out * torch.rsqrt(out.square().mean(-1, keepdim=True) + 1e-5) * s["w"].float()
            out = out * 0.8
            lse = lse.view(nb, Hkv // 2, 2, G, N).permute(0, 4, 1, 3, 2)
        else:
            lse = lse.permute(0, 3, 1, 2)
        outs.append(out.to(s["t"]))
        lses.append(lse.reshape(nb, N, H)[live])
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def run(state):
    s = state
    if not own:
        return _plain(s)
    if s["case"]["diff"]:
        out, lse = s["step"].attend_diff(s["q"], s["lam"], norm=s["w"], eps=1e-5, gain=0.8, return_lse=True)
    else:
        out, lse = s["step"].attend(s["q"], return_lse=True)
    return {"out": out, "lse": lse}


def exact(case, seed):
    """In 64 bits, one sequence and one head after another, over all of a sequence's keys."""
    s = prepare(case, seed)
    n, kv, first, prefix = _sizes(case)
    H, Hkv, D, page, d = case["H"], case["Hkv"], case["D"], case["page"], torch.float64
    G, dev = H // Hkv, s["q"].device
    if 2 * sum(a * k for a, k in zip(n, kv)) * H * D > 4e12:
        return None

    def rows(pool, scale, pages):
        at = pages.long()
        x = pool[at].to(d)
        if scale is not None:
            x = x * scale[at].to(d).permute(0, 2, 1)[..., None]
        return x.reshape(-1, Hkv, D)

    outs, lses, row = [], [], 0
    for g in range(len(prefix)):
        P = prefix[g]
        common = {}
        for b in range(first[g], first[g + 1]):
            both = []
            for name, scale in (("K", "ks"), ("V", "vs")):
                if name not in common:
                    common[name] = rows(s[name], s[scale], s["table"][first[g], :-(-P // page)])[:P]
                mine = rows(s[name], s[scale], s["table"][b, P // page:-(-(P + kv[b]) // page)])
                both.append(torch.cat((common[name], mine[P % page:P % page + kv[b]])).transpose(0, 1).contiguous())
            K, V = both
            keys = P + kv[b]
            pos = torch.arange(keys - n[b], keys, device=dev)[:, None]
            key = torch.arange(keys, device=dev)
            keep = torch.ones(n[b], keys, dtype=torch.bool, device=dev)
            if case["causal"]:
                keep = (key <= pos) & (key > pos - (case["window"] or keys + 1))
            lse = torch.empty(n[b], H, dtype=d, device=dev)
            wide = 2 * D if case["diff"] else D
            out = torch.empty(n[b], H * D // wide, wide, dtype=d, device=dev)

            def weights(h, kvh):
                x = s["q"][row:row + n[b], h].to(d) @ K[kvh].T / D ** 0.5
                x = torch.where(keep, x, float("-inf"))
                lse[:, h] = torch.logsumexp(x, -1)
                return torch.exp(x - lse[:, h, None])

            for h in range(out.shape[1]):
                if not case["diff"]:
                    out[:, h] = weights(h, h // G) @ V[h // G]
                    continue
                j = 2 * (h // G)
                lam = (s["lam"][row:row + n[b], h, None] if case["per_token"] else s["lam"][h]).to(d)
                w = weights(2 * h, j) - lam * weights(2 * h + 1, j + 1)
                y = torch.cat((w @ V[j], w @ V[j + 1]), -1)
                if case["norm"]:
                    y = y / (y.square().mean(-1, keepdim=True) + 1e-5).sqrt() * s["w"].to(d)
                out[:, h] = 0.8 * y
            outs.append(out)
            lses.append(lse)
            row += n[b]
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
