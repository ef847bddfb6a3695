"""The paged-cache operators as a user's program calls them, in a plain form and through the library.

Three operators that belong together: ``santa_kv_append`` (queries and keys normalised per head and rotated by
their positions, keys and values written into the pages of a cache, in 16 bits or in e4m3 with one scale for each row
and head), ``santa_paged_attention`` (a chunk of new tokens, or one token, of each sequence over its pages) and
``santa_kv_read`` (the pages of a batch back as packed rows, the layout that ``santa_decode`` reads).

``own`` false: elementary torch operations in 32 bits, rounded once at the end.  ``own`` true: the library's calls.
"""
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0
FLOOR = 2.0 ** -60   # a row whose largest magnitude is below this is stored relative to it

# (query heads, KV heads, head dim, type): the decode geometries of this repository's workloads and tests
HEADS = ((32, 8, 128, "bf16"), (28, 4, 128, "fp16"), (16, 2, 64, "fp16"), (8, 2, 128, "bf16"), (14, 2, 128, "fp16"),
         (6, 2, 128, "bf16"), (10, 2, 64, "bf16"))


def _attend(name, batch, chunk, keys, heads, page, chunk_lo=0, keys_lo=0, e4m3=False, causal=True, window=0):
    return {"name": name, "op": "attend", "batch": batch, "chunk_lo": chunk_lo or chunk, "chunk": chunk,
            "keys_lo": keys_lo or keys, "keys": keys, "H": heads[0], "Hkv": heads[1], "D": heads[2], "type": heads[3],
            "page": page, "e4m3": e4m3, "causal": causal, "window": window}


def _append(name, batch, chunk, keys, heads, page, chunk_lo=0, keys_lo=0, e4m3=False, norm=True, rotated=128,
            interleaved=False):
    return {"name": name, "op": "append", "batch": batch, "chunk_lo": chunk_lo or chunk, "chunk": chunk,
            "keys_lo": keys_lo or keys, "keys": keys, "H": heads[0], "Hkv": heads[1], "D": heads[2], "type": heads[3],
            "page": page, "e4m3": e4m3, "norm": norm, "rotated": rotated, "interleaved": interleaved}


def _read(name, batch, keys, heads, page, keys_lo=0, e4m3=False):
    return {"name": name, "op": "read", "batch": batch, "chunk_lo": 1, "chunk": 1, "keys_lo": keys_lo or keys,
            "keys": keys, "H": heads[0], "Hkv": heads[1], "D": heads[2], "type": heads[3], "page": page, "e4m3": e4m3}


def listed():
    return [
        # one user's next token over a short context: latency
        _attend("token_1x1000", 1, 1, 1000, HEADS[0], 16),
        # a serving batch's next tokens, contexts of all lengths
        _attend("tokens_16x32768_ragged", 16, 1, 32768, HEADS[1], 64, keys_lo=1024),
        # two very long contexts in an 8-bit cache
        _attend("tokens_2x131072_e4m3", 2, 1, 131072, HEADS[0], 128, e4m3=True),
        # a few proposed tokens of each sequence checked at once
        _attend("verify_8x5_8192", 8, 5, 8191, HEADS[2], 32, chunk_lo=2, keys_lo=300),
        # a chunk of a long prompt behind what is already cached
        _attend("chunk_2048_in_32768", 1, 2048, 32768, HEADS[0], 64),
        # prompts and single tokens of several users in one call, an 8-bit cache, a sliding window
        _attend("mixed_6x700_e4m3_window", 6, 700, 6001, HEADS[0], 16, chunk_lo=1, keys_lo=900, e4m3=True, window=4096),
        # decoder tokens over an encoder's states
        _attend("cross_4x448_1500", 4, 448, 1500, (16, 16, 64, "fp16"), 64, causal=False, keys_lo=700),
        # the next token of each sequence of a batch written to the cache
        _append("write_tokens_32", 32, 1, 200, HEADS[0], 16, keys_lo=10),
        # a chunk of a prompt quantised as it is written
        _append("write_8192_e4m3", 1, 8192, 9001, HEADS[0], 64, e4m3=True, norm=False),
        # prompts of several users, part of each head rotated, neighbours paired
        _append("write_4x1500_partial", 4, 1500, 2001, HEADS[1], 32, chunk_lo=333, keys_lo=400, rotated=64,
                interleaved=True),
        # a small batch's cache laid out for the sampler
        _read("read_3x777", 3, 777, HEADS[2], 16, keys_lo=5),
        # a batch of long contexts back from 8 bits
        _read("read_8x32768_e4m3", 8, 32768, HEADS[0], 64, keys_lo=20000, e4m3=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    heads = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128))
    e4m3 = rng.random() < 0.4
    op = rng.choice(("token", "verify", "chunk", "cross", "append", "append", "read"))
    if op in ("token", "verify"):
        keys = _log(rng, 200, 100000)
        batch = max(1, min(_log(rng, 1, 64), 400000 // keys))
        lo = 1 if op == "token" else rng.randint(1, 3)
        hi = 1 if op == "token" else rng.randint(3, 9)
        case = _attend("", batch, hi, keys, heads, page, chunk_lo=lo, keys_lo=max(10, keys // rng.randint(1, 12)),
                       e4m3=e4m3, window=rng.choice((0, 0, _log(rng, 50, keys))))
    elif op == "chunk":
        keys = _log(rng, 300, 30000)
        chunk = min(keys, _log(rng, 17, 2000))
        batch = max(1, min(rng.randint(1, 6), 60000 // keys, 30000000 // (keys * chunk)))
        case = _attend("", batch, chunk, keys, heads, page, chunk_lo=rng.randint(1, chunk),
                       keys_lo=max(chunk, keys // rng.randint(1, 5)), e4m3=e4m3,
                       window=rng.choice((0, 0, _log(rng, 100, keys))))
    elif op == "cross":
        keys, chunk = _log(rng, 60, 3000), _log(rng, 1, 600)
        case = _attend("", rng.randint(1, 8), chunk, keys, heads, page, chunk_lo=rng.randint(1, chunk),
                       keys_lo=max(1, keys // 3), e4m3=e4m3, causal=False)
    elif op == "append":
        chunk = _log(rng, 1, 4000)
        batch = max(1, min(_log(rng, 1, 128), 8000 // chunk))
        keys = chunk + _log(rng, 1, 1000)
        case = _append("", batch, chunk, keys, heads, page, chunk_lo=max(1, chunk // rng.randint(1, 4)),
                       keys_lo=keys - rng.randint(0, keys - chunk), e4m3=e4m3, norm=rng.random() < 0.6,
                       rotated=rng.choice((0, heads[2] // 2, heads[2], heads[2])), interleaved=rng.random() < 0.4)
    else:
        keys = _log(rng, 20, 32768)
        batch = max(1, min(_log(rng, 1, 32), 200000 // keys))
        case = _read("", batch, keys, heads, page, keys_lo=max(1, keys // rng.randint(1, 6)), e4m3=e4m3)
    del case["name"]
    return case


def _lengths(case):
    """(new tokens, keys with them) of each sequence: the case's ranges, the first sequence at their ends."""
    rng = random.Random("%d %d %d %d %d" % (case["batch"], case["chunk_lo"], case["chunk"], case["keys_lo"], case["keys"]))
    n = [case["chunk"]] + [rng.randint(case["chunk_lo"], case["chunk"]) for _ in range(case["batch"] - 1)]
    kv = [case["keys"]] + [rng.randint(case["keys_lo"], case["keys"]) for _ in range(case["batch"] - 1)]
    if case["op"] == "append" or (case["op"] == "attend" and case["causal"]):
        kv = [max(a, b) for a, b in zip(n, kv)]
    return n, kv


def _visible(case):
    """Pairs of a query token and a key that it sees, and keys that some token sees, over the batch."""
    pairs = seen = 0
    for n, kv in zip(*_lengths(case)):
        if not case["causal"]:
            pairs, seen = pairs + n * kv, seen + kv
            continue
        w = case["window"] or kv
        first = kv - n   # position of the first new token
        pairs += sum(min(first + i + 1, w) for i in range(n))
        seen += kv - max(0, first - w + 1)
    return pairs, seen


def work(case):
    n, kv = _lengths(case)
    tokens, keys = sum(n), sum(kv)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    row = Hkv * (D + 4 if case["e4m3"] else 2 * D)   # one row of K or of V in the cache
    if case["op"] == "attend":
        pairs, seen = _visible(case)
        return {"bytes": 2 * seen * row + tokens * H * (4 * D + 4) + 4 * (keys // case["page"]), "flops": 4 * pairs * H * D}
    if case["op"] == "append":
        return {"bytes": tokens * (4 * H * D + 4 * Hkv * D + 2 * row + 4 * case["rotated"]),
                "flops": tokens * (H + Hkv) * D * 8}
    return {"bytes": keys * (2 * row + 4 * Hkv * D), "flops": keys * Hkv * D * 2}


def _quantised(x):
    """e4m3 values and the scale of each row: x is their product, but for the rounding."""
    amax = x.abs().amax(-1, keepdim=True).clamp(min=FLOOR)
    inverse = torch.div(torch.full_like(amax, E4M3_MAX), amax)
    return (x * inverse).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), torch.div(amax, E4M3_MAX).squeeze(-1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    n, kv = _lengths(case)
    B, H, Hkv, D, page = case["batch"], case["H"], case["Hkv"], case["D"], case["page"]
    t = TYPES[case["type"]]
    most = -(-max(kv) // page)
    pages = B * most + 3
    table = torch.randperm(pages, generator=gen, device=dev)[:B * most].view(B, most).to(torch.int32)
    used = torch.tensor([-(-k // page) for k in kv], device=dev)
    table = torch.where(torch.arange(most, device=dev) < used[:, None], table, -1).contiguous()
    s = {"case": case, "t": t, "table": table, "kv": torch.tensor(kv, dtype=torch.int32, device=dev),
         "offsets": torch.tensor([sum(n[:b]) for b in range(B + 1)], device=dev), "nk": max(kv), "max_q": max(n),
         "tokens": sum(n), "total": sum(kv), "uniform": min(n) == max(n)}
    s["q"] = torch.randn(s["tokens"], H, D, generator=gen, device=dev).to(t)

    def pool(planted):
        x = torch.randn(pages * page, Hkv, D, generator=gen, device=dev)
        if planted:   # one key in fifty leans towards a query, as in attention that has learned
            x = x + torch.where(torch.rand(pages * page, 1, 1, generator=gen, device=dev) < 0.02,
                                1.2 * s["q"][0].float().view(Hkv, H // Hkv, D).mean(1), 0.0)
        if not case["e4m3"]:
            return x.to(t).view(pages, page, Hkv, D), None
        code, scale = _quantised(x.to(t).float())
        return code.view(pages, page, Hkv, D), scale.view(pages, page, Hkv).transpose(1, 2).contiguous()

    (s["K"], s["ks"]), (s["V"], s["vs"]) = pool(True), pool(False)
    if case["op"] == "append":
        # the projections of one matrix product: a token's queries, keys and values side by side
        rows = torch.randn(s["tokens"], (H + 2 * Hkv) * D, generator=gen, device=dev).to(t)
        a, b = H * D, (H + Hkv) * D
        s["q"] = rows[:, :a].unflatten(1, (H, D))
        s["k"], s["v"] = rows[:, a:b].unflatten(1, (Hkv, D)), rows[:, b:].unflatten(1, (Hkv, D))
        if case["norm"]:
            s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(t) for _ in range(2))
        if case["rotated"]:
            angle = torch.arange(max(kv), device=dev, dtype=torch.float64)[:, None] * 500000.0 ** (
                -torch.arange(0, case["rotated"], 2, device=dev, dtype=torch.float64) / case["rotated"])
            s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float()   # [positions, rotated / 2, 2]
    if case["op"] == "read":
        s["rows"] = torch.tensor([sum(kv[:b]) for b in range(B + 1)], device=dev)
    if own:
        import stochastic_sparse_decode_split_gb300 as santa
        cache = santa.PagedCache.of(s["K"], s["V"], s["ks"], s["vs"])
        s["step"] = santa.PagedStep(cache, table, s["kv"], n_q_heads=H, dtype=t, nk=s["nk"], max_q=s["max_q"],
                                    total_q=s["tokens"], q_offsets=None if s["uniform"] else s["offsets"],
                                    causal=case.get("causal", True), window=case.get("window", 0))
    return s


def _tokens(s):
    """Of each new token: its sequence, its place in the chunk, its position."""
    n = s["offsets"].diff()
    row = torch.arange(s["tokens"], device=n.device)
    b = torch.searchsorted(s["offsets"], row, right=True) - 1
    i = row - s["offsets"][b]
    return b, i, s["kv"][b] - n[b] + i


def _padded(s, wide):
    """K and V of every sequence, [B, Hkv, keys, D], rows behind the last key zero."""
    B, page = s["table"].shape[0], s["case"]["page"]
    at = s["table"].clamp(min=0).long()
    live = torch.arange(at.shape[1] * page, device=at.device) < s["kv"][:, None]

    def rows(pool, scale):
        x = pool[at].to(wide)
        if scale is not None:
            x = x * scale[at].transpose(2, 3).unsqueeze(-1).to(wide)
        x = x.flatten(1, 2)
        return torch.where(live[..., None, None], x, 0).transpose(1, 2)

    return rows(s["K"], s["ks"]), rows(s["V"], s["vs"]), live


def _plain_attend(s):
    case = s["case"]
    H, Hkv, D, B = case["H"], case["Hkv"], case["D"], case["batch"]
    K, V, live = _padded(s, torch.float32)
    b, i, pos = _tokens(s)
    q = torch.zeros(B, s["max_q"], H, D, device=K.device)
    q[b, i] = s["q"].float()
    q = q.view(B, s["max_q"], Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, K.transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, H // Hkv, s["max_q"], -1)
    key = torch.arange(x.shape[-1], device=x.device)
    where = (s["kv"] - s["offsets"].diff())[:, None] + torch.arange(s["max_q"], device=x.device)
    hidden = ~live[:, None, :]
    if case["causal"]:
        hidden = hidden | (key > where[..., None])
        if case["window"]:
            hidden = hidden | (key <= where[..., None] - case["window"])
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(top.clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, Hkv, -1, x.shape[-1]), V).view(*x.shape[:-1], D) / total.clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], H, D)[b, i]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, s["max_q"], H)[b, i]
    return {"out": out.to(s["t"]), "lse": lse}


def _normed_rotated(s, x, weight, pos, wide):
    case = s["case"]
    x = x.to(wide)
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.to(wide)
    r = case["rotated"]
    if not r:
        return x
    cos, sin = s["rope"][pos.long()].to(wide)[:, None].unbind(-1)
    y = x[..., :r]
    if case["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_append(s):
    b, i, pos = _tokens(s)
    page = s["case"]["page"]
    at, slot = s["table"][b, (pos // page).long()].long(), (pos % page).long()
    q = _normed_rotated(s, s["q"], s.get("qw"), pos, torch.float32).to(s["t"])
    k = _normed_rotated(s, s["k"], s.get("kw"), pos, torch.float32)
    if s["ks"] is None:
        s["K"][at, slot] = k.to(s["t"])
        s["V"][at, slot] = s["v"]
        return {"q": q, "K": s["K"], "V": s["V"]}
    for x, pool, scales in ((k, s["K"], s["ks"]), (s["v"].float(), s["V"], s["vs"])):
        code, scale = _quantised(x)
        pool.view(torch.uint8)[at, slot] = code.view(torch.uint8)
        scales[at, :, slot] = scale
    return {"q": q, "K": s["K"], "V": s["V"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _plain_read(s):
    K, V, live = _padded(s, torch.float32)
    return {"K": K.transpose(1, 2)[live].to(s["t"]), "V": V.transpose(1, 2)[live].to(s["t"])}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "read": _plain_read}[op](s)
    step = s["step"]
    if op == "attend":
        out, lse = step.attend(s["q"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "read":
        K, V = step.read(s["rows"], s["total"])
        return {"K": K, "V": V}
    q = step.append(s["q"], s["k"], s["v"], rope=s.get("rope"), interleaved=s["case"]["interleaved"],
                    q_norm=s.get("qw"), k_norm=s.get("kw"), eps=1e-6)
    if s["ks"] is None:
        return {"q": q, "K": s["K"], "V": s["V"]}
    return {"q": q, "K": s["K"], "V": s["V"], "k_scale": s["ks"], "v_scale": s["vs"]}


def exact(case, seed):
    """In 64 bits, one sequence after another."""
    s = prepare(case, seed)
    n, kv = _lengths(case)
    B, H, Hkv, D, page = case["batch"], case["H"], case["Hkv"], case["D"], case["page"]
    d = torch.float64

    def rows(pool, scale, b):   # [keys, Hkv, D]
        at = s["table"][b, :-(-kv[b] // page)].long()
        x = pool[at].to(d)
        if scale is not None:
            x = x * scale[at].to(d).permute(0, 2, 1)[..., None]
        return x.reshape(-1, Hkv, D)[:kv[b]]

    if case["op"] == "read":
        return {"K": torch.cat([rows(s["K"], s["ks"], b) for b in range(B)]),
                "V": torch.cat([rows(s["V"], s["vs"], b) for b in range(B)])}
    if case["op"] == "attend":
        outs, lses, first = [], [], 0
        for b in range(B):
            K, V = rows(s["K"], s["ks"], b), rows(s["V"], s["vs"], b)
            pos = torch.arange(kv[b] - n[b], kv[b], device=K.device)[:, None]
            key = torch.arange(kv[b], device=K.device)
            keep = torch.ones(n[b], kv[b], dtype=torch.bool, device=K.device)
            if case["causal"]:
                keep = (key <= pos) & (key > pos - (case["window"] or kv[b] + 1))
            out, lse = torch.empty(n[b], H, D, dtype=d, device=K.device), torch.empty(n[b], H, dtype=d, device=K.device)
            for h in range(H):
                x = s["q"][first:first + n[b], h].to(d) @ K[:, h * Hkv // H].T / D ** 0.5
                x = torch.where(keep, x, float("-inf"))
                lse[:, h] = torch.logsumexp(x, -1)
                out[:, h] = torch.exp(x - lse[:, h, None]) @ V[:, h * Hkv // H]
            outs.append(out)
            lses.append(lse)
            first += n[b]
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    b, i, pos = _tokens(s)

    def turned(x, weight):
        x = x.to(d)
        if weight is not None:
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.to(d)
        r = case["rotated"]
        if r:
            z = torch.view_as_complex(s["rope"].to(d).contiguous())[pos.long()][:, None]
            y = x[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
            y = torch.view_as_complex((y if case["interleaved"] else y.transpose(-1, -2)).contiguous())
            y = torch.view_as_real(y * z)
            x = torch.cat(((y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2), x[..., r:]), -1)
        return x

    at, slot = s["table"][b, (pos // page).long()].long(), (pos % page).long()
    got = {"q": turned(s["q"], s.get("qw"))}
    for name, x in (("K", turned(s["k"], s.get("kw"))), ("V", s["v"].to(d))):
        pool = s[name].to(d)
        if case["e4m3"]:
            scale = x.abs().amax(-1).clamp(min=FLOOR) / E4M3_MAX
            pool[at, slot] = x / scale[..., None]
            scales = s[{"K": "ks", "V": "vs"}[name]].to(d)
            scales[at, :, slot] = scale
            got[{"K": "k_scale", "V": "v_scale"}[name]] = scales
        else:
            pool[at, slot] = x
        got[name] = pool
    return got
