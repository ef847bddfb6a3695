"""Calls of joined attention that are meant for one kernel: (what ``route`` takes, the kernels that it is to go to[, the
fewest blocks of 128 keys that a CTA has on the whole]).  The GPU tests run them, a host test checks the way that they
take."""

# differential chunks and prefix passes of many blocks per CTA
LONG_PIECES = [
    (dict(kv=[4000], n=[1200], H=8, Hkv=2, D=128, page=32, diff=True), ["own:{wide}"], 8),
    (dict(kv=[2500, 3000, 700], n=[900, 1000, 700], H=14, Hkv=2, D=128, page=64, diff=True), ["own:{wide}"], 8),
    (dict(kv=[30 + 3 * i for i in range(40)], n=[1] * 40, H=16, Hkv=4, D=128, page=128, diff=True, prefix=[40000], first=[0, 40]),
     ["prefix:{wide}", "own:tokens"], 8),
    (dict(kv=[3000], n=[1000], H=16, Hkv=4, D=64, page=16, diff=True), ["own:chunk"], 4),
]

# chunks behind prefixes, whose first block of 128 keys begins before pages that lie wholly inside the prefix
OWN_CHUNKS = [
    (dict(kv=[400, 310, 333], n=[300, 310, 200], H=32, Hkv=8, D=128, page=16, prefix=[192], first=[0, 3]), ["prefix:chunk", "own:chunk"]),
    (dict(kv=[500, 420, 600, 380], n=[400, 300, 450, 200], H=16, Hkv=8, D=64, page=32, prefix=[250, 1000], first=[0, 2, 4]),
     ["prefix:chunk", "own:chunk"]),
    (dict(kv=[700, 450, 651], n=[500, 450, 300], H=28, Hkv=4, D=128, page=64, prefix=[1000], first=[0, 3]), ["prefix:chunk", "own:chunk"]),
    (dict(kv=[390, 2, 300, 640], n=[380, 1, 290, 333], H=32, Hkv=16, D=64, page=16, prefix=[0, 127], first=[0, 1, 4]),
     ["prefix:chunk", "own:chunk"]),
    (dict(kv=[400, 310, 333], n=[300, 310, 200], H=8, Hkv=2, D=128, page=16, prefix=[1216], first=[0, 3], diff=True),
     ["prefix:{wide}", "own:{wide}"]),
    (dict(kv=[500, 420, 600, 380], n=[400, 300, 450, 200], H=8, Hkv=4, D=64, page=32, prefix=[250, 1000], first=[0, 2, 4], diff=True),
     ["prefix:chunk", "own:chunk"]),
    (dict(kv=[700, 450, 651], n=[500, 450, 300], H=14, Hkv=2, D=128, page=64, prefix=[1000], first=[0, 3], diff=True),
     ["prefix:{wide}", "own:{wide}"]),
    (dict(kv=[400, 310, 333], n=[300, 310, 200], H=32, Hkv=8, D=128, page=16, prefix=[20], first=[0, 3]), ["prefix:tokens", "own:chunk"]),
    (dict(kv=[400, 310, 333], n=[300, 310, 200], H=8, Hkv=2, D=128, page=16, prefix=[20], first=[0, 3], diff=True),
     ["prefix:tokens", "own:{wide}"]),
]

# every form of the chunk kernels, for what goes beyond lengths: odd values, bad pages, padding, replays
FORMS = [
    OWN_CHUNKS[1], OWN_CHUNKS[2], OWN_CHUNKS[5], OWN_CHUNKS[6],
    (dict(kv=[2000, 1500], n=[700, 400], H=8, Hkv=2, D=128, page=32, diff=True), ["own:{wide}"]),
    (dict(kv=[2000, 1500], n=[700, 400], H=8, Hkv=2, D=64, page=16, diff=True), ["own:chunk"]),
]

# differential chunks in a window, unmasked, and with rows that see nothing
WINDOWS = [(dict(kv=[2500, 900], n=[700, 300], H=8, Hkv=2, D=D, page=page, diff=True, window=w), ["own:{wide}" if D == 128 else "own:chunk"])
           for D, page in ((128, 32), (64, 16)) for w in (1, 16, 100, 128, 1000)]
UNMASKED = [
    (dict(kv=[1500, 5, 700], n=[448, 300, 200], H=16, Hkv=4, D=128, page=64, diff=True, causal=False), ["own:{wide}"]),
    (dict(kv=[1500, 5, 700], n=[448, 300, 200], H=16, Hkv=4, D=64, page=16, diff=True, causal=False), ["own:chunk"]),
    (dict(kv=[300, 5, 420], n=[448, 600, 200], H=16, Hkv=8, D=128, page=16, prefix=[250], first=[0, 3], causal=False), ["prefix:chunk", "own:chunk"]),
    (dict(kv=[300, 5, 420], n=[448, 600, 200], H=16, Hkv=4, D=64, page=32, prefix=[250], first=[0, 3], causal=False, diff=True),
     ["prefix:chunk", "own:chunk"]),
    (dict(kv=[300, 5, 420], n=[448, 600, 200], H=16, Hkv=4, D=128, page=16, prefix=[1400], first=[0, 3], causal=False, diff=True),
     ["prefix:{wide}", "own:{wide}"]),
]
NOTHING_SEEN = [
    (dict(kv=[0, 40, 698, 600], n=[700, 700, 700, 1], H=8, Hkv=2, D=D, page=page, diff=True), ["own:{wide}" if D == 128 else "own:chunk"])
    for D, page in ((128, 32), (64, 16))]


def kernels(case, e4m3):
    """The names, with {wide} the kernel for heads of 128 over 16 bits."""
    return [x.format(wide="chunk" if e4m3 else "wide") for x in case[1]]


def blocks_per_cta(case, e4m3, ctas=152):
    """Blocks of a differential call's chunk pass (its first) over its CTAs."""
    c = case[0]
    G, parts = c["H"] // c["Hkv"], 1
    per, items = 128 // G, c["Hkv"] // 2
    if e4m3 or c["D"] == 128:
        parts = 2
    if "prefix" in c:
        total = sum(-(-p // 128) * -(-sum(c["n"][a:b]) // per) for p, a, b in zip(c["prefix"], c["first"], c["first"][1:]))
    else:
        total = 0
        for kv, n in zip(c["kv"], c["n"]):
            total += sum(-(-(kv - n + min(n, i + per)) // 128) for i in range(0, n, per))
    return total * items * parts / ctas
