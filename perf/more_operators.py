"""The paged cache's further operators, case by case: what each is given, its plain form in elementary
torch operations, the framework's own call, the work that it cannot do without, and its exact result in
64 bits.

Four kinds of case:
  rotate  the new tokens' keys and values written into the pages, the keys and the queries turned by
          their positions on the way (a draft tree's nodes by their depth)
  window  attention of the new tokens over the last `window` positions and the first `sinks` ones
  shared  attention of a batch whose requests share the pages of a long prefix, read once for all
  share   which requests share a prefix, from the page table: the plan that the attention above takes
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
POSITIONS = 32768  # rows of the rotation table


def listed():
    return [
        # a decoding step's rows with a few drafts each: latency
        dict(name="rotate-decode", kind="rotate", B=32, n_min=1, n_max=9, tree=False, ctx_min=0, ctx_max=900, hkv=8,
             group=4, d=128, rotary=128, interleaved=False, page=16, dtype="bf16", layout=1),
        # draft trees, positions by depth, a part of each head turned, neighbouring elements paired
        dict(name="rotate-tree", kind="rotate", B=64, n_min=20, n_max=64, tree=True, ctx_min=100, ctx_max=700, hkv=4,
             group=7, d=80, rotary=32, interleaved=True, page=24, dtype="f16", layout=2),
        # prompt chunks: bandwidth
        dict(name="rotate-prompt", kind="rotate", B=6, n_min=2000, n_max=5000, tree=False, ctx_min=0, ctx_max=3000,
             hkv=8, group=4, d=128, rotary=128, interleaved=False, page=32, dtype="bf16", layout=3),
        # one user's long conversation, one token: the latency of a single decoding step
        dict(name="window-one-token", kind="window", B=1, n_min=1, n_max=1, tree=False, ctx_min=20000, ctx_max=20000,
             window=1024, sinks=4, hkv=8, group=4, d=128, page=16, dtype="bf16", layout=4),
        # a batch in plain decoding, contexts below and far above the window
        dict(name="window-decode", kind="window", B=64, n_min=1, n_max=1, tree=False, ctx_min=1, ctx_max=20000,
             window=4096, sinks=4, hkv=8, group=4, d=128, page=16, dtype="bf16", layout=5),
        # draft trees over a short window, an odd number of query heads per kv head, small heads
        dict(name="window-tree", kind="window", B=24, n_min=20, n_max=64, tree=True, ctx_min=500, ctx_max=2600,
             window=300, sinks=70, hkv=4, group=7, d=64, page=64, dtype="f16", layout=6),
        # chunks of two prompts: every token has a window of its own
        dict(name="window-prompt", kind="window", B=2, n_min=1500, n_max=2111, tree=False, ctx_min=4000, ctx_max=6100,
             window=1024, sinks=16, hkv=8, group=4, d=128, page=32, dtype="bf16", layout=7),
        # a few samples of one prompt: latency
        dict(name="shared-few", kind="shared", B=8, groups=1, prefix_min=2000, prefix_max=2000, n_min=1, n_max=1,
             tree=False, ctx_min=1, ctx_max=60, hkv=8, group=4, d=128, page=16, dtype="bf16", layout=8),
        # two system prompts under a batch in plain decoding
        dict(name="shared-decode", kind="shared", B=64, groups=2, prefix_min=8000, prefix_max=9000, n_min=1, n_max=1,
             tree=False, ctx_min=1, ctx_max=500, hkv=8, group=4, d=128, page=16, dtype="bf16", layout=9),
        # the verify step of 128 requests with 8 drafts each, behind four documents
        dict(name="shared-verify", kind="shared", B=128, groups=4, prefix_min=3000, prefix_max=12000, n_min=9, n_max=9,
             tree=False, ctx_min=0, ctx_max=1000, hkv=8, group=4, d=128, page=32, dtype="bf16", layout=10),
        # the plan of a few samples
        dict(name="share-few", kind="share", B=9, groups=2, prefix_min=300, prefix_max=2000, ctx_min=1, ctx_max=100,
             page=16, min_tokens=256, layout=11),
        # the plan of a large batch with long prefixes
        dict(name="share-many", kind="share", B=512, groups=24, prefix_min=500, prefix_max=30000, ctx_min=1,
             ctx_max=2000, page=16, min_tokens=256, layout=12),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One case of the listed ones' ranges, drawn again where it would cost more than they do."""
    case = _drawn(rng)
    while not _affordable(case):
        case = _drawn(rng)
    return case


def _affordable(case):
    n, ctx, _ = _sizes(case)
    if case["kind"] in ("rotate", "share"):
        return sum(n) < 24000 and sum(ctx) < 8e6
    keys = max(ctx) + max(n)
    if case["kind"] == "window":
        keys = min(keys, case["window"] + case["sinks"] + max(n))
    scores = len(n) * case["hkv"] * case["group"] * max(max(n), 1) * keys
    gathered = len(n) * keys * case["hkv"] * case["d"]
    cost = work(case)
    stored = sum(ctx) * case["hkv"] * case["d"] * 4 if case["kind"] == "window" else 0
    return cost["bytes"] < 1.05e9 and cost["flops"] < 1.3e11 and scores < 2e9 and gathered < 1.4e9 and stored < 3e9


def _drawn(rng):
    kind = rng.choice(["rotate", "window", "window", "shared", "shared", "share"])
    case = dict(kind=kind, page=rng.choice([8, 16, 24, 32, 64, 128]), layout=rng.randrange(1 << 20))
    if kind == "share":
        case["B"] = _log_uniform(rng, 1, 512)
        case["groups"] = rng.randint(1, case["B"])
        case["prefix_max"] = _log_uniform(rng, 1, 30000)
        case["prefix_min"] = rng.randint(0, case["prefix_max"])
        case["ctx_min"], case["ctx_max"] = 0, _log_uniform(rng, 1, 2000)
        case["min_tokens"] = rng.choice([0, 128, 256, 1000])
        return case
    case.update(hkv=rng.choice([1, 2, 3, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 7, 8]), dtype=rng.choice(["bf16", "f16"]),
                d=rng.choice([64, 80, 96, 128]), tree=rng.random() < 0.3)
    if kind == "rotate":
        case["rotary"] = rng.choice([16, 32, 64, case["d"]])
        case["interleaved"] = rng.random() < 0.5
        case["B"] = _log_uniform(rng, 1, 128)
        case["n_max"] = rng.randint(1, 100) if case["tree"] else _log_uniform(rng, 1, 20000 // case["B"])
        case["n_min"] = rng.randint(0, case["n_max"])
        case["ctx_min"], case["ctx_max"] = 0, _log_uniform(rng, 10, 1000)
        return case
    form = "tree" if case["tree"] else rng.choice(["decode", "verify", "verify", "prompt"])
    if form == "decode":
        case["n_min"] = case["n_max"] = 1
    elif form == "verify":
        case["n_min"], case["n_max"] = rng.choice([(0, 9), (1, 33), (5, 5), (0, 3)])
    elif form == "tree":
        case["n_min"], case["n_max"] = rng.choice([(1, 64), (17, 100), (64, 64)])
    else:
        case["n_max"] = _log_uniform(rng, 100, 2000 if kind == "window" else 300)
        case["n_min"] = rng.randint(1, case["n_max"])
    most = 3 if form == "prompt" else 96
    if kind == "window":
        case["B"] = _log_uniform(rng, 1, most)
        case["ctx_max"] = _log_uniform(rng, 20, min(20000, 600000 // case["B"]))
        case["ctx_min"] = rng.randint(0, case["ctx_max"])
        case["window"] = _log_uniform(rng, 1, 8192)
        case["sinks"] = rng.choice([0, 1, 4, 16, 64, 130, 300])
    else:
        case["B"] = _log_uniform(rng, 2, 12 if form == "prompt" else 128)
        case["groups"] = _log_uniform(rng, 1, max(1, case["B"] // 2))
        case["prefix_max"] = _log_uniform(rng, 100, min(12000, 600000 // case["B"]))
        case["prefix_min"] = rng.randint(0, case["prefix_max"])
        case["ctx_min"], case["ctx_max"] = 0, _log_uniform(rng, 1, 1000)
    return case


# ---------------------------------------------------------------------------------------
# Shapes that follow from the case alone
# ---------------------------------------------------------------------------------------


def _sizes(case):
    """Per request: new tokens, committed tokens; the groups (first request, end, shared tokens)."""
    rng = random.Random(case["layout"])
    B = case["B"]
    n = [rng.randint(case.get("n_min", 0), case.get("n_max", 0)) for _ in range(B)]
    ctx = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in range(B)]
    groups = []
    if "groups" in case:
        cuts = [0] + sorted(rng.sample(range(1, B), case["groups"] - 1)) + [B]
        for a, b in zip(cuts, cuts[1:]):
            tokens = rng.randint(case["prefix_min"], case["prefix_max"]) // case["page"] * case["page"]
            groups.append((a, b, tokens))
            for r in range(a, b):
                ctx[r] += tokens
    return n, ctx, groups


def _trees(case, n):
    """Draft trees as level-order drafting makes them: a parent index per node (-1 at the root)."""
    rng = random.Random(case["layout"] + 1)
    parent = []
    for size in n:
        par = [-1] * min(size, 1)
        for i in range(1, size):
            par.append(rng.randint(max(0, (i - 1) // 4 - 1), max(0, (i - 1) // 2)))
        parent += par
    return parent


def _pages(tokens, page):
    return -(-tokens // page)


def _depths(parent, n):
    depth, at = [], 0
    for m in n:
        for i in range(m):
            depth.append(0 if parent[at + i] < 0 else depth[at + parent[at + i]] + 1)
        at += m
    return depth


def work(case):
    n, ctx, groups = _sizes(case)
    if case["kind"] == "share":
        compared = sum(min(ctx[r - 1], ctx[r]) // case["page"] for a, b, tokens in groups if tokens
                       for r in range(a + 1, b))
        return {"bytes": 4 * (2 * compared + case["B"]) + 16 * case["B"], "flops": 0}
    N, hkv, d = sum(n), case["hkv"], case["d"]
    hq = hkv * case["group"]
    row = 2 * hkv * d * 2  # one token's keys and values in one layer
    depth = _depths(_trees(case, n), n) if case["tree"] else [i for m in n for i in range(m)]
    if case["kind"] == "rotate":
        at, positions = 0, set()
        for c, m in zip(ctx, n):
            positions.update(c + i for i in depth[at:at + m])
            at += m
        return {"bytes": 2 * N * (row + hq * d * 2) + len(positions) * case["rotary"] * 4,
                "flops": 3 * N * (hq + hkv) * case["rotary"]}
    seen, keys, at = 0, 0, 0
    W, S = case.get("window", 1 << 30), case.get("sinks", 0)
    for c, m in zip(ctx, n):
        low = c
        for i in depth[at:at + m]:
            # of the context, the sinks and the window's; of the new tokens on the way to this one, the last W
            lo = min(c, max(0, c + i - W + 1))
            low = min(low, lo)
            seen += c - max(0, lo - S) if lo > S else c
            seen += min(i + 1, max(W, 1)) if c >= S else i + 1
        if m:
            keys += m + (c - max(0, low - S) if low > S else c)
        at += m
    keys -= sum(tokens * (sum(n[r] > 0 for r in range(a, b)) - 1) for a, b, tokens in groups if any(n[a:b]))
    return {"bytes": keys * row + 2 * N * hq * d * 2, "flops": 4 * d * hq * seen}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = random.Random(seed)
    n, ctx, groups = _sizes(case)
    page, hkv, d = case["page"], case.get("hkv", 1), case.get("d", 8)
    dt = DTYPES[case.get("dtype", "bf16")]
    R, N = len(n), sum(n)
    need = [_pages(c + m, page) for c, m in zip(ctx, n)]
    shared = [0] * R  # leading pages that are the group's
    for a, b, tokens in groups:
        shared[a:b] = [tokens // page] * (b - a)
        if case["kind"] == "share":  # branches that left the prefix before its end
            shared[a:b] = [x - host.randint(0, x // 8) for x in shared[a:b]]
    max_pages = max(max(need), 1)
    total = sum(need) - sum(shared) + sum(tokens // page for _, _, tokens in groups)
    num_pages = total + 3
    order = list(range(num_pages))
    host.shuffle(order)
    table = [[-1] * max_pages for _ in range(R)]
    ref, used = [0] * num_pages, 0
    for a, b, tokens in groups:
        pages = order[used:used + tokens // page]
        used += len(pages)
        for r in range(a, b):
            table[r][:shared[r]] = pages[:shared[r]]
    for r in range(R):
        table[r][shared[r]:need[r]] = order[used:used + need[r] - shared[r]]
        used += need[r] - shared[r]
        for p in table[r][:need[r]]:
            ref[p] += 1
    free = sorted(order[used:])
    s = dict(kind=case["kind"], page=page, hkv=hkv, d=d, n=n, ctx=ctx, total=N, most=max(max(n), 1),
             keys=max(max(c + m for c, m in zip(ctx, n)), 1))
    kv = torch.empty((1, num_pages, 2, page, hkv, d), dtype=dt, device="cuda")
    if case["kind"] == "share":
        kv.zero_()
    else:
        for i in range(0, num_pages, 4096):
            part = kv[:, i:i + 4096]
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    s["table"], s["held"], s["ref"], s["lens"] = _ints(table), _ints(need), _ints(ref), _ints(ctx)
    s["free"], s["num_free"] = _ints(free + [0] * (num_pages - len(free))), _ints([len(free)])
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    s["cu"], s["parent"] = _ints(cu), None
    if case["kind"] == "share":
        s["min_tokens"] = case["min_tokens"]
        return s
    s["group"], s["scale"] = case["group"], 1.0 / math.sqrt(d)
    # scores of standard deviation 2: softmax rows neither flat nor one-hot
    s["q"] = (2 * torch.randn((N, hkv * case["group"], d), generator=gen, device="cuda")).to(dt)
    if case["tree"]:
        s["parent"] = _ints(_trees(case, n))
    if case["kind"] == "rotate":
        s["k_new"] = torch.randn((N, hkv, d), generator=gen, device="cuda").to(dt)
        s["v_new"] = torch.randn((N, hkv, d), generator=gen, device="cuda").to(dt)
        s["interleaved"], half = case["interleaved"], case["rotary"] // 2
        speed = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(POSITIONS, dtype=torch.float64, device="cuda")[:, None] * speed
        s["rotation"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if case["kind"] == "window":
        s["window"], s["sinks"] = case["window"], case["sinks"]
    if case["kind"] == "shared":
        # made once for the steps of these requests: per request its group and the tokens that are shared
        plan = [(r, r + 1, 0, 0) for r in range(R)]
        for a, b, tokens in groups:
            if b - a > 1 and tokens:
                plan[a:b] = [(a, b, tokens, 0)] * (b - a)
        s["plan"] = _ints(plan)
    return s


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------


def run(state):
    if own:
        return _OWN[state["kind"]](state)
    return _PLAIN[state["kind"]](state)


def _handle(s):
    """The framework's cache over the state's tensors, made once, as a serving program keeps it."""
    from speculative_decoding_rejection_spec_gb300 import cache
    if "handle" not in s:
        s["handle"] = cache.PagedCache(s["k"], s["v"], page_table=s["table"], lens=s["lens"], held=s["held"],
                                       ref_counts=s["ref"], free_pages=s["free"], num_free=s["num_free"])
    return cache, s["handle"]


def _own_rotate(s):
    cache, c = _handle(s)
    q = cache.append_rotated(c, 0, s["q"], s["k_new"], s["v_new"], s["cu"], s["rotation"], parent=s["parent"],
                             interleaved=s["interleaved"])
    return q, s["k"], s["v"]


def _own_window(s):
    cache, c = _handle(s)
    return cache.attention(c, 0, s["q"], s["cu"], parent=s["parent"], scale=s["scale"], window=s["window"],
                           sinks=s["sinks"])


def _own_shared(s):
    cache, c = _handle(s)
    return cache.attention(c, 0, s["q"], s["cu"], parent=s["parent"], scale=s["scale"], shared=s["plan"])


def _own_share(s):
    cache, c = _handle(s)
    return cache.share(c, min_tokens=s["min_tokens"])


_OWN = dict(rotate=_own_rotate, window=_own_window, shared=_own_shared, share=_own_share)


def _request_of(s):
    """Per new token: its request, its index there."""
    counts = (s["cu"][1:] - s["cu"][:-1]).long()
    request = torch.repeat_interleave(torch.arange(len(s["n"]), device="cuda"), counts, output_size=s["total"])
    return request, torch.arange(s["total"], device="cuda") - s["cu"].long()[request]


def _reach(s, request, index):
    """[requests, most, most]: whether node i is j or has it among its ancestors."""
    most = s["most"]
    reach = torch.zeros((len(s["n"]), most, most), device="cuda")
    i = torch.arange(most, device="cuda")
    reach[:, i, i] = 1
    reach[request, index, torch.where(s["parent"] < 0, index, s["parent"].long())] = 1
    for _ in range(max(1, (most - 1).bit_length())):
        reach = (reach @ reach).clamp_(max=1)
    return reach


def _plain_rotate(s):
    request, index = _request_of(s)
    depth = index
    if s["parent"] is not None:
        depth = _reach(s, request, index).sum(-1).long()[request, index] - 1
    lens = s["lens"].long()[request]
    table = s["rotation"][lens + depth][:, None, :]
    half = table.shape[-1] // 2
    cos, sin = table[..., :half], table[..., half:]

    def turned(x):
        x = x.float()
        y = x.clone()
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"] else (slice(half), slice(half, 2 * half))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        return y.to(s["q"].dtype)

    page, row = s["table"].long()[request, (lens + index) // s["page"]], (lens + index) % s["page"]
    s["k"][0][page, row] = turned(s["k_new"])
    s["v"][0][page, row] = s["v_new"]
    return turned(s["q"]), s["k"], s["v"]


def _plain_attention(s):
    R, most, hkv, G, d = len(s["n"]), s["most"], s["hkv"], s["group"], s["d"]
    W, S = s.get("window", 1 << 30), s.get("sinks", 0)
    lens = s["lens"].long()[:, None]
    # the keys that any row of a request may see: the sinks, then the window of the first row and what follows
    low = (lens - W + 1).clamp(min=S)
    span = min(s["keys"], W + most)
    t = torch.cat([torch.arange(S, device="cuda").expand(R, S), low + torch.arange(span, device="cuda")], 1)
    if W > s["keys"]:
        t = torch.arange(s["keys"], device="cuda").expand(R, s["keys"])
    pages = s["table"].long().gather(1, (t // s["page"]).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k = s["k"][0][pages, t % s["page"]].float().permute(0, 2, 1, 3)
    v = s["v"][0][pages, t % s["page"]].float().permute(0, 2, 1, 3)
    request, index = _request_of(s)
    q = torch.zeros((R, most, hkv, G, d), device="cuda")
    q[request, index] = s["q"].float().view(-1, hkv, G, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(R, hkv, most * G, d)
    scores = (q @ k.transpose(2, 3)).mul_(s["scale"])
    new = t - lens  # position among the new tokens, below zero in the context
    i = torch.arange(most, device="cuda")
    if s["parent"] is None:
        depth = i.expand(R, most)
        among = new[:, None, :] <= i[None, :, None]
        place = t
    else:
        reach = _reach(s, request, index)
        depth = reach.sum(-1).long() - 1
        clamped = new.clamp(0, most - 1)
        among = reach.gather(2, clamped[:, None, :].expand(R, most, t.shape[1])) > 0
        place = torch.where(new < 0, t, lens + depth.gather(1, clamped))  # positions, by depth
    # rows of no token (requests of fewer tokens than the longest) see what is there, and are dropped
    seen = (new < 0)[:, None, :] | (among & (new < most)[:, None, :])
    seen &= (place < S)[:, None, :] | (place[:, None, :] > (lens + depth)[:, :, None] - W)
    hidden = ~seen[:, None, :, None, :].expand(R, hkv, most, G, t.shape[1]).reshape(R, hkv, most * G, t.shape[1])
    scores.masked_fill_(hidden, -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    out = (scores @ v) / scores.sum(-1, keepdim=True)
    out = out.view(R, hkv, most, G, d).permute(0, 2, 1, 3, 4)[request, index]
    return out.reshape(s["total"], hkv * G, d).to(s["q"].dtype)


def _plain_share(s):
    table, page = s["table"], s["page"]
    R = table.shape[0]
    r = torch.arange(R, device="cuda")
    full = torch.minimum(s["lens"][1:], s["lens"][:-1]).long() // page
    column = torch.arange(table.shape[1], device="cuda")
    differs = (table[1:] != table[:-1]) | (column >= full[:, None])
    common = torch.where(differs, column, table.shape[1]).amin(1) if R > 1 else full
    linked = torch.zeros(R + 1, dtype=torch.bool, device="cuda")  # with the request before
    linked[1:R] = common * page >= max(s["min_tokens"], 1)
    first = torch.where(linked[:R], 0, r).cummax(0).values
    end = R - torch.where(linked[1:], 0, R - 1 - r).flip(0).cummax(0).values.flip(0)
    tokens = torch.full((R,), 1 << 30, device="cuda", dtype=torch.long)
    tokens[1:] = torch.where(linked[1:R], common * page, 1 << 30)
    tokens = tokens.scatter_reduce(0, first, tokens, "amin")[first]
    tokens = torch.where(end - first > 1, tokens, 0)
    return torch.stack([first, end, tokens, torch.zeros_like(first)], 1).int()


_PLAIN = dict(rotate=_plain_rotate, window=_plain_attention, shared=_plain_attention, share=_plain_share)


# ---------------------------------------------------------------------------------------
# Exact results
# ---------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return dict(rotate=_exact_rotate, window=_exact_attention, shared=_exact_attention,
                share=_exact_share)[case["kind"]](case, s)


def _exact_rotate(case, s):
    n, ctx, page = s["n"], s["ctx"], case["page"]
    table = s["table"].tolist()
    depth = _depths(s["parent"].tolist(), n) if case["tree"] else [i for m in n for i in range(m)]
    pages, rows, positions, at = [], [], [], 0
    for r, m in enumerate(n):
        for i in range(m):
            pages.append(table[r][(ctx[r] + i) // page])
            rows.append((ctx[r] + i) % page)
            positions.append(ctx[r] + depth[at + i])
        at += m
    # a pair of elements is a complex number, its turn another one
    angles = s["rotation"].double()[torch.tensor(positions, dtype=torch.long, device="cuda")]
    half = case["rotary"] // 2
    turn = torch.complex(angles[:, :half].contiguous(), angles[:, half:].contiguous())[:, None, :]
    results = []
    for x in (s["q"].double(), s["k_new"].double()):
        head, rest = x[..., :2 * half], x[..., 2 * half:]
        if case["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) * turn
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn
            head = torch.cat([z.real, z.imag], -1)
        results.append(torch.cat([head, rest], -1))
    k, v = s["k"].double(), s["v"].double()
    if pages:
        k[0, pages, rows] = results[1]
        v[0, pages, rows] = s["v_new"].double()
    return results[0], k, v


def _exact_attention(case, s):
    n, ctx, page, G, H, d = s["n"], s["ctx"], case["page"], case["group"], case["hkv"], case["d"]
    W, S = case.get("window"), case.get("sinks", 0)
    parent = s["parent"].tolist() if s["parent"] is not None else None
    table = s["table"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for r, m in enumerate(n):
        if not m:
            continue
        c, L = ctx[r], ctx[r] + m
        pages = torch.tensor(table[r][:_pages(L, page)], device="cuda")
        among = torch.tril(torch.ones((m, m), dtype=torch.bool))
        depth = torch.arange(m)
        if parent is not None:
            among = torch.zeros((m, m), dtype=torch.bool)
            for i in range(m):
                if parent[at + i] >= 0:
                    among[i] = among[parent[at + i]]
                among[i, i] = True
            depth = among.sum(1) - 1
        seen = torch.cat([torch.ones((m, c), dtype=torch.bool), among], 1)
        if W is not None:
            place = torch.cat([torch.arange(c), c + depth])
            seen &= (place < S)[None, :] | ((c + depth)[:, None] - place[None, :] < W)
        cols = seen.any(0).nonzero().squeeze(1).cuda()
        seen = seen.cuda()[:, cols]
        where = pages[cols // page], cols % page
        k, v = s["k"][0][where].double(), s["v"][0][where].double()
        q = s["q"][at:at + m].double().view(m, H, G, d)
        for h in range(H):
            x = torch.einsum("igd,td->igt", q[:, h], k[:, h]) * s["scale"]
            x = x.masked_fill(~seen[:, None, :], -math.inf)
            x = torch.exp(x - x.max(-1, keepdim=True).values)
            out[at:at + m, h * G:(h + 1) * G] = torch.einsum("igt,td->igd", x, v[:, h]) / x.sum(-1, keepdim=True)
        at += m
    return out


def _exact_share(case, s):
    table, lens, page = s["table"].tolist(), s["lens"].tolist(), case["page"]
    R, plan, first = len(lens), [], 0
    common = [0] * R
    for r in range(1, R):
        full = min(lens[r], lens[r - 1]) // page
        while common[r] < full and table[r][common[r]] == table[r - 1][common[r]]:
            common[r] += 1
    least = max(case["min_tokens"], 1)
    while first < R:
        end = first + 1
        while end < R and common[end] * page >= least:
            end += 1
        tokens = min(common[first + 1:end]) * page if end - first > 1 else 0
        plan += [(first, end, tokens, 0)] * (end - first)
        first = end
    return _ints(plan)
