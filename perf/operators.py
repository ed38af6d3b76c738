"""The paged key/value cache's operators, case by case: what each is given, its plain form in
elementary torch operations, the framework's own call, the work that it cannot do without, and its
exact result in 64 bits.

Four kinds of case:
  attention  attention of the new tokens of every request (a chain of drafts, a draft tree, a prompt
             chunk, a single token) over its cached context, in the pages that a table names
  append     the new tokens' keys and values written into the pages, behind the committed tokens
  commit     one step's rows appended in every layer, then the step committed: lengths advance by the
             accepted path, whose rows move together
  pages      the branches of the last step released, new ones forked, room for their new tokens
             reserved (a shared last page is copied before it is written)
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one user's request, one token: the latency of a single decoding step
        dict(name="attention-one-token", kind="attention", B=1, n_min=1, n_max=1, tree=False, ctx_min=700, ctx_max=700,
             hkv=8, group=4, d=128, page=16, dtype="bf16", layout=1),
        # a batch in plain decoding, contexts of very different lengths
        dict(name="attention-decode", kind="attention", B=64, n_min=1, n_max=1, tree=False, ctx_min=1, ctx_max=8191,
             hkv=8, group=4, d=128, page=16, dtype="bf16", layout=2),
        # the verify step of 128 requests with 8 drafts each (the large-128 batch)
        dict(name="attention-verify", kind="attention", B=128, n_min=9, n_max=9, tree=False, ctx_min=200, ctx_max=4000,
             hkv=8, group=4, d=128, page=32, dtype="bf16", layout=3),
        # draft trees of up to 64 nodes, fp16, an odd number of query heads per kv head, small heads
        dict(name="attention-tree", kind="attention", B=24, n_min=20, n_max=64, tree=True, ctx_min=500, ctx_max=2600,
             hkv=4, group=7, d=64, page=64, dtype="f16", layout=4),
        # one long context and 5 drafts: few rows, work split along the context
        dict(name="attention-long", kind="attention", B=1, n_min=6, n_max=6, tree=False, ctx_min=130001, ctx_max=130001,
             hkv=4, group=8, d=128, page=64, dtype="bf16", layout=5),
        # chunks of two prompts behind a cached prefix: the compute-bound end
        dict(name="attention-prompt", kind="attention", B=2, n_min=1500, n_max=2111, tree=False, ctx_min=4000,
             ctx_max=6100, hkv=8, group=4, d=128, page=32, dtype="bf16", layout=6),
        # a decoding step's rows: latency
        dict(name="append-decode", kind="append", B=32, n_min=1, n_max=9, ctx_min=0, ctx_max=900, hkv=8, d=128, page=16,
             dtype="bf16", layout=7),
        # prompt chunks: bandwidth
        dict(name="append-prompt", kind="append", B=6, n_min=2000, n_max=5000, ctx_min=0, ctx_max=3000, hkv=8, d=128,
             page=32, dtype="bf16", layout=8),
        # a few trees in a shallow cache
        dict(name="commit-few", kind="commit", B=4, n_min=8, n_max=33, ctx_min=50, ctx_max=400, hkv=8, d=64, page=16,
             layers=2, dtype="f16", layout=9),
        # a batch of 64-node trees in a deeper cache
        dict(name="commit-trees", kind="commit", B=64, n_min=30, n_max=64, ctx_min=0, ctx_max=500, hkv=8, d=128, page=32,
             layers=8, dtype="bf16", layout=10),
        # a few branches of two requests
        dict(name="pages-few", kind="pages", parents=2, forks=6, n_min=1, n_max=6, ctx_min=10, ctx_max=900, hkv=2, d=64,
             page=16, layers=4, dtype="bf16", layout=11),
        # parallel samples of a batch of prompts
        dict(name="pages-samples", kind="pages", parents=32, forks=96, n_min=1, n_max=40, ctx_min=100, ctx_max=2000,
             hkv=8, d=128, page=64, layers=4, dtype="bf16", layout=12),
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
    n, ctx = _sizes(case)
    scores = len(n) * case["hkv"] * case.get("group", 0) * max(n) * (max(ctx) + max(n))
    cost = work(case)
    return cost["bytes"] < 1.1e9 and cost["flops"] < 3.5e11 and scores < 2e9


def _drawn(rng):
    kind = rng.choice(["attention", "attention", "attention", "append", "commit", "pages"])
    case = dict(kind=kind, hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 80, 96, 128]),
                page=rng.choice([8, 16, 24, 32, 64, 128]), dtype=rng.choice(["bf16", "f16"]),
                layout=rng.randrange(1 << 20))
    if kind == "attention":
        case["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8])
        form = rng.choice(["decode", "verify", "verify", "tree", "prompt"])
        case["tree"] = form == "tree"
        if form == "decode":
            case["n_min"] = case["n_max"] = 1
        elif form == "verify":
            case["n_min"], case["n_max"] = rng.choice([(0, 9), (1, 33), (5, 5), (0, 3)])
        elif form == "tree":
            case["n_min"], case["n_max"] = rng.choice([(1, 64), (17, 100), (64, 64)])
        else:
            case["n_max"] = _log_uniform(rng, 100, 2000)
            case["n_min"] = rng.randint(1, case["n_max"])
        case["B"] = _log_uniform(rng, 1, 3 if form == "prompt" else 96)
        top = min(8000 if form == "prompt" else 20000, 400000 // case["B"])
        case["ctx_max"] = _log_uniform(rng, 20, top)
        case["ctx_min"] = rng.randint(0, case["ctx_max"])
    elif kind == "append":
        case["B"] = _log_uniform(rng, 1, 128)
        case["n_max"] = _log_uniform(rng, 1, 20000 // case["B"])
        case["n_min"] = rng.randint(0, case["n_max"])
        case["ctx_min"], case["ctx_max"] = 0, _log_uniform(rng, 10, 1000)
    elif kind == "commit":
        case["B"] = _log_uniform(rng, 1, 64)
        case["n_max"] = rng.randint(2, 100 if case["B"] < 40 else 64)
        case["n_min"] = rng.randint(1, case["n_max"])
        case["ctx_min"], case["ctx_max"] = 0, _log_uniform(rng, 10, 400)
        case["layers"] = rng.randint(1, 6)
    else:
        case["parents"] = _log_uniform(rng, 1, 32)
        case["forks"] = _log_uniform(rng, 1, 96)
        case["n_max"] = rng.randint(1, 40)
        case["n_min"] = rng.randint(1, case["n_max"])
        case["ctx_min"], case["ctx_max"] = 0, _log_uniform(rng, 20, 2000)
        case["layers"] = rng.randint(1, 4)
    return case


# ---------------------------------------------------------------------------------------
# Shapes that follow from the case alone
# ---------------------------------------------------------------------------------------


def _sizes(case):
    """Per request: new tokens, committed tokens."""
    rng = random.Random(case["layout"])
    B = case["parents"] + case["forks"] if case["kind"] == "pages" else case["B"]
    n = [rng.randint(case["n_min"], case["n_max"]) for _ in range(B)]
    ctx = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in range(B)]
    return n, ctx


def _trees(case, n):
    """Draft trees as level-order drafting makes them: a parent index per node (-1 at the root), and
    per request the nodes of one root-to-leaf walk, the accepted path."""
    rng = random.Random(case["layout"] + 1)
    parent, paths = [], []
    for size in n:
        par = [-1] * min(size, 1)
        for i in range(1, size):
            par.append(rng.randint(max(0, (i - 1) // 4 - 1), max(0, (i - 1) // 2)))
        path = [0] if size else []
        while path:
            children = [i for i in range(path[-1] + 1, size) if par[i] == path[-1]]
            if not children or rng.random() < 0.15:
                break
            path.append(rng.choice(children))
        parent += par
        paths.append(path)
    return parent, paths


def _fork_plan(case):
    """Requests 0 .. forks-1 are branches, the rest their parents; the parent of each branch."""
    rng = random.Random(case["layout"] + 2)
    F, Pn = case["forks"], case["parents"]
    return [F + rng.randrange(Pn) for _ in range(F)]


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    n, ctx = _sizes(case)
    row = 2 * case["hkv"] * case["d"] * 2  # one token's keys and values in one layer
    if case["kind"] == "attention":
        hq = case["hkv"] * case["group"]
        keys = sum(c + m for c, m in zip(ctx, n) if m)
        if case["tree"]:
            parent, _ = _trees(case, n)
            seen, at = 0, 0
            for c, m in zip(ctx, n):
                depth = []
                for i in range(m):
                    p = parent[at + i]
                    depth.append(1 if p < 0 else depth[p] + 1)
                seen += m * c + sum(depth)
                at += m
        else:
            seen = sum(m * c + m * (m + 1) // 2 for c, m in zip(ctx, n))
        return {"bytes": keys * row + 2 * sum(n) * hq * case["d"] * 2, "flops": 4 * case["d"] * hq * seen}
    if case["kind"] == "append":
        return {"bytes": 2 * sum(n) * row, "flops": 0}
    if case["kind"] == "commit":
        _, paths = _trees(case, n)
        moved = sum(sum(node != i for i, node in enumerate(path)) for path in paths)
        return {"bytes": 2 * (sum(n) + moved) * row * case["layers"] + 4 * (2 * sum(n) + 4 * case["B"]), "flops": 0}
    F, page = case["forks"], case["page"]
    parents = _fork_plan(case)
    shared = sum(_pages(ctx[p], page) for p in parents)
    copied = sum(ctx[p] % page for i, p in enumerate(parents) if n[i])
    fresh = sum(_pages(c + m, page) - _pages(c, page) if m else 0
                for c, m in [(ctx[p], n[i]) for i, p in enumerate(parents)] + list(zip(ctx[F:], n[F:])))
    return {"bytes": 2 * copied * row * case["layers"] + 4 * (4 * shared + 4 * fresh), "flops": 0}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = random.Random(seed)
    n, ctx = _sizes(case)
    page, hkv, d, dt = case["page"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    layers, R, N = case.get("layers", 1), len(n), sum(n)
    forked = case["forks"] if case["kind"] == "pages" else 0
    starts = ctx if not forked else [ctx[p] for p in _fork_plan(case)] + ctx[forked:]
    need = [_pages(c + m, page) for c, m in zip(starts, n)]
    max_pages = max(max(need), 1)
    num_pages = sum(need) + R + 3
    order = list(range(num_pages))
    host.shuffle(order)
    table = [[-1] * max_pages for _ in range(R)]
    held, used = [0] * R, 0
    for r in range(R):
        # pages: branches hold nothing yet, parents their context; elsewhere room for the new tokens is there
        count = (0 if r < forked else _pages(ctx[r], page)) if case["kind"] == "pages" else need[r]
        table[r][:count] = order[used:used + count]
        held[r], used = count, used + count
    ref = [0] * num_pages
    for p in order[:used]:
        ref[p] = 1
    free = sorted(order[used:])
    s = dict(kind=case["kind"], page=page, hkv=hkv, d=d, n=n, ctx=starts, layers=layers, total=N,
             most=max(max(n), 1), keys=max(max(c + m for c, m in zip(starts, n)), 1))
    kv = torch.randn((layers, num_pages, 2, page, hkv, d), generator=gen, device="cuda", dtype=torch.float32)
    kv = kv.to(dt)
    s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    s["table"], s["held"], s["ref"] = _ints(table), _ints(held), _ints(ref)
    s["lens"] = _ints([0] * forked + ctx[forked:])
    s["free"] = _ints(free + [0] * (num_pages - len(free)))
    s["num_free"] = _ints([len(free)])
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    s["cu"] = _ints(cu)
    s["parent"] = None
    if case["kind"] == "attention":
        s["group"], s["scale"] = case["group"], 1.0 / math.sqrt(d)
        # scores of standard deviation 2: softmax rows neither flat nor one-hot
        s["q"] = (2 * torch.randn((N, hkv * case["group"], d), generator=gen, device="cuda")).to(dt)
        if case["tree"]:
            s["parent"] = _ints(_trees(case, n)[0])
    if case["kind"] in ("append", "commit"):
        s["k_new"] = torch.randn((layers, N, hkv, d), generator=gen, device="cuda").to(dt)
        s["v_new"] = torch.randn((layers, N, hkv, d), generator=gen, device="cuda").to(dt)
    if case["kind"] == "commit":
        parent, paths = _trees(case, n)
        s["parent"] = _ints(parent)
        s["accepted"] = _ints([len(p) - 1 for p in paths])
        s["last"] = _ints([p[-1] if p else 0 for p in paths])
        s["out_lens"] = torch.zeros_like(s["lens"])
        s["depth"] = max(max(len(p) for p in paths), 1)
    if case["kind"] == "pages":
        s["src"], s["dst"] = _ints(_fork_plan(case)), _ints(list(range(forked)))
        s["keep"] = s["lens"].clone()
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


def _own_attention(s):
    cache, c = _handle(s)
    return cache.attention(c, 0, s["q"], s["cu"], parent=s["parent"], scale=s["scale"])


def _own_append(s):
    cache, c = _handle(s)
    cache.append(c, 0, s["k_new"][0], s["v_new"][0], s["cu"])
    return s["k"], s["v"]


def _own_commit(s):
    cache, c = _handle(s)
    for layer in range(s["layers"]):
        cache.append(c, layer, s["k_new"][layer], s["v_new"][layer], s["cu"])
    cache.commit(c, s["cu"], s["accepted"], parent=s["parent"], last_node=s["last"], out_lens=s["out_lens"])
    return s["k"], s["v"], s["out_lens"]


def _own_pages(s):
    cache, c = _handle(s)
    cache.release(c, s["keep"])
    cache.fork(c, s["src"], s["dst"])
    cache.reserve(c, s["cu"])
    return tuple(s[name] for name in ("table", "lens", "held", "ref", "free", "num_free", "k", "v"))


_OWN = dict(attention=_own_attention, append=_own_append, commit=_own_commit, pages=_own_pages)


def _request_of(s):
    """Per new token: its request, its index there."""
    counts = (s["cu"][1:] - s["cu"][:-1]).long()
    request = torch.repeat_interleave(torch.arange(len(s["n"]), device="cuda"), counts, output_size=s["total"])
    return request, torch.arange(s["total"], device="cuda") - s["cu"].long()[request]


def _plain_attention(s):
    R, most, keys, hkv, G, d = len(s["n"]), s["most"], s["keys"], s["hkv"], s["group"], s["d"]
    t = torch.arange(keys, device="cuda")
    pages = s["table"].long()[:, t // s["page"]].clamp(min=0)
    k = s["k"][0][pages, t % s["page"]].float().permute(0, 2, 1, 3)
    v = s["v"][0][pages, t % s["page"]].float().permute(0, 2, 1, 3)
    request, index = _request_of(s)
    q = torch.zeros((R, most, hkv, G, d), device="cuda")
    q[request, index] = s["q"].float().view(-1, hkv, G, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(R, hkv, most * G, d)
    scores = (q @ k.transpose(2, 3)).mul_(s["scale"])
    lens = s["lens"].long()
    new = t[None, :] - lens[:, None]  # position among the new tokens, below zero in the context
    i = torch.arange(most, device="cuda")
    if s["parent"] is None:
        seen = new[:, None, :] <= i[None, :, None]
    else:
        reach = torch.zeros((R, most, most), device="cuda")
        reach[:, i, i] = 1
        reach[request, index, torch.where(s["parent"] < 0, index, s["parent"].long())] = 1
        for _ in range(max(1, (most - 1).bit_length())):
            reach = (reach @ reach).clamp_(max=1)
        among = reach.gather(2, new.clamp(0, most - 1)[:, None, :].expand(R, most, keys)) > 0
        seen = (new < 0)[:, None, :] | (among & (new < most)[:, None, :])
    # rows of no token (requests of fewer tokens than the longest) see what is there, and are dropped
    hidden = ~seen[:, None, :, None, :].expand(R, hkv, most, G, keys).reshape(R, hkv, most * G, keys)
    scores.masked_fill_(hidden, -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    out = (scores @ v) / scores.sum(-1, keepdim=True)
    out = out.view(R, hkv, most, G, d).permute(0, 2, 1, 3, 4)[request, index]
    return out.reshape(s["total"], hkv * G, d).to(s["q"].dtype)


def _slots(s, request, position):
    return s["table"].long()[request, position // s["page"]], position % s["page"]


def _plain_append(s):
    request, index = _request_of(s)
    page, row = _slots(s, request, s["lens"].long()[request] + index)
    s["k"][0][page, row] = s["k_new"][0]
    s["v"][0][page, row] = s["v_new"][0]
    return s["k"], s["v"]


def _plain_commit(s):
    request, index = _request_of(s)
    page, row = _slots(s, request, s["lens"].long()[request] + index)
    s["k"][:, page, row] = s["k_new"]
    s["v"][:, page, row] = s["v_new"]
    R = len(s["n"])
    accepted, lens, first = s["accepted"].long(), s["lens"].long(), s["cu"].long()[:-1]
    at = torch.where(accepted < 0, 0, s["last"].long())
    depth = accepted
    r = torch.arange(R, device="cuda")
    path = torch.zeros((R, s["depth"]), dtype=torch.long, device="cuda")
    for _ in range(s["depth"]):  # from the last accepted node up
        path[r, depth.clamp(min=0)] = torch.where(depth >= 0, at, path[r, depth.clamp(min=0)])
        up = s["parent"].long()[(first + at).clamp(max=max(s["total"] - 1, 0))]
        at = torch.where(depth > 0, up.clamp(min=0), at)
        depth = depth - 1
    level = torch.arange(s["depth"], device="cuda")[None, :]
    moves = (level <= accepted[:, None]) & (path != level)
    request, level = moves.nonzero(as_tuple=True)
    old = _slots(s, request, lens[request] + path[request, level])
    new = _slots(s, request, lens[request] + level)
    s["k"][:, new[0], new[1]] = s["k"][:, old[0], old[1]]
    s["v"][:, new[0], new[1]] = s["v"][:, old[0], old[1]]
    s["out_lens"].copy_(s["lens"] + s["accepted"] + 1)
    return s["k"], s["v"], s["out_lens"]


def _plain_pages(s):
    page, table, ref = s["page"], s["table"], s["ref"]
    column = torch.arange(table.shape[1], device="cuda")[None, :]
    # release: what lies behind the kept tokens
    s["lens"].copy_(torch.minimum(s["lens"], s["keep"]))
    kept = (s["lens"] + (page - 1)) // page
    drop = (column >= kept[:, None]) & (column < s["held"][:, None])
    dropped = table[drop].long()
    ref.index_add_(0, dropped, torch.full_like(dropped, -1, dtype=torch.int32))
    gone = torch.zeros(ref.shape, dtype=torch.bool, device="cuda")
    gone[dropped] = True
    freed = (gone & (ref == 0)).nonzero().squeeze(1)
    s["free"][s["num_free"].long() + torch.arange(freed.numel(), device="cuda")] = freed.int()
    s["num_free"].add_(freed.numel())
    table.masked_fill_(drop, -1)
    s["held"].copy_(torch.minimum(s["held"], kept))
    # fork: the parent's pages, one count more each
    src, dst = s["src"].long(), s["dst"].long()
    count = (s["lens"][src] + (page - 1)) // page
    taken = column < count[:, None]
    table[dst] = torch.where(taken, table[src], torch.full_like(table[src], -1))
    pages = table[src][taken].long()
    ref.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    s["lens"][dst] = s["lens"][src]
    s["held"][dst] = count
    # reserve: shared pages that will be written are copied, in the order of requests while they stay shared
    lens, held = s["lens"].long(), s["held"].long()
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    need = torch.where(n > 0, (lens + n + (page - 1)) // page, 0)
    tail = lens // page
    r = torch.arange(lens.numel(), device="cuda")
    writes = (n > 0) & (lens % page != 0)
    last = torch.where(writes, table[r, tail.clamp(max=table.shape[1] - 1)].long(), -1)
    same = (last[:, None] == last[None, :]) & writes[:, None] & writes[None, :]
    before = (same & (r[None, :] < r[:, None])).sum(1)
    copies = writes & (ref[last.clamp(min=0)] - before > 1)
    fresh = (need - held).clamp(min=0) + copies
    base = fresh.cumsum(0) - fresh
    top = s["num_free"].long() - 1
    grown = (column >= held[:, None]) & (column < need[:, None])
    rank = base[:, None] + copies[:, None] + column - held[:, None]
    free = s["free"].long()
    who = copies.nonzero().squeeze(1)
    old, new = last[who], free[top - base[who]]
    ref.index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    ref[new] = 1
    taken = free[(top - rank)[grown]]
    table[grown] = taken.int()
    ref[taken] = 1
    table[who, tail[who]] = new.int()
    s["held"].copy_(torch.maximum(held, need))
    s["num_free"].sub_(fresh.sum().int())
    valid = torch.arange(page, device="cuda")[None, :] < (lens[who] % page)[:, None]
    pair, row = valid.nonzero(as_tuple=True)
    s["k"][:, new[pair], row] = s["k"][:, old[pair], row]
    s["v"][:, new[pair], row] = s["v"][:, old[pair], row]
    return tuple(s[name] for name in ("table", "lens", "held", "ref", "free", "num_free", "k", "v"))


_PLAIN = dict(attention=_plain_attention, append=_plain_append, commit=_plain_commit, pages=_plain_pages)


# ---------------------------------------------------------------------------------------
# Exact results
# ---------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    n, ctx, page = s["n"], s["ctx"], case["page"]
    if case["kind"] == "attention":
        return _exact_attention(case, s)
    table, held = s["table"].tolist(), s["held"].tolist()
    k, v = s["k"].double(), s["v"].double()
    if case["kind"] in ("append", "commit"):
        paths = _trees(case, n)[1] if case["kind"] == "commit" else [[] for _ in n]
        spot, moves, at = [], [], 0
        for r, m in enumerate(n):
            where = lambda t: (table[r][t // page], t % page)  # noqa: E731
            spot += [where(ctx[r] + i) for i in range(m)]
            # an accepted path's row ends as the row of its node: taken from the new rows themselves
            moves += [(where(ctx[r] + i), at + node) for i, node in enumerate(paths[r])]
            at += m
        for cache, rows in ((k, s["k_new"].double()), (v, s["v_new"].double())):
            if spot:
                p, i = zip(*spot)
                cache[:, list(p), list(i)] = rows
            if moves:
                p, i = zip(*[m[0] for m in moves])
                cache[:, list(p), list(i)] = rows[:, [m[1] for m in moves]]
        if case["kind"] == "append":
            return k, v
        return k, v, _ints([c + len(p) for c, p in zip(ctx, paths)])
    # pages: one request after the other, as bookkeeping on the host would go
    ref, free = s["ref"].tolist(), s["free"].tolist()
    lens, num_free = s["lens"].tolist(), int(s["num_free"].item())
    for child, parent in zip(s["dst"].tolist(), s["src"].tolist()):
        held[child] = _pages(lens[parent], page)
        lens[child] = lens[parent]
        for i in range(held[child]):
            table[child][i] = table[parent][i]
            ref[table[parent][i]] += 1
    for r, m in enumerate(n):
        if not m:
            continue
        if lens[r] % page:
            old = table[r][lens[r] // page]
            if ref[old] > 1:
                num_free -= 1
                new = free[num_free]
                ref[old] -= 1
                ref[new] = 1
                table[r][lens[r] // page] = new
                rows = lens[r] % page
                k[:, new, :rows] = k[:, old, :rows]
                v[:, new, :rows] = v[:, old, :rows]
        while held[r] < _pages(lens[r] + m, page):
            num_free -= 1
            table[r][held[r]] = free[num_free]
            ref[free[num_free]] = 1
            held[r] += 1
    return (_ints(table), _ints(lens), _ints(held), _ints(ref), _ints(free), _ints([num_free]), k, v)


def _exact_attention(case, s):
    n, ctx, page, G = s["n"], s["ctx"], case["page"], case["group"]
    parent = s["parent"].tolist() if s["parent"] is not None else None
    table = s["table"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for r, m in enumerate(n):
        if not m:
            continue
        L = ctx[r] + m
        pages = torch.tensor(table[r][:_pages(L, page)], device="cuda")
        seen = torch.ones((m, L), dtype=torch.bool)
        if parent is None:
            seen[:, ctx[r]:] = torch.tril(torch.ones((m, m), dtype=torch.bool))
        else:
            seen[:, ctx[r]:] = False
            for i in range(m):
                if parent[at + i] >= 0:
                    seen[i, ctx[r]:] = seen[parent[at + i], ctx[r]:]
                seen[i, ctx[r] + i] = True
        seen = seen.cuda()
        for h in range(case["hkv"]):
            k = s["k"][0][pages, :, h].reshape(-1, case["d"])[:L].double()
            v = s["v"][0][pages, :, h].reshape(-1, case["d"])[:L].double()
            for g in range(h * G, h * G + G):
                x = s["q"][at:at + m, g].double() @ k.T * s["scale"]
                x = x.masked_fill(~seen, -math.inf)
                x = torch.exp(x - x.max(1, keepdim=True).values)
                out[at:at + m, g] = (x @ v) / x.sum(1, keepdim=True)
        at += m
    return out
