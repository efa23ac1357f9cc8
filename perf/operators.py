"""The cases by which the paged FP8 KV-cache operators are measured, with their plain forms.

The operators serve a decode loop that verifies a drafted tree: nvfp4_kv_append writes the nodes' keys and values into
the cache's pages, nvfp4_kv_attention reads them back, nvfp4_kv_compact keeps the accepted path, nvfp4_kv_fork and
nvfp4_kv_resize share and free pages between agent turns.  Where `own` is false, run() computes them with elementary
torch operations; where it is true, it calls the library.  exact() has the same results from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BIG = 2 ** 31 - 1


def listed():
    return [
        # one token of one short conversation: the smallest call, all latency
        dict(name="decode_one", op="attention", dtype="bf16", seqs=1, nodes=1, tree=False, heads=8, group=5, dim=128,
             page=16, context=511, ragged=False),
        # a 16-node drafted tree at the end of the longest agent context
        dict(name="tree_long", op="attention", dtype="bf16", seqs=1, nodes=16, tree=True, heads=8, group=5, dim=128,
             page=64, context=23552, ragged=False),
        # a ragged batch of small trees in float32, each sequence with its own length and node count
        dict(name="tree_ragged_f32", op="attention", dtype="f32", seqs=16, nodes=5, tree=True, heads=4, group=4,
             dim=64, page=32, context=4099, ragged=True),
        # the suffix of a new turn over a reused prefix
        dict(name="suffix_512", op="attention", dtype="bf16", seqs=1, nodes=512, tree=False, heads=8, group=5, dim=128,
             page=64, context=23040, ragged=False),
        # the 16 nodes of a drafted tree, one layer
        dict(name="append_tree", op="append", dtype="bf16", seqs=1, nodes=16, heads=8, dim=128, page=64, context=23552,
             ragged=False),
        # prompts of four new conversations in float32
        dict(name="append_prompts_f32", op="append", dtype="f32", seqs=4, nodes=2047, heads=8, dim=128, page=64,
             context=77, ragged=False),
        # the accepted path of one tree, over 16 layers
        dict(name="compact_one", op="compact", layers=16, seqs=1, nodes=16, heads=8, dim=128, page=64, context=1000),
        # a batch of accepted paths over many layers
        dict(name="compact_batch", op="compact", layers=24, seqs=32, nodes=33, heads=4, dim=256, page=16, context=200),
        # a turn that starts from one cached conversation
        dict(name="fork_one", op="fork", layers=16, seqs=1, heads=8, dim=128, page=64, context=5000),
        # many turns from many conversations
        dict(name="fork_many", op="fork", layers=16, seqs=33, heads=4, dim=128, page=128, context=500),
        # pages for the next tree of one conversation, given back after it
        dict(name="resize_step", op="resize", seqs=1, page=16, context=23552, step=16, pages=4096),
        # a batch of conversations admitted and dropped
        dict(name="resize_batch", op="resize", seqs=20, page=64, context=0, step=23552, pages=8192),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "compact", "fork", "resize"])
    page, dim, heads = rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 5, 8])
    if op == "attention":
        tree = rng.random() < 0.5
        seqs = log_int(rng, 1, 40)
        nodes = log_int(rng, 1, 64 if tree else 700 // seqs + 1)
        group = rng.choice([1, 2, 3, 4, 5, 8])
        # no more scores than the suffix's, and a cache that fits beside its 32-bit form
        most = min(24000, 450_000_000 // (seqs * heads * group * nodes), 200_000_000 // (seqs * heads * dim))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), seqs=seqs, nodes=nodes, tree=tree, heads=heads,
                    group=group, dim=dim, page=page, context=log_int(rng, 1, max(2, most - nodes)),
                    ragged=rng.random() < 0.5)
    if op == "append":
        seqs = log_int(rng, 1, 40)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), seqs=seqs, nodes=log_int(rng, 1, 8000 // seqs),
                    heads=heads, dim=dim, page=page, context=log_int(rng, 1, 24000 // seqs),
                    ragged=rng.random() < 0.3)
    if op == "compact":
        heads, page = rng.choice([1, 2, 4]), rng.choice([16, 32])
        layers, seqs, nodes = log_int(rng, 1, 48), log_int(rng, 1, 32), log_int(rng, 1, 64)
        return dict(op=op, layers=layers, seqs=seqs, nodes=nodes, heads=heads, dim=dim, page=page,
                    context=log_int(rng, 1, max(8, 150_000_000 // (layers * seqs * heads * dim) - nodes) // 8))
    if op == "fork":
        heads, layers, seqs = rng.choice([1, 2, 4]), log_int(rng, 1, 32), log_int(rng, 1, 32)
        return dict(op=op, layers=layers, seqs=seqs, heads=heads, dim=dim, page=page,
                    context=log_int(rng, page + 1, max(page + 2, min(6000, 80_000_000 // (layers * seqs * heads * dim)))))
    return dict(op=op, seqs=log_int(rng, 1, 64), page=page, context=log_int(rng, 1, 12000),
                step=log_int(rng, 1, 8000), pages=rng.choice([40000, 65536, 100003]))


# ---------------------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randint(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _values(g, shape, dtype=torch.float32):
    """Keys and values as layers make them: normal, one channel in a hundred eight times as large."""
    x = torch.randn(shape, generator=g, device=DEV)
    dim = shape[-1]
    x[..., torch.randperm(dim, generator=g, device=DEV)[: max(1, dim // 100)]] *= 8.0
    return x.to(dtype)


def _pages(g, shape):
    """E4M3 bytes of such values under a calibrated scale, and the scale."""
    codes = torch.empty(shape, dtype=torch.uint8, device=DEV)
    scale = 40.0 / 448.0
    for part in codes.view(-1, shape[-1]).split(1 << 21):
        part.copy_((_values(g, part.shape) / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return codes, torch.full((1,), scale, device=DEV)


def _table(g, tokens, page, spare):
    """A table in which each sequence holds the pages of `tokens` tokens, in no physical order; how many pages in all."""
    seqs = len(tokens)
    need = [-(-t // page) for t in tokens]
    total, width = sum(need), max(1, max(need))
    order = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(seqs):
        table[b, : need[b]] = order[at:at + need[b]]
        at += need[b]
    return table, need, total + spare, order[at:]


def _lens(g, case):
    if not case["ragged"]:
        return [case["context"]] * case["seqs"]
    return _randint(g, 0, case["context"] + 1, (case["seqs"],)).tolist()


def _trees(g, seqs, nodes):
    """Parents of drafted trees: each node hangs on one of the four before it."""
    v = torch.arange(nodes, device=DEV, dtype=torch.int32)
    back = 1 + _randint(g, 0, 4, (seqs, nodes))
    parent = torch.maximum(v[None] - back, torch.zeros_like(v)[None])
    parent[:, 0] = -1
    return parent


def _accepted(g, parent):
    """Results as the acceptance gives them (end, accepted count, bonus token, path, -1 ...) for random end nodes."""
    rows = []
    tree = parent.tolist()
    ends = _randint(g, 0, parent.shape[1], (parent.shape[0],)).tolist()
    for up, end in zip(tree, ends):
        path, v = [], end
        while v > 0:
            path.append(v)
            v = up[v]
        rows.append([end, len(path), 17] + path[::-1] + [-1] * (len(up) - len(path)))
    return torch.tensor(rows, dtype=torch.int32, device=DEV)


def _pool(g, tokens, page, pages, width):
    """A page pool in which sequence b holds the pages of tokens[b] tokens: table, held, refs, free list."""
    need = [-(-t // page) for t in tokens]
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(tokens), width), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    refs[order[:at].long()] = 1
    free = torch.full((pages + 1,), -1, dtype=torch.int32, device=DEV)
    free[0] = pages - at
    free[1:1 + pages - at] = order[at:]
    return dict(table=table, held=torch.tensor(need, dtype=torch.int32, device=DEV), refs=refs, free=free)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if op in ("attention", "append"):
        lens = _lens(g, case)
        table, _, pages, _ = _table(g, [n + case["nodes"] for n in lens], case["page"], 5)
        shape = (pages, case["heads"], case["page"], case["dim"])
        s["k_pages"], s["k_scale"] = _pages(g, shape)
        s["v_pages"], s["v_scale"] = _pages(g, shape)
        s["table"], s["lens"] = table, ints(lens)
        s["counts"] = _randint(g, 1, case["nodes"] + 1, (case["seqs"],)) if case["ragged"] else None
    if op == "attention":
        shape = (case["seqs"], case["nodes"], case["heads"] * case["group"], case["dim"])
        # queries with which some keys stand out, as they do in a trained layer
        s["q"] = (2.0 * torch.randn(shape, generator=g, device=DEV)).to(_dtype(case))
        s["parent"] = _trees(g, case["seqs"], case["nodes"]) if case["tree"] else None
    elif op == "append":
        shape = (case["seqs"], case["nodes"], case["heads"], case["dim"])
        s["k"], s["v"] = _values(g, shape, _dtype(case)), _values(g, shape, _dtype(case))
    elif op == "compact":
        lens = [max(0, case["context"] - 7 * b) for b in range(case["seqs"])]
        table, _, pages, _ = _table(g, [n + case["nodes"] for n in lens], case["page"], 1)
        shape = (case["layers"], pages, case["heads"], case["page"], case["dim"])
        s["k_pages"], _ = _pages(g, shape)
        s["v_pages"], _ = _pages(g, shape)
        s["table"], s["lens"] = table, ints(lens)
        s["result"] = _accepted(g, _trees(g, case["seqs"], case["nodes"]))
    elif op == "fork":
        n, page = case["seqs"], case["page"]
        tokens = [case["context"] + 3 * b for b in range(n)]
        width = -(-max(tokens) // page)
        # the first n sequences are cached conversations, the next n their new turns, not begun yet
        pages = sum(-(-t // page) for t in tokens) + 2 * n
        s.update(_pool(g, tokens + [0] * n, page, pages, width))
        shape = (case["layers"], pages, case["heads"], page, case["dim"])
        s["k_pages"], _ = _pages(g, shape)
        s["v_pages"], _ = _pages(g, shape)
        s["src"], s["dst"] = ints(list(range(n))), ints([2 * n - 1 - b for b in range(n)])
        keep = _randint(g, 1, case["context"] + 1, (n,))
        s["tokens"] = torch.where(keep % page == 0, keep - 1, keep).to(torch.int32)
    elif op == "resize":
        n, page = case["seqs"], case["page"]
        now = [max(0, case["context"] - 5 * b) for b in range(n)]
        up = [t + case["step"] for t in now]
        width = -(-max(up) // page) + 1
        pages = max(case["pages"], sum(-(-t // page) for t in up))
        s.update(_pool(g, now, page, pages, width))
        s["ids"] = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        s["up"], s["down"] = ints(up)[s["ids"].long()], ints(now)[s["ids"].long()]
    return s


# ---------------------------------------------------------------------------------------------- plain forms


def _plain_attention(s):
    B, M, H, G, D = s["seqs"], s["nodes"], s["heads"], s["group"], s["dim"]
    N = s["table"].shape[1] * s["page"]

    def gathered(pages, scale):
        x = pages[s["table"].clamp(min=0).long()].view(torch.float8_e4m3fn)  # [B, W, H, page, D]
        return x.transpose(1, 2).float().reshape(B, H, N, D) * scale

    q = s["q"].float().reshape(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    k = gathered(s["k_pages"], s["k_scale"]).transpose(2, 3).contiguous()
    scores = torch.matmul(q, k) * (1.0 / math.sqrt(D))
    # who sees what: the prefix, and of the nodes one's own line (or every node before, in a chain)
    v = torch.arange(M, device=DEV)
    if s["parent"] is None:
        line = (v[:, None] >= v[None]).expand(B, M, M)
    else:
        step = torch.eye(M, device=DEV) + (s["parent"][:, :, None] == v).float()
        line = torch.linalg.matrix_power(step, 64) > 0
    count = s["counts"] if s["counts"] is not None else torch.full_like(s["lens"], M)
    line = line & (v[None] < count[:, None])[:, :, None]
    at = torch.arange(N, device=DEV)[None] - s["lens"][:, None]  # [B, N]: node index of each slot
    node = at.clamp(0, M - 1)[:, None].expand(B, M, N)
    seen = ((at < 0)[:, None] & (v[None] < count[:, None])[:, :, None]) | (
        (at >= 0)[:, None] & (at < M)[:, None] & torch.gather(line, 2, node))
    seen = seen[:, None, :, None, :]  # [B, 1, M, 1, N]
    scores = scores.view(B, H, M, G, N).masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, H, M * G, N), gathered(s["v_pages"], s["v_scale"])).view(B, H, M, G, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (total.log() + base)[..., 0]
    out = out.permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D).to(s["q"].dtype)
    return dict(out=out, lse=lse.permute(0, 2, 1, 3).reshape(B, M, H * G))


def _slots(s, position):
    """Page and slot of the tokens at `position` [B, ...]."""
    flat = position.reshape(position.shape[0], -1).long()
    page = torch.gather(s["table"].long(), 1, flat // s["page"])
    return page, flat % s["page"]


def _plain_append(s):
    B, M = s["seqs"], s["nodes"]
    v = torch.arange(M, device=DEV)
    page, slot = _slots(s, s["lens"][:, None] + v)
    if s["counts"] is not None:
        here = v[None] < s["counts"][:, None]
        page, slot = page[here], slot[here]
    else:
        here = torch.ones((), dtype=torch.bool, device=DEV).expand(B, M)
        page, slot = page.reshape(-1), slot.reshape(-1)
    for x, scale, pages in ((s["k"], s["k_scale"], s["k_pages"]), (s["v"], s["v_scale"], s["v_pages"])):
        x = x[here] if s["counts"] is not None else x.reshape(B * M, s["heads"], s["dim"])
        y = (x.float() * (1.0 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pages[page, :, slot] = y
    return _page_values(s)


def _plain_compact(s):
    M = s["nodes"]
    L = s["result"][:, 1:2]
    i = torch.arange(M, device=DEV)[None]
    # entries behind the path stay where they are: node i + 1 (the last one's own place at the end)
    stay = (i + 1).clamp(max=M - 1)
    node = torch.where(i < L, s["result"][:, 3:], stay)
    to = torch.where(i < L, i + 1, stay)
    page, slot = _slots(s, s["lens"][:, None] + node)
    page2, slot2 = _slots(s, s["lens"][:, None] + to)
    for pages in (s["k_pages"], s["v_pages"]):
        pages[:, page2, :, slot2] = pages[:, page, :, slot]
    return dict(_page_values(s), lens=s["lens"] + 1 + L[:, 0])


def _page_values(s):
    """The cache as the E4M3 values that its bytes stand for."""
    return dict(k=s["k_pages"].view(torch.float8_e4m3fn), v=s["v_pages"].view(torch.float8_e4m3fn))


def _longer(x):
    """x with one more entry, for what is to go nowhere."""
    return torch.cat([x, x[:1]])


def _earlier(x):
    """Which entries of the list x repeat an earlier one."""
    return ((x[:, None] == x[None]) & torch.ones_like(x[:, None] == x[None]).tril(-1)).any(1)


def _release(s, rows, gone, free, top, refs):
    """Pages where gone [n, W] leave their holders: refs - 1, and those at zero onto the free list, first come first."""
    P, W = s["refs"].shape[0], s["table"].shape[1]
    page = torch.where(gone, rows, torch.full_like(rows, P)).long()
    refs.index_add_(0, page.reshape(-1), -torch.ones_like(rows).reshape(-1))
    order = torch.arange(page.numel(), device=DEV).view(page.shape)
    first = torch.full((P + 1,), BIG, dtype=torch.int64, device=DEV)
    first.scatter_reduce_(0, page.reshape(-1), order.reshape(-1), "amin")
    back = gone & (refs[page] == 0) & (first[page] == order)
    rank = back.reshape(-1).cumsum(0).view(page.shape)
    free.scatter_(0, torch.where(back, top + rank, torch.full_like(rank, P + 1)).reshape(-1),
                  torch.where(back, rows, free[-1]).reshape(-1))
    free[0] = top + rank.reshape(-1)[-1]
    s["refs"].copy_(refs[:P])
    s["free"].copy_(free[: P + 1])


def _plain_resize(s, tokens):
    S, W, P = s["table"].shape[0], s["table"].shape[1], s["refs"].shape[0]
    table, held, refs, free = _longer(s["table"]), _longer(s["held"]), _longer(s["refs"]), _longer(s["free"])
    need = (tokens + s["page"] - 1) // s["page"]
    valid = (s["ids"] >= 0) & (s["ids"] < S) & (tokens >= 0) & (need <= W) & ~_earlier(s["ids"])
    seq = torch.where(valid, s["ids"], torch.full_like(s["ids"], S)).long()
    have = held[seq]
    grow = (need - have).clamp(min=0) * valid
    total, F = grow.sum(), s["free"][0].long()
    fits = total <= F
    col = torch.arange(W, device=DEV)[None]
    new = (col >= have[:, None]) & (col < need[:, None]) & (valid & fits)[:, None]
    gone = (col >= need[:, None]) & (col < have[:, None]) & (valid & fits)[:, None]
    at = F - (grow.cumsum(0) - grow)[:, None] - (col - have[:, None])
    page = free[torch.where(new, at, torch.zeros_like(at)).long()]
    refs.scatter_(0, torch.where(new, page, torch.full_like(page, P)).long().reshape(-1),
                  torch.ones_like(page).reshape(-1))
    rows = table[seq]
    table[seq] = torch.where(new, page, torch.where(gone, torch.full_like(rows, -1), rows))
    held[seq] = torch.where(valid & fits, need, have).to(torch.int32)
    s["table"].copy_(table[:S])
    s["held"].copy_(held[:S])
    _release(s, rows, gone, free, torch.where(fits, F - total, F), refs)
    return torch.where(fits, torch.zeros_like(total), total - F).to(torch.int32).view(1)


def _plain_fork(s):
    S, W, P = s["table"].shape[0], s["table"].shape[1], s["refs"].shape[0]
    src, dst, tokens, page = s["src"], s["dst"], s["tokens"], s["page"]
    table, held, refs, free = _longer(s["table"]), _longer(s["held"]), _longer(s["refs"]), _longer(s["free"])
    inside = (src >= 0) & (src < S) & (dst >= 0) & (dst < S) & (tokens >= 0)
    valid = inside & ~_earlier(dst) & ~(src[:, None] == dst[None]).any(1)
    a = torch.where(valid, src, torch.zeros_like(src)).long()
    b = torch.where(valid, dst, torch.full_like(dst, S)).long()
    valid = valid & (tokens.long() <= held[a].long() * page)
    b = torch.where(valid, b, torch.full_like(b, S))
    full, part = tokens // page, (tokens % page > 0) & valid
    total, F = part.sum(), s["free"][0].long()
    fits = total <= F
    part = part & fits
    fresh = free[torch.where(part, F + 1 - part.cumsum(0), torch.zeros_like(F)).long()]
    col = torch.arange(W, device=DEV)[None]
    from_, old = table[a], table[b]
    ok = (valid & fits)[:, None]
    shared = (col < full[:, None]) & ok
    gone = (col < held[b][:, None]) & ok
    nowhere = torch.full_like(from_, P)
    refs.index_add_(0, torch.where(shared, from_, nowhere).long().reshape(-1), torch.ones_like(from_).reshape(-1))
    refs.scatter_(0, torch.where(part, fresh, torch.full_like(fresh, P)).long(), torch.ones_like(fresh))
    rows = torch.where(shared, from_, torch.where((col == full[:, None]) & part[:, None], fresh[:, None].expand(-1, W),
                                                  torch.full_like(from_, -1)))
    table[b] = torch.where(ok, rows, old)
    held[b] = torch.where(valid & fits, (tokens + page - 1) // page, held[b]).to(torch.int32)
    # the used slots of the partial pages; an entry without one copies its page onto itself
    last = torch.gather(from_, 1, full.clamp(max=W - 1)[:, None].long())[:, 0].clamp(min=0).long()
    to = torch.where(part, fresh.long(), last)
    used = (torch.arange(page, device=DEV)[None] < (tokens % page)[:, None])[None, :, None, :, None]
    for pages in (s["k_pages"], s["v_pages"]):
        pages[:, to] = torch.where(used, pages[:, last], pages[:, to])
    s["table"].copy_(table[:S])
    s["held"].copy_(held[:S])
    _release(s, old, gone, free, torch.where(fits, F - total, F), refs)
    return torch.where(fits, torch.zeros_like(total), total - F).to(torch.int32).view(1)


def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op == "attention":
        return _plain_attention(s)
    if op == "append":
        return _plain_append(s)
    if op == "compact":
        return _plain_compact(s)
    if op == "fork":
        short = _plain_fork(s)
        return dict(_page_values(s), shortage=short, **_pool_state(s))
    short = [_plain_resize(s, s["up"]), _plain_resize(s, s["down"])]
    return dict(shortage=short, **_pool_state(s))


def _pool_state(s):
    return dict(table=s["table"], held=s["held"], refs=s["refs"], free=s["free"])


def _own(s):
    from nvfp4_w4a4_block_amd import binding as B
    op = s["op"]
    if op == "attention":
        out, lse = B.nvfp4_kv_attention(s["q"], s["k_scale"], s["v_scale"], s["k_pages"], s["v_pages"], s["table"],
                                        s["lens"], parent=s["parent"], counts=s["counts"], want_lse=True)
        return dict(out=out, lse=lse)
    if op == "append":
        B.nvfp4_kv_append(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_pages"], s["v_pages"], s["table"],
                          s["lens"], counts=s["counts"])
        return _page_values(s)
    if op == "compact":
        lens = B.nvfp4_kv_compact(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["result"])
        return dict(_page_values(s), lens=lens)
    pool = (s["table"], s["held"], s["refs"], s["free"])
    if op == "fork":
        short = B.nvfp4_kv_fork(*pool, s["k_pages"], s["v_pages"], s["src"], s["dst"], s["tokens"])
        return dict(_page_values(s), shortage=short, **_pool_state(s))
    short = [B.nvfp4_kv_resize(*pool, s["page"], s["ids"], s["up"]),
             B.nvfp4_kv_resize(*pool, s["page"], s["ids"], s["down"])]
    return dict(shortage=short, **_pool_state(s))


# ---------------------------------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "attention":
        size = 2 if case["dtype"] == "bf16" else 4
        B, M, H, G, D = case["seqs"], case["nodes"], case["heads"], case["group"], case["dim"]
        tokens = B * (case["context"] / 2 if case["ragged"] else case["context"])  # ragged: the mean length
        rows = B * M * (0.5 if case["ragged"] else 1.0)
        keys = rows * (tokens / B + (M + 1) / 2)
        return dict(bytes=2 * H * D * (tokens + rows) + 2 * B * M * H * G * D * size + B * M * H * G * 4,
                    flops=4 * H * G * D * keys)
    if op == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        rows = case["seqs"] * case["nodes"] * (0.5 if case["ragged"] else 1.0)
        return dict(bytes=2 * rows * case["heads"] * case["dim"] * (size + 1), flops=0)
    if op == "compact":
        # a random end node's line holds about two nodes in five of those before it
        moved = case["seqs"] * max(1.0, 0.2 * case["nodes"])
        return dict(bytes=2 * 2 * case["layers"] * moved * case["heads"] * case["dim"], flops=0)
    if op == "fork":
        return dict(bytes=2 * 2 * case["layers"] * case["seqs"] * case["heads"] * case["dim"] * case["page"] / 2
                    + 24 * case["seqs"] * case["context"] / case["page"] / 2, flops=0)
    # each page taken and given back: its table entry, its count and its place in the list, written twice
    return dict(bytes=case["seqs"] * (40 + 2 * 3 * 4 * 2 * max(1.0, case["step"] / case["page"])), flops=0)


# ---------------------------------------------------------------------------------------------- exact results


def _e4m3(codes):
    """The E4M3 values of bytes, from the format's definition, in 64 bits."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.bitwise_left_shift(torch.ones_like(e), e) * 2.0 ** -10)
    return torch.where(c >= 128, -mag, mag)


def _exact_attention(s):
    B, M, H, G, D, page = s["seqs"], s["nodes"], s["heads"], s["group"], s["dim"], s["page"]
    out = torch.zeros((B, M, H * G, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, M, H * G), -math.inf, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    counts = s["counts"].tolist() if s["counts"] is not None else [M] * B
    parents = s["parent"].tolist() if s["parent"] is not None else None
    ks, vs = s["k_scale"].double(), s["v_scale"].double()
    for b in range(B):
        n, c = lens[b], counts[b]
        ids = s["table"][b, : -(-(n + c) // page)].long()
        seen = torch.zeros((c, n + c), dtype=torch.bool)
        seen[:, :n] = True
        for v in range(c):
            if parents is None:
                seen[v, n:n + v + 1] = True
                continue
            u = v
            while u >= 0:
                seen[v, n + u] = True
                u = parents[b][u]
        seen = seen.to(DEV)
        for h in range(H):
            k = _e4m3(s["k_pages"][ids, h].reshape(-1, D)[: n + c]) * ks
            v = _e4m3(s["v_pages"][ids, h].reshape(-1, D)[: n + c]) * vs
            for j in range(h * G, (h + 1) * G):
                z = s["q"][b, :c, j].double() @ k.T / math.sqrt(D)
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                t = torch.logsumexp(z, 1)
                out[b, :c, j] = torch.exp(z - t[:, None]) @ v
                lse[b, :c, j] = t
    return dict(out=out, lse=lse)


def _nearest_e4m3(y):
    """E4M3 value nearest to y, ties to the even code, at most 448 in magnitude."""
    grid = _e4m3(torch.arange(127, device=DEV))
    mid = (grid[1:] + grid[:-1]) / 2
    a = y.abs()
    up, down = torch.searchsorted(mid, a, right=True), torch.searchsorted(mid, a, right=False)
    at = torch.where(up % 2 == 0, up, down)  # equal unless a is a midpoint
    return torch.where(y < 0, -grid[at], grid[at])


def _exact_append(s):
    got = {}
    for name in ("k", "v"):
        pages = _e4m3(s[name + "_pages"])
        inv = (1.0 / s[name + "_scale"]).double()
        y = _nearest_e4m3((s[name].double() * inv).float().double())
        for b, n in enumerate(s["lens"].tolist()):
            c = s["nodes"] if s["counts"] is None else int(s["counts"][b])
            at = torch.arange(n, n + c, device=DEV)
            pages[s["table"][b].long()[at // s["page"]], :, at % s["page"]] = y[b, :c]
        got[name] = pages
    return got


def _exact_compact(s):
    table, page = s["table"].tolist(), s["page"]
    got = {}
    for name in ("k", "v"):
        codes = s[name + "_pages"]
        pages = codes.clone()
        for b, row in enumerate(s["result"].tolist()):
            for i in range(row[1]):
                x, y = s["lens"][b].item() + row[3 + i], s["lens"][b].item() + 1 + i
                pages[:, table[b][y // page], :, y % page] = codes[:, table[b][x // page], :, x % page]
        got[name] = _e4m3(pages)
    return dict(got, lens=None)


def _exact_fork(s):
    table, page, free = s["table"].tolist(), s["page"], s["free"].tolist()
    top = free[0]
    got = {}
    moves = []
    for a, t in zip(s["src"].tolist(), s["tokens"].tolist()):
        if t % page:
            moves.append((table[a][t // page], free[top], t % page))
            top -= 1
    for name in ("k", "v"):
        pages = s[name + "_pages"].clone()
        for x, y, n in moves:
            pages[:, y, :, :n] = pages[:, x, :, :n]
        got[name] = _e4m3(pages)
    return dict(got, shortage=None, table=None, held=None, refs=None, free=None)


def exact(case, seed):
    op = case["op"]
    if op == "resize":
        return None  # whole numbers alone
    s = prepare(case, seed)
    return dict(attention=_exact_attention, append=_exact_append, compact=_exact_compact, fork=_exact_fork)[op](s)
