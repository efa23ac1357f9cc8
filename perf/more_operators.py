"""The cases by which the operators of a hybrid model's decode step are measured, with their plain forms.

Next to the paged attention layers such a model has layers with a recurrent state: nvfp4_delta_rule runs the gated delta
rule over a chain of tokens, nvfp4_delta_tree over a drafted tree, without touching the states, and nvfp4_delta_commit
puts the accepted path into them.  nvfp4_kv_append_rope gives queries and keys their rotary positions on the way into
the cache.  nvfp4_token_logprobs scores tokens under the LM head's logits.  Where `own` is false, run() computes them
with elementary torch operations; where it is true, it calls the library.  exact() has the same results from the
definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64  # tokens of a block in the plain delta rule, at most


def listed():
    return [
        # one token of one conversation: the smallest call, all latency
        dict(name="delta_one", op="delta", dtype="bf16", seqs=1, nodes=1, key_heads=16, heads=48, dk=128, dv=128,
             norm=True, ragged=False),
        # the next token of a batch of conversations: all states read and written
        dict(name="delta_batch", op="delta", dtype="bf16", seqs=64, nodes=1, key_heads=16, heads=48, dk=128, dv=128,
             norm=True, ragged=False),
        # the suffix of a new turn, from the state that the turn before it left
        dict(name="delta_suffix_512", op="delta", dtype="bf16", seqs=1, nodes=512, key_heads=16, heads=48, dk=128,
             dv=128, norm=True, ragged=False),
        # prompts of new conversations, each with its own length, in float32
        dict(name="delta_prompts_f32", op="delta", dtype="f32", seqs=3, nodes=4099, key_heads=4, heads=8, dk=64,
             dv=128, norm=False, ragged=True),
        # a 16-node drafted tree of one conversation
        dict(name="tree_16", op="tree", dtype="bf16", seqs=1, nodes=16, key_heads=16, heads=48, dk=128, dv=128,
             norm=True, ragged=False),
        # a ragged batch of wider trees in float32
        dict(name="tree_ragged_f32", op="tree", dtype="f32", seqs=16, nodes=33, key_heads=4, heads=8, dk=64, dv=128,
             norm=False, ragged=True),
        # the accepted path of one tree, in all recurrent layers
        dict(name="commit_one", op="commit", layers=48, seqs=1, nodes=16, key_heads=16, heads=48, dk=128, dv=128),
        # a batch of accepted paths in a few layers
        dict(name="commit_batch", op="commit", layers=5, seqs=24, nodes=33, key_heads=4, heads=8, dk=64, dv=128),
        # the 16 nodes of a drafted tree at the end of the longest agent context, one layer
        dict(name="rope_tree", op="rope", dtype="bf16", seqs=1, nodes=16, tree=True, heads=8, group=5, dim=128,
             rotary=64, interleaved=False, scaling="none", page=64, context=23552, ragged=False),
        # prompts in float32 at far positions of a stretched context
        dict(name="rope_prompts_f32", op="rope", dtype="f32", seqs=4, nodes=2047, tree=False, heads=8, group=2,
             dim=128, rotary=128, interleaved=True, scaling="yarn", page=64, context=60000, ragged=False),
        # the rows of a verified tree, twenty alternatives each
        dict(name="logprobs_tree", op="logprobs", dtype="f32", rows=16, vocab=151936, top=20),
        # the tokens of a suffix scored
        dict(name="logprobs_suffix", op="logprobs", dtype="bf16", rows=512, vocab=151936, top=5),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "tree", "tree", "commit", "rope", "logprobs"])
    key_heads, heads = rng.choice([(1, 1), (1, 4), (2, 4), (4, 4), (4, 8), (5, 15), (8, 16), (16, 32), (16, 48)])
    dk, dv = rng.choice([64, 128, 128, 256]), rng.choice([64, 128, 128, 256])
    shape = dict(key_heads=key_heads, heads=heads, dk=dk, dv=dv)
    state = heads * dk * dv
    if op == "delta":
        seqs = log_int(rng, 1, max(1, min(64, 50_000_000 // state)))
        nodes = log_int(rng, 1, max(2, min(4100, 400_000_000 // (state * seqs), 12000 // seqs)))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), seqs=seqs, nodes=nodes,
                    norm=rng.random() < 0.6, ragged=rng.random() < 0.4, **shape)
    if op == "tree":
        seqs = log_int(rng, 1, max(1, min(32, 25_000_000 // state)))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), seqs=seqs, nodes=log_int(rng, 1, 64),
                    norm=rng.random() < 0.6, ragged=rng.random() < 0.4, **shape)
    if op == "commit":
        layers = log_int(rng, 1, max(1, min(48, 37_000_000 // state)))
        return dict(op=op, layers=layers, seqs=log_int(rng, 1, max(1, min(24, 37_000_000 // (state * layers)))),
                    nodes=log_int(rng, 1, 64), **shape)
    if op == "rope":
        tree = rng.random() < 0.5
        seqs = log_int(rng, 1, 40)
        dim = rng.choice([64, 128, 256])
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), seqs=seqs,
                    nodes=log_int(rng, 1, 64 if tree else 4000 // seqs), tree=tree, heads=rng.choice([1, 2, 4, 5, 8]),
                    group=rng.choice([1, 2, 3, 5]), dim=dim, rotary=rng.choice([32, dim // 2, dim]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    page=rng.choice([16, 32, 64, 128]), context=log_int(rng, 1, 200_000 // seqs),
                    ragged=rng.random() < 0.3)
    vocab = log_int(rng, 1000, 260_000)
    return dict(op="logprobs", dtype=rng.choice(["bf16", "f32"]), rows=log_int(rng, 1, min(512, 60_000_000 // vocab)),
                vocab=vocab, top=rng.choice([1, 2, 5, 8, 20, 50]))


# ---------------------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _randint(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


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
    ends = _randint(g, 0, parent.shape[1], (parent.shape[0],)).tolist()
    for up, end in zip(parent.tolist(), ends):
        path, v = [], end
        while v > 0:
            path.append(v)
            v = up[v]
        rows.append([end, len(path), 17] + path[::-1] + [-1] * (len(up) - len(path)))
    return _ints(rows)


def _decays(g, *shape):
    """Log decays of a trained layer: most heads forget slowly, some tokens wipe much of the state."""
    return -torch.exp(1.5 * _randn(g, *shape) - 3.0)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _frequencies(case):
    """Radians per position of each rotated pair in 64 bits, and the factor of the rotated values."""
    R, base, factor, trained = case["rotary"], 10000.0, 8.0, 8192
    if case["scaling"] == "ntk":
        base *= factor ** (R / (R - 2))
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] != "yarn":
        return f.to(DEV), 1.0
    # pairs that turn often within the trained length stay, those that turn less than once are stretched
    turns = trained * f / (2 * math.pi)
    stay = ((turns.log2()) / math.log2(32.0)).clamp(0, 1)
    return (f * stay + f / factor * (1 - stay)).to(DEV), 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op, B = case["op"], case.get("seqs")
    if op in ("delta", "tree"):
        M, Hk, H, dk, dv = (case[n] for n in ("nodes", "key_heads", "heads", "dk", "dv"))
        # keys of a layer are not independent: they share a mean direction
        k = _randn(g, B, M, Hk, dk) + 0.5 * _randn(g, B, 1, Hk, dk)
        q = _randn(g, B, M, Hk, dk)
        if not case["norm"]:
            q, k = _unit(q), _unit(k)
        s["q"], s["k"], s["v"] = (x.to(_dtype(case)) for x in (q, k, _randn(g, B, M, H, dv)))
        s["g"], s["beta"] = _decays(g, B, M, H), torch.sigmoid(1.5 * _randn(g, B, M, H))
        slots = torch.randperm(2 * B, generator=g, device=DEV).to(torch.int32)
        s["states"] = _randn(g, 2 * B, H, dv, dk) * (2.0 / math.sqrt(dk))
        s["src"], s["dst"] = slots[:B].contiguous(), slots[B:].contiguous()
        s["counts"] = _randint(g, 1, M + 1, (B,)) if case["ragged"] else None
        if op == "tree":
            s["parent"] = _trees(g, B, M)
        elif case["ragged"]:
            s["src"][::2] = -1  # every other conversation is new
    elif op == "commit":
        L, M, Hk, H, dk, dv = (case[n] for n in ("layers", "nodes", "key_heads", "heads", "dk", "dv"))
        s["keys"], s["updates"] = _unit(_randn(g, L, B, M, Hk, dk)), _randn(g, L, B, M, H, dv)
        s["g"] = _decays(g, L, B, M, H)
        slots = torch.randperm(2 * B, generator=g, device=DEV).to(torch.int32)
        s["states"] = torch.empty((L, 2 * B, H, dv, dk), device=DEV)
        for layer in s["states"]:
            layer.copy_(_randn(g, *layer.shape) * (2.0 / math.sqrt(dk)))
        s["src"], s["dst"] = slots[:B].contiguous(), slots[B:].contiguous()
        s["result"] = _accepted(g, _trees(g, B, M))
    elif op == "rope":
        M, H, D, page = case["nodes"], case["heads"], case["dim"], case["page"]
        lens = _randint(g, 0, case["context"] + 1, (B,)).tolist() if case["ragged"] else [case["context"]] * B
        # the new tokens' pages alone exist here: what the committed tokens' pages hold is not read
        first = [n // page for n in lens]
        need = [-(-(n + M) // page) - f for n, f in zip(lens, first)]
        pages = B * ((M + page - 2) // page + 1) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((B, max(f + n for f, n in zip(first, need))), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            s["table"][b, first[b]:first[b] + need[b]] = order[at:at + need[b]]
            at += need[b]
        s["k_pages"] = torch.zeros((pages, H, page, D), dtype=torch.uint8, device=DEV)
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        s["k_scale"] = s["v_scale"] = torch.full((1,), 8.0 / 448.0, device=DEV)
        s["lens"] = _ints(lens)
        s["counts"] = _randint(g, 1, M + 1, (B,)) if case["ragged"] else None
        s["parent"] = _trees(g, B, M) if case["tree"] else None
        s["q"] = _randn(g, B, M, H * case["group"], D).to(_dtype(case))
        s["k"], s["v"] = (_randn(g, B, M, H, D).to(_dtype(case)) for _ in range(2))
        s["inv_freq"], s["scale"] = _frequencies(case)
    else:
        rows, N = case["rows"], case["vocab"]
        # logits of a model that is sure of some tokens and torn on others
        s["logits"] = torch.empty((rows, N), dtype=_dtype(case), device=DEV)
        for part in s["logits"].split(64):
            part.copy_(2.0 * _randn(g, *part.shape))
        hot = torch.randint(0, N, (rows, 8), generator=g, device=DEV)
        lift = 6.0 + 6.0 * torch.rand((rows, 8), generator=g, device=DEV)
        s["logits"].scatter_(1, hot, lift.to(_dtype(case)))
        s["tokens"] = hot[:, 0].to(torch.int32)
    return s


# ---------------------------------------------------------------------------------------------- plain forms


def _inputs(s):
    """Queries, keys and values in 32 bits as [B, H, M, dim], normalised where the case asks for it; decays and rates."""
    group = s["heads"] // s["key_heads"]
    q, k, v = (s[n].float().transpose(1, 2) for n in ("q", "k", "v"))
    if s["norm"]:
        q, k = (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    keys = k
    q, k = (x.repeat_interleave(group, 1) for x in (q, k))
    g, beta = s["g"].transpose(1, 2), s["beta"].transpose(1, 2)
    if s["counts"] is not None:  # rows behind a sequence's last change nothing
        here = (torch.arange(s["nodes"], device=DEV)[None] < s["counts"][:, None])[:, None]
        g, beta = g * here, beta * here
        keys = keys * here[..., None]
        q, v = q * here[..., None], v * here[..., None]
    return q, k, v, g, beta, keys


def _start(s):
    """The states that the sequences begin with, as [B, H, dk, dv]."""
    begin = s["states"][s["src"].clamp(min=0).long()] * (s["src"] >= 0)[:, None, None, None]
    return begin.transpose(2, 3).contiguous()


def _blocks(x, n):
    """[B, H, M, ...] as [B, H, n, tokens of a block, ...], zeros behind M."""
    size = -(-x.shape[2] // n)
    x = torch.cat([x, x.new_zeros(x.shape[:2] + (n * size - x.shape[2],) + x.shape[3:])], 2)
    return x.view(x.shape[:2] + (n, size) + x.shape[3:])


def _solve(beta, decay, k, right):
    """(I + A)^-1 right, A = beta_i exp(G_i - G_j) k_i . k_j below the diagonal."""
    if k.shape[-2] == 1:
        return right
    near = torch.matmul(k, k.transpose(-1, -2).contiguous()) * decay * beta[..., None]
    return torch.linalg.solve_triangular(near.tril(-1), right, upper=False, unitriangular=True)


def _plain_delta(s):
    q, k, v, g, beta, _ = _inputs(s)
    M, dv = s["nodes"], s["dv"]
    n = -(-M // CHUNK)
    q, k, v, g, beta = (_blocks(x, n) for x in (q, k, v, g, beta))
    G = g.double().cumsum(-1)
    seen = torch.ones(G.shape[-1:] * 2, dtype=torch.bool, device=DEV).tril()
    far = (G[..., :, None] - G[..., None, :]).masked_fill(~seen, -math.inf)
    decay, into, out_of = far.exp().float(), G.exp().float(), (G[..., -1:] - G).exp().float()
    both = _solve(beta, decay, k, torch.cat([v * beta[..., None], k * (beta * into)[..., None]], -1))
    near, read = both[..., :dv], both[..., dv:]
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * decay
    late, q = (k * out_of[..., None]).transpose(-1, -2).contiguous(), q * into[..., None]
    state, rows = _start(s), []
    for c in range(n):  # a block needs the state that the one before it leaves
        u = near[:, :, c] - torch.matmul(read[:, :, c], state)
        rows.append(torch.matmul(q[:, :, c], state) + torch.matmul(score[:, :, c], u))
        state = state * into[:, :, c, -1, None, None] + torch.matmul(late[:, :, c], u)
    out = torch.cat(rows, 2)[:, :, :M] * (1.0 / math.sqrt(s["dk"]))
    s["states"][s["dst"].long()] = state.transpose(2, 3)
    return dict(out=out.transpose(1, 2).contiguous().to(s["v"].dtype), states=s["states"])


def _lines(parent):
    """[B, M, M] truth values: node u is v or an ancestor of v."""
    v = torch.arange(parent.shape[1], device=DEV)
    step = torch.eye(len(v), device=DEV) + (parent[:, :, None] == v).float()
    return torch.linalg.matrix_power(step, 64) > 0


def _plain_tree(s):
    q, k, v, g, beta, keys = _inputs(s)
    line = _lines(s["parent"])[:, None]
    G = torch.matmul(line.double(), g.double()[..., None])[..., 0]
    far = (G[..., :, None] - G[..., None, :]).masked_fill(~line, -math.inf)
    decay, into = far.exp().float(), G.exp().float()
    state = _start(s)
    u = _solve(beta, decay, k, beta[..., None] * (v - into[..., None] * torch.matmul(k, state)))
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * decay
    out = (into[..., None] * torch.matmul(q, state) + torch.matmul(score, u)) * (1.0 / math.sqrt(s["dk"]))
    return dict(out=out.transpose(1, 2).contiguous().to(s["v"].dtype), keys=keys.transpose(1, 2).contiguous(),
                updates=u.transpose(1, 2).contiguous())


def _plain_commit(s):
    L, B, M, group = s["layers"], s["seqs"], s["nodes"], s["heads"] // s["key_heads"]
    path = torch.cat([torch.zeros_like(s["result"][:, :1]), s["result"][:, 3:]], 1)[:, :M]  # the root, then the path
    here = torch.arange(M, device=DEV)[None] <= s["result"][:, 1:2]
    path = torch.where(here, path, torch.zeros_like(path)).long()

    def along(x):  # [L, B, M, H, ...] -> [L, B, H, M, ...] in the path's order
        index = path.view((1, B, M) + (1,) * (x.dim() - 3)).expand_as(x)
        return torch.gather(x, 2, index).transpose(2, 3)

    G = (along(s["g"]).double() * here[None, :, None]).cumsum(-1)
    weight = (G[..., -1:] - G).exp().float() * here[None, :, None]
    k = along(s["keys"]).repeat_interleave(group, 2)
    u = (along(s["updates"]) * weight[..., None]).transpose(-1, -2).contiguous()
    state = s["states"][:, s["src"].long()] * G[..., -1].exp().float()[..., None, None]
    s["states"][:, s["dst"].long()] = state + torch.matmul(u, k)
    return dict(states=s["states"])


def _plain_rope(s):
    B, M, R, dt = s["seqs"], s["nodes"], s["rotary"], s["q"].dtype
    v = torch.arange(M, device=DEV)
    depth = v[None] if s["parent"] is None else _lines(s["parent"]).sum(-1) - 1
    angle = (s["lens"][:, None] + depth).double()[..., None] * s["inv_freq"]  # far positions: 64 bits
    cos, sin = (f(angle).mul(s["scale"]).float()[:, :, None] for f in (torch.cos, torch.sin))

    def turned(x):
        x = x.float()
        if s["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
        else:
            a, b = x[..., : R // 2], x[..., R // 2:R]
        a, b = a * cos - b * sin, b * cos + a * sin
        near = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([near, x[..., R:]], -1)

    at = s["lens"][:, None] + v
    slot, entry = at % s["page"], torch.gather(s["table"].long(), 1, (at // s["page"]).long())
    here = torch.ones((B, M), dtype=torch.bool, device=DEV) if s["counts"] is None else v[None] < s["counts"][:, None]
    q = turned(s["q"]) * here[..., None, None]
    for x, scale, pages in ((turned(s["k"]), s["k_scale"], s["k_pages"]), (s["v"].float(), s["v_scale"], s["v_pages"])):
        y = (x * (1.0 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        if s["counts"] is None:
            pages[entry, :, slot] = y
        else:
            pages[entry[here], :, slot[here]] = y[here]
    return dict(_page_values(s), q=q.to(dt))


def _page_values(s):
    """The cache as the E4M3 values that its bytes stand for."""
    return dict(k=s["k_pages"].view(torch.float8_e4m3fn), v=s["v_pages"].view(torch.float8_e4m3fn))


def _plain_logprobs(s):
    z = s["logits"].float()
    N = s["vocab"]
    z_top = z.amax(-1, keepdim=True)
    e = torch.exp(z - z_top)
    total = e.sum(-1, keepdim=True)
    entropy = total.log() - (e * (z - z_top)).sum(-1, keepdim=True) / total
    lse = z_top + total.log()
    token = torch.gather(z, 1, s["tokens"].long()[:, None]) - lse
    # order by value, the lower index first: one whole number for both
    bits = z.view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits + 2 ** 31) - 1, bits)
    order = bits * 2 ** 32 + (2 ** 32 - 1 - torch.arange(N, device=DEV))
    best = 2 ** 32 - 1 - (torch.topk(order, s["top"], dim=-1).values & (2 ** 32 - 1))
    return dict(logprobs=token[:, 0], entropy=entropy[:, 0], top_logprobs=torch.gather(z, 1, best) - lse,
                top_tokens=best.to(torch.int32))


def run(s):
    if own:
        return _own(s)
    return dict(delta=_plain_delta, tree=_plain_tree, commit=_plain_commit, rope=_plain_rope,
                logprobs=_plain_logprobs)[s["op"]](s)


def _own(s):
    from nvfp4_w4a4_block_amd import binding as B
    op = s["op"]
    if op == "delta":
        out = B.nvfp4_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["src"], s["dst"],
                                 counts=s["counts"], norm_eps=1e-6 if s["norm"] else None)
        return dict(out=out, states=s["states"])
    if op == "tree":
        out, keys, updates = B.nvfp4_delta_tree(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["src"],
                                                s["parent"], counts=s["counts"], norm_eps=1e-6 if s["norm"] else None)
        return dict(out=out, keys=keys, updates=updates)
    if op == "commit":
        B.nvfp4_delta_commit(s["states"], s["keys"], s["updates"], s["g"], s["result"], s["src"], s["dst"])
        return dict(states=s["states"])
    if op == "rope":
        q = B.nvfp4_kv_append_rope(s["q"], s["k"], s["v"], s["inv_freq"], s["k_scale"], s["v_scale"], s["k_pages"],
                                   s["v_pages"], s["table"], s["lens"], parent=s["parent"], counts=s["counts"],
                                   interleaved=s["interleaved"], rope_scale=s["scale"])
        return dict(_page_values(s), q=q)
    logprobs, entropy, top_logprobs, top_tokens = B.nvfp4_token_logprobs(s["logits"], s["tokens"], s["top"])
    return dict(logprobs=logprobs, entropy=entropy, top_logprobs=top_logprobs, top_tokens=top_tokens)


# ---------------------------------------------------------------------------------------------- work


def work(case):
    op, B = case["op"], case.get("seqs")
    size = 2 if case.get("dtype") == "bf16" else 4
    if op in ("delta", "tree"):
        M, Hk, H, dk, dv = (case[n] for n in ("nodes", "key_heads", "heads", "dk", "dv"))
        rows = B * M * (0.5 if case["ragged"] else 1.0)
        moved = rows * (2 * Hk * dk * size + 8 * H + H * dv * size) + B * M * H * dv * size
        if op == "tree":
            return dict(bytes=moved + 4 * B * M * (Hk * dk + H * dv) + 4 * B * H * dk * dv,
                        flops=rows * H * (4 * dk * dv + 2 * (M / 2) * (dk + dv)))
        begun = B if not case["ragged"] else B // 2
        return dict(bytes=moved + 4 * (begun + B) * H * dk * dv, flops=7 * rows * H * dk * dv)
    if op == "commit":
        L, M, Hk, H, dk, dv = (case[n] for n in ("layers", "nodes", "key_heads", "heads", "dk", "dv"))
        path = B * max(1.0, 0.2 * M)  # a random end node's line holds about two nodes in five of those before it
        return dict(bytes=L * (8 * B * H * dk * dv + 4 * path * (Hk * dk + H * dv + H)),
                    flops=L * H * dk * dv * (B + 2 * path))
    if op == "rope":
        rows = B * case["nodes"] * (0.5 if case["ragged"] else 1.0)
        H, D = case["heads"], case["dim"]
        return dict(bytes=rows * H * D * (2 * case["group"] * size + 2 * size + 2),
                    flops=rows * H * (1 + case["group"]) * 3 * case["rotary"])
    return dict(bytes=case["rows"] * (case["vocab"] * size + 12 + 8 * case["top"]),
                flops=4 * case["rows"] * case["vocab"])


# ---------------------------------------------------------------------------------------------- exact results


def _exact_rows(s):
    """q, k, v, g, beta of the definition in 64 bits, [B, M, H, ...]."""
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    if s["norm"]:
        q, k = (x / ((x ** 2).sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    return q, k, v, s["g"].double(), s["beta"].double()


def _exact_step(state, q, k, v, g, beta):
    """One token: the state after it, what it writes and what it reads (before the factor); state [..., dv, dk]."""
    state = state * torch.exp(g)[..., None, None]
    u = beta[..., None] * (v - (state * k[..., None, :]).sum(-1))
    state = state + u[..., :, None] * k[..., None, :]
    return state, u, (state * q[..., None, :]).sum(-1)


def _exact_delta(s):
    q, k, v, g, beta = _exact_rows(s)
    group = s["heads"] // s["key_heads"]
    states = s["states"].double()
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    for b in range(s["seqs"]):
        src, dst = int(s["src"][b]), int(s["dst"][b])
        state = states[src].clone() if src >= 0 else torch.zeros_like(states[0])
        for t in range(s["nodes"] if s["counts"] is None else int(s["counts"][b])):
            kt, qt = (x[b, t].repeat_interleave(group, 0) for x in (k, q))
            state, _, out[b, t] = _exact_step(state, qt, kt, v[b, t], g[b, t], beta[b, t])
        states[dst] = state
    return dict(out=out / math.sqrt(s["dk"]), states=states)


def _exact_tree(s):
    q, k, v, g, beta = _exact_rows(s)
    group = s["heads"] // s["key_heads"]
    out, updates = (torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV) for _ in range(2))
    keys = torch.zeros_like(k)
    for b in range(s["seqs"]):
        parent, after = s["parent"][b].tolist(), []
        first = s["states"][int(s["src"][b])].double()
        for t in range(s["nodes"] if s["counts"] is None else int(s["counts"][b])):
            kt, qt = (x[b, t].repeat_interleave(group, 0) for x in (k, q))
            state, updates[b, t], out[b, t] = _exact_step(after[parent[t]] if t else first, qt, kt, v[b, t], g[b, t],
                                                          beta[b, t])
            keys[b, t] = k[b, t]
            after.append(state)
    return dict(out=out / math.sqrt(s["dk"]), keys=keys, updates=updates)


def _exact_commit(s):
    group = s["heads"] // s["key_heads"]
    states = s["states"].double()
    for b, row in enumerate(s["result"].tolist()):
        state = states[:, int(s["src"][b])].clone()
        for t in [0] + row[3:3 + row[1]]:
            k = s["keys"][:, b, t].double().repeat_interleave(group, 1)
            state = state * torch.exp(s["g"][:, b, t].double())[..., None, None]
            state = state + s["updates"][:, b, t].double()[..., :, None] * k[..., None, :]
        states[:, int(s["dst"][b])] = state
    return dict(states=states)


def _e4m3(codes):
    """The E4M3 values of bytes, from the format's definition, in 64 bits."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.bitwise_left_shift(torch.ones_like(e), e) * 2.0 ** -10)
    return torch.where(c >= 128, -mag, mag)


def _nearest_e4m3(y):
    """E4M3 value nearest to y, ties to the even code, at most 448 in magnitude."""
    grid = _e4m3(torch.arange(127, device=DEV))
    mid = (grid[1:] + grid[:-1]) / 2
    a = y.abs()
    up, down = torch.searchsorted(mid, a, right=True), torch.searchsorted(mid, a, right=False)
    at = torch.where(up % 2 == 0, up, down)  # equal unless a is a midpoint
    return torch.where(y < 0, -grid[at], grid[at])


def _exact_rope(s):
    R = s["rotary"]
    pairs = [(2 * j, 2 * j + 1) if s["interleaved"] else (j, j + R // 2) for j in range(R // 2)]
    a, b = (torch.tensor(x, device=DEV) for x in zip(*pairs))
    got = dict(k=_e4m3(s["k_pages"]), v=_e4m3(s["v_pages"]),
               q=torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV))
    for i, n in enumerate(s["lens"].tolist()):
        c = s["nodes"] if s["counts"] is None else int(s["counts"][i])
        depth = list(range(c))
        if s["parent"] is not None:
            parent = s["parent"][i].tolist()
            for t in range(c):
                depth[t] = depth[parent[t]] + 1 if t else 0
        angle = (n + torch.tensor(depth, device=DEV, dtype=torch.float64))[:, None, None] * s["inv_freq"]
        turn = torch.polar(torch.full_like(angle, s["scale"]), angle)
        at = torch.arange(n, n + c, device=DEV)
        for name in ("q", "k", "v"):
            x = s[name][i, :c].double()
            if name != "v":
                z = torch.complex(x[..., a], x[..., b]) * turn
                x[..., a], x[..., b] = z.real, z.imag
            if name == "q":
                got["q"][i, :c] = x
                continue
            y = _nearest_e4m3(x * (1.0 / s[name + "_scale"]).double())
            got[name][s["table"][i].long()[at // s["page"]], :, at % s["page"]] = y
    return got


def _exact_logprobs(s):
    parts = []
    for z, token in zip(s["logits"].split(32), s["tokens"].split(32)):
        p = torch.log_softmax(z.double(), -1)
        parts.append((torch.gather(p, 1, token.long()[:, None])[:, 0], -(p.exp() * p).sum(-1),
                      torch.topk(p, s["top"]).values))
    logprobs, entropy, top = (torch.cat(x) for x in zip(*parts))
    return dict(logprobs=logprobs, entropy=entropy, top_logprobs=top, top_tokens=None)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(delta=_exact_delta, tree=_exact_tree, commit=_exact_commit, rope=_exact_rope,
                logprobs=_exact_logprobs)[case["op"]](s)
