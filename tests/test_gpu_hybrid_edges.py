"""GPU parity of the gated delta rule, the rotary append and the token log probabilities against oracle/ where sizes,
lengths and values go to their ends.  Pages "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x Faster on
Jetson AGX Thor", sections on KV-cache reuse (a hybrid's recurrent states are kept with its pages) and tree-based
multi-token prediction.

The bounds of the delta rule are oracle/delta.py's, taken as tests/test_gpu_hybrid.py takes them."""
import numpy as np
import pytest
import torch

import gpu_util as U
import test_gpu_hybrid as T

pytestmark = pytest.mark.gpu
BF, FP = T.BF, T.FP


@pytest.fixture(scope="module", autouse=True)
def _lib():
    U.require_gpu_lib()


def scaled_values(c, at, ratio):
    c.v[:, at] *= ratio
    c.vf = c.v.float().cpu().numpy()


# ----------------------------------------------------------------------------------------------- forgotten values


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,shape", [(4, (1, 2, 128, 64)), (8, (1, 2, 64, 64)), (33, (1, 2, 128, 64)),
                                     (64, (1, 1, 256, 64)), (130, (1, 2, 128, 64)), (200, (1, 1, 64, 64))])
@pytest.mark.parametrize("decay", [-12.0, -30.0, -np.inf])
@pytest.mark.parametrize("ratio", [1e4, 1e7, 1e10])
def test_tokens_behind_a_large_forgotten_one(dtype, M, shape, decay, ratio):
    """A token's value `ratio` times the others', and the next token's decay takes it away: what follows keeps the
    bits that its own sizes ask for."""
    c = T.Delta(dtype, 2, M, *shape, seed=M)
    for at in (0, M // 2):
        scaled_values(c, at, ratio)
        if at + 1 < M:
            c.g[:, at + 1] = decay
    c.check_chain(*c.chain())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,shape", [(3, (1, 2, 128, 64)), (12, (1, 2, 64, 64)), (30, (1, 1, 256, 64)),
                                     (48, (1, 2, 128, 64)), (60, (1, 1, 256, 64)), (64, (1, 2, 64, 64))])
@pytest.mark.parametrize("ratio", [1e4, 1e10, 1e25])
def test_nodes_beside_a_large_sibling(dtype, M, shape, ratio):
    """Node 1 and every fifth one have a large value; the others hang on the root and on each other and see none."""
    rng = np.random.default_rng(M)
    c = T.Delta(dtype, 2, M, *shape, seed=M)
    large = [v for v in range(1, M) if v % 5 == 1]
    scaled_values(c, large, ratio)
    parent = np.full((2, M), -1, dtype=np.int32)
    for b in range(2):
        for v in range(1, M):
            parent[b, v] = rng.choice([u for u in range(max(0, v - 6), v) if u not in large])
    T.check_tree(c, parent, T.run_tree(c, parent))


# ----------------------------------------------------------------------------------------------- rounds


def some_heads(c, out, states, heads):
    """The step c, its outputs and its states, of some value heads alone (heads are independent of each other)."""
    nb, M, Hk, H, Dk, Dv = c.dims
    kh = np.asarray(heads) // (H // Hk)
    for name in ("q", "k", "qf", "kf"):
        setattr(c, name, getattr(c, name)[:, :, kh])
    for name in ("v", "vf", "g", "beta"):
        setattr(c, name, getattr(c, name)[:, :, heads])
    c.states = np.ascontiguousarray(c.states[:, heads])
    c.dims = (nb, M, len(heads), len(heads), Dk, Dv)
    return out[:, :, heads], states[:, heads].contiguous()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_states_carried_from_round_to_round(dtype):
    """1,024 heads: a round has room for a few blocks.  A sequence that reaches the last round, one that ends in the
    first, and one that begins from zeros."""
    M, heads = 430, [0, 255, 256, 700, 1023]
    c = T.Delta(dtype, 3, M, 4, 1024, 64, 64, counts=[M, 130, 300], slots=5, src=[0, 1, -1], dst=[3, 1, 4], seed=5,
                decay=5.0)
    need = T.B.load().nvfp4_delta_rule_workspace_bytes(3, M, 4, 1024, 64, 64, T.B.NVFP4_BF16 if dtype == BF else T.B.NVFP4_F32)
    assert need <= 128 << 20
    out, states = c.chain()
    c.check_chain(*some_heads(c, out, states, heads))


# ----------------------------------------------------------------------------------------------- every form


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Dk", [64, 128, 256])
@pytest.mark.parametrize("M", [5, 16, 17, 32, 33, 48, 49, 64, 65])
def test_blocks_of_every_width(dtype, Dk, M):
    """Chains and trees at the ends of each number of row tiles, ragged, with roots and decays at their ends."""
    rng = np.random.default_rng(M)
    c = T.Delta(dtype, 4, M, 1, 3, Dk, 64, counts=[M, M - 1, (M + 1) // 2, 0], slots=9, src=[0, -1, 2, 3],
                dst=[4, 5, 6, 7], seed=M + Dk)
    c.g[:, ::5, 0] = -np.inf
    c.g[:, :, 1], c.beta[:, :, 1] = 0.0, 1.0
    c.g[:, :, 2] *= 300
    c.check_chain(*c.chain())
    if M > 64:
        return
    c.counts, c.src = [M, M - 1, M, 0], np.array([0, -1, 99, 3], dtype=np.int32)
    parent = T.random_trees(rng, 4, M)
    parent[:, 3], parent[0, M // 2], parent[1, 4] = -1, M, 4
    got = T.run_tree(c, parent)
    T.check_tree(c, parent, got)
    for x in got:
        assert not x[1, M - 1:].any() and not x[2:].any()


@pytest.mark.parametrize("nb,M", [(2, 65), (2, 200), (3, 130), (6, 100)])
def test_several_sequences_of_the_models_shape(nb, M):
    """16 key and 48 value heads of 128: from two sequences on a workgroup has 64 columns of a state."""
    heads = [0, 1, 20, 47]
    c = T.Delta(BF, nb, M, 16, 48, 128, 128, counts=[M, 70, M - 1, 64, 1, 0][:nb], seed=M, decay=4.0)
    out, states = c.chain()
    c.check_chain(*some_heads(c, out, states, heads))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (256, 128)])
def test_several_sequences_of_many_heads(dtype, Dk, Dv):
    c = T.Delta(dtype, 3, 135, 8, 64, Dk, Dv, counts=[135, 64, 100], seed=Dk, decay=4.0)
    out, states = c.chain()
    c.check_chain(*some_heads(c, out, states, [0, 7, 33, 63]))


# ----------------------------------------------------------------------------------------------- NaN and infinity


def lines_of(parent):
    seen = np.eye(len(parent), dtype=bool)
    for v, p in enumerate(parent):
        if 0 <= p < v:
            seen[v] |= seen[p]
    return seen


def spoil(c, b, t, what, value):
    """Puts value into one place of token t of sequence b: of head 1's (and key head 0's) of four heads."""
    if what in ("k", "q", "v"):
        getattr(c, what)[b, t, 0 if what != "v" else 1, 3] = value
    else:
        getattr(c, what)[b, t, 1] = value


SPOILT = [("k", np.nan), ("k", np.inf), ("q", np.nan), ("v", np.nan), ("v", -np.inf), ("g", np.nan), ("g", np.inf),
          ("beta", np.nan), ("beta", -np.inf)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("what,value", SPOILT)
@pytest.mark.parametrize("M,Dk", [(7, 128), (16, 64), (33, 128), (64, 64), (50, 256)])
def test_a_spoilt_node_reaches_what_sees_it(dtype, what, value, M, Dk):
    """Other branches, and where a value is spoilt other columns, keep every bit; a path without the node commits."""
    c = T.Delta(dtype, 2, M, 2, 4, Dk, 64, src=[0, 1], slots=2, seed=M)
    parent = T.random_trees(np.random.default_rng(M), 2, M)
    parent[:, 2] = 0
    ref = [x.clone() for x in T.run_tree(c, parent)]
    spoil(c, 0, 2, what, value)
    out, keys, updates = T.run_tree(c, parent)
    seen = lines_of(parent[0])[:, 2]
    assert seen.any() and not seen.all()
    heads = [0, 1] if what in ("k", "q") else [1]
    hit = torch.zeros((2, M, 4, 64), dtype=torch.bool, device=T.DEV)
    for h in heads:
        rows = torch.from_numpy(np.flatnonzero(seen)).to(T.DEV)
        if what == "q":
            hit[0, 2, h] = True
        elif what == "v":
            hit[0, rows, h, 3] = True
        else:
            hit[0, rows, h] = True
    bad = lambda x: ~x.float().isfinite()  # noqa: E731
    assert torch.equal(bad(out), hit)
    assert torch.equal(out[~hit], ref[0][~hit])
    if what == "q":
        hit = torch.zeros_like(hit)
    assert torch.equal(bad(updates), hit) and torch.equal(updates[~hit], ref[2][~hit])
    spoilt_keys = torch.zeros((2, M, 2), dtype=torch.bool, device=T.DEV)
    spoilt_keys[0, 2, 0] = what == "k"
    assert torch.equal(bad(keys).any(-1), spoilt_keys) and torch.equal(keys[~spoilt_keys], ref[1][~spoilt_keys])
    # the longest path without the node, and one through it
    g = torch.nan_to_num(T.floats(c.g), 0.0, 0.0) if what == "g" else T.floats(c.g)
    for through in (False, True):
        v = max(i for i in range(M) if seen[i] == through)
        path = [i for i in range(1, M) if lines_of(parent[0])[v, i]]
        result = T.ints([[v, len(path), 0] + path + [-1] * (M - len(path)), [0, 0, 0] + [-1] * M])
        states = [T.floats(c.states)[None] for _ in range(2)]
        for st, k, u in zip(states, (keys, ref[1]), (updates, ref[2])):
            T.B.nvfp4_delta_commit(st, k[None], u[None], g[None], result, T.ints([0, 1]), T.ints([0, 1]))
        gone = bad(states[0])
        if through and what != "q":
            assert gone[0, 0, heads].any(-1).any(-1).all() and not gone[0, 0, 2:].any() and not gone[0, 1].any()
            assert what != "v" or torch.equal(gone[0, 0, 1].any(-1).nonzero()[:, 0].cpu(), torch.tensor([3]))
        else:
            assert torch.equal(states[0], states[1])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("what,value", SPOILT)
@pytest.mark.parametrize("M,at", [(3, 1), (9, 4), (40, 17), (64, 63), (150, 20), (150, 64), (200, 149), (2200, 700)])
def test_a_spoilt_token_reaches_what_follows(dtype, what, value, M, at):
    c = T.Delta(dtype, 2, M, 2, 4, 64, 64, src=[0, 1], dst=[2, 3], slots=4, seed=M, decay=4.0)
    ref, ref_states = (x.clone() for x in c.chain())
    spoil(c, 0, at, what, value)
    out, states = c.chain()
    heads, columns = [0, 1] if what in ("k", "q") else [1], 3 if what == "v" else slice(None)
    hit = torch.zeros((2, M, 4, 64), dtype=torch.bool, device=T.DEV)
    for h in heads:
        hit[0, at if what == "q" else slice(at, None), h, columns] = True
    assert torch.equal(out[~hit], ref[~hit])
    assert not out[hit].float().isfinite().any()
    lost = torch.zeros((4, 4, 64), dtype=torch.bool, device=T.DEV)
    for h in heads:
        lost[2, h, columns] = what != "q"
    assert torch.equal(states[~lost], ref_states[~lost])
    assert not states[lost].isfinite().all(-1).any()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [2, 30, 64, 130])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_a_spoilt_row_of_a_state_stays_in_its_column(dtype, M, value):
    c = T.Delta(dtype, 2, M, 1, 2, 128, 64, src=[0, 1], dst=[0, 1], slots=2, seed=M)
    ref, ref_states = (x.clone() for x in c.chain())
    c.states[0, 1, 7, 5] = value
    out, states = c.chain()
    hit = torch.zeros((2, M, 2, 64), dtype=torch.bool, device=T.DEV)
    hit[0, :, 1, 7] = True
    assert torch.equal(out[~hit], ref[~hit]) and not out[hit].float().isfinite().any()
    assert not states[0, 1, 7].isfinite().all()
    states[0, 1, 7] = ref_states[0, 1, 7]
    assert torch.equal(states, ref_states)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [4, 9, 40, 64, 100])
def test_a_key_that_has_no_direction_reaches_what_sees_it(dtype, M):
    """Zeros divided by their length with norm_eps 0 are NaN: of that token's key head, from that token on."""
    c = T.Delta(dtype, 2, M, 2, 4, 64, 64, src=[0, 1], dst=[2, 3], slots=4, seed=M)
    c.eps = 0.0
    parent = T.random_trees(np.random.default_rng(M), 2, M)
    parent[:, 2] = 0
    ref, ref_states = (x.clone() for x in c.chain())
    tree_ref = [x.clone() for x in T.run_tree(c, parent)] if M <= 64 else None
    c.k[0, 2, 0] = 0
    out, states = c.chain()
    hit = torch.zeros((2, M, 4, 64), dtype=torch.bool, device=T.DEV)
    hit[0, 2:, :2] = True
    assert torch.equal(out[~hit], ref[~hit]) and not out[hit].float().isfinite().any()
    assert torch.equal(states[3], ref_states[3]) and torch.equal(states[2, 2:], ref_states[2, 2:])
    assert not states[2, :2].isfinite().all(-1).any()
    if tree_ref:
        out, keys, updates = T.run_tree(c, parent)
        hit[0] = False
        hit[0, torch.from_numpy(np.flatnonzero(lines_of(parent[0])[:, 2])).to(T.DEV), :2] = True
        for got, want in ((out, tree_ref[0]), (updates, tree_ref[2])):
            assert torch.equal(got[~hit], want[~hit]) and not got[hit].float().isfinite().any()


@pytest.mark.parametrize("M", [3, 20, 100])
def test_a_spoilt_state_without_tokens_is_copied_as_it_is(M):
    c = T.Delta(FP, 2, M, 1, 2, 64, 64, counts=[0, M], src=[0, 1], dst=[2, 3], slots=4, seed=M)
    c.states[0, 1, 7, 5], c.states[0, 0, 3, 2] = np.nan, np.inf
    _, states = c.chain()
    assert np.array_equal(states[2].cpu().numpy(), c.states[0], equal_nan=True) and states[3].isfinite().all()


# ----------------------------------------------------------------------------------------------- lengths of rows


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [1, 4, 5, 65])
@pytest.mark.parametrize("power,eps", [(70, 1e-6), (110, 1e-6), (-70, 0.0), (-110, 0.0), (-70, 1e-30), (62, 0.0)])
def test_rows_of_any_length_are_normalised(dtype, M, power, eps):
    """Rows whose squares are past fp32's range, or below it, at every form's number of tokens."""
    c = T.Delta(dtype, 1, M, 2, 4, 128, 64, seed=M)
    for name in ("q", "k"):
        x = getattr(c, name)
        x.copy_((x.double() * 2.0 ** power).to(dtype))
        if M > 2:  # rows of either size beside them
            x[:, 1] = x[:, 1].double().mul(2.0 ** -power).to(dtype)
        setattr(c, name + "f", x.float().cpu().numpy())
    c.eps = eps
    c.check_chain(*c.chain())
    parent = np.arange(M, dtype=np.int32)[None] - 1
    if M <= 64:
        T.check_tree(c, parent, T.run_tree(c, parent))


# ----------------------------------------------------------------------------------------------- commit


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 2, 7, 5, 0, -1, -2 ** 31])
def test_a_commit_of_any_written_length(length):
    """A length past the nodes counts as all of them, one below none as none, to the ends of its type."""
    rng = np.random.default_rng(0)
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    states, keys, updates, g = f32(1, 2, 1, 64, 64), f32(1, 1, 6, 1, 64), f32(1, 1, 6, 1, 64), -np.abs(f32(1, 1, 6, 1))
    got = []
    for n in (length, max(0, min(5, length))):
        st = T.floats(states)
        T.B.nvfp4_delta_commit(st, T.floats(keys), T.floats(updates), T.floats(g), T.ints([[0, n, 0, 1, 2, 3, 4, 5, -1]]),
                               T.ints([0]), T.ints([1]))
        got.append(st)
    assert torch.equal(*got)
def test_a_commit_of_padded_trees():
    """Sequences without tokens, with some and with all; what stands in g behind them is not read."""
    M = 12
    c = T.Delta(FP, 4, M, 1, 2, 64, 64, counts=[0, 5, M, -3], src=[0, 1, 2, -1], dst=[4, 5, 6, 7], slots=9, seed=3)
    parent = np.tile(np.arange(M, dtype=np.int32)[None] - 1, (4, 1))
    for b, n in enumerate(c.counts):
        c.g[b, max(0, n):] = np.nan
    out, keys, updates = T.run_tree(c, parent)
    path = list(range(1, M))
    result = T.ints([[M - 1, M - 1, 0] + path + [-1]] * 4)
    st = T.floats(c.states)
    T.B.nvfp4_delta_commit(st[None], keys[None], updates[None], T.floats(c.g)[None], result, T.ints(c.src), T.ints(c.dst),
                           counts=T.ints(c.counts))
    assert torch.equal(st[4], T.floats(c.states)[0]) and not st[7].any()  # no tokens: the state is copied
    after, off = c.chain_ref()[2:4]
    err = np.sqrt(((st.double().cpu().numpy() - after) ** 2).sum(-1))
    assert (err <= 8 * off + 100 * 2.0 ** -23 * np.sqrt((after ** 2).sum(-1))).all()
    with pytest.raises(ValueError, match="counts"):
        T.B.nvfp4_delta_commit(st[None], keys[None], updates[None], T.floats(c.g)[None], result, T.ints(c.src),
                               T.ints(c.dst), counts=T.ints([1]))




# ----------------------------------------------------------------------------------------------- log probabilities


def exact_row(z, token, top):
    """As oracle/logprobs.py, with the bounds of an fp32 implementation: every e^(z - m) is off by 2^-22 and by 2^-23
    |z - m| (the difference and its product with log2 e are rounded), and passes through at most 64 + N / 8192 roundings
    of sums (16 of a lane's batch, its batches, 9 of lanes and waves, the parts)."""
    lp, ent, best, ids = T.LP.row(z, token, top)
    m = z.max()
    d = z - m
    p = np.exp(d)
    w = p.sum()
    sums = (64 + len(z) / 8192) * 2.0 ** -24
    off = np.abs(np.where(p > 0, d, 0))
    rel = 2.0 ** -22 + 2.0 ** -23 * (p * off).sum() / w + sums
    # the largest's own 1 is exact
    small, l = 1 - 1 / w, np.log(w)
    t = (p * off).sum() / w
    t_off = (p * off * (2.0 ** -22 + 2.0 ** -23 * off + 2.0 ** -23)).sum() / w + t * (sums + rel)
    last = lambda y: 2.0 ** -23 * (abs(y + l) + 2 * l + abs(y))  # noqa: E731
    tol = lambda y: rel * small + last(y) + 1e-37 if np.isfinite(y) else 0.0  # noqa: E731
    return (lp, tol(lp)), (ent, rel * small + t_off + 2.0 ** -22 * (l + t) + 1e-37), (best, [tol(y) for y in best]), ids


def check_rows(t, tokens, top, got, rows):
    lp, ent, best, ids = got
    for i in rows:
        a, e, b, o = exact_row(t[i].double().cpu().numpy(), int(tokens[i]), top)
        assert np.array_equal(ids[i].cpu().numpy(), o), (i, ids[i].tolist(), o)
        assert abs(lp[i].item() - a[0]) <= a[1], (i, "logprob", lp[i].item(), a)
        assert abs(ent[i].item() - e[0]) <= e[1], (i, "entropy", ent[i].item(), e)
        assert (np.abs(best[i].double().cpu().numpy() - b[0]) <= b[1]).all(), (i, "top")


def some_logits(dtype, M, N, seed):
    """Rows as a model gives them, and in every eighth one maxima that rise or fall with every batch, come first or
    last, or stand in the middle."""
    g = torch.Generator(device=T.DEV).manual_seed(seed)
    t = torch.empty((M, N), dtype=dtype, device=T.DEV)
    for part in t.split(32):
        part.copy_(torch.randn(part.shape, generator=g, device=T.DEV) * 2)
    line = torch.linspace(-9, 9, N, device=T.DEV)
    for i, row in enumerate(t):
        if i % 8 == 1:
            row.copy_(line)
        elif i % 8 == 2:
            row.copy_(-line)
        elif i % 8 in (3, 4, 5):
            row[{3: 0, 4: N - 1, 5: N // 2}[i % 8]] = 15.0
    return t


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,N,top", [(600, 20000, 7), (512, 151936, 5), (512, 151936, 0), (520, 151935, 64),
                                     (64, 151936, 20), (16, 151936, 64), (2, 300000, 33), (600, 300000, 5),
                                     (1, 600000, 64), (3, 1000003, 10), (300, 50257, 1)])
def test_logprobs_of_rows_of_many_batches(dtype, M, N, top):
    """One part a row, several, more than 64, and more blocks than LDS has room for."""
    t = some_logits(dtype, M, N, N)
    tokens = torch.randint(0, N, (M,), device=T.DEV, dtype=torch.int32)
    got = T.B.nvfp4_token_logprobs(t, tokens, top)
    rows = sorted({i for i in list(range(8)) + [M // 2, M - 1] if i < M})
    check_rows(t, tokens, top, got, rows)
    if top:  # the others: their first one, and a sum of p that is 1
        z = t.float()
        assert torch.equal(z.gather(1, got[3][:, :1].long())[:, 0], z.max(1).values)
        assert (got[0] <= got[2][:, 0]).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,N", [(1, 50257), (600, 50257), (1, 151935), (3, 151936), (520, 151937), (2, 600001)])
def test_logprobs_count_every_column_once(dtype, M, N):
    """Equal logits: whole numbers are summed, exactly, and a column more or less is 1 / N of the sum."""
    t = torch.full((M, N), -3.25, dtype=dtype, device=T.DEV)
    lp, ent, best, ids = T.B.nvfp4_token_logprobs(t, torch.full((M,), N - 1, device=T.DEV, dtype=torch.int32), 3)
    want = -np.log(N)  # of log1p: 2^-23 of it, and rounded once more (up to 160,000 columns that tells half of one)
    assert np.abs(lp.double().cpu().numpy() - want).max() <= 2.0 ** -22 * -want
    assert np.abs(ent.double().cpu().numpy() + want).max() <= 2.0 ** -22 * -want
    assert (ids == torch.arange(3, device=T.DEV)).all() and torch.equal(best, lp[:, None].expand(-1, 3))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,N", [(4, 700), (4, 20000), (600, 20000), (2, 300000)])
def test_logprobs_order_zeros_across_blocks(dtype, M, N):
    """+0.0 in some blocks of a row of -0.0, first, last and in the middle of a block."""
    t = torch.full((M, N), -0.0, dtype=dtype, device=T.DEV)
    at = [N - 1, N // 2, 64 * 5, 64 * 5 + 31, 64 * 7 - 1, 1]
    t[:, at] = 0.0
    _, _, _, ids = T.B.nvfp4_token_logprobs(t, torch.zeros((M,), device=T.DEV, dtype=torch.int32), 8)
    want = sorted(set(at)) + [c for c in range(N) if c not in at][: 8 - len(set(at))]
    assert ids.tolist() == [want] * M


# ----------------------------------------------------------------------------------------------- rotary append


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("start", [0, 60000, 1 << 20, (1 << 24) + 1, (1 << 27) - 40, (1 << 29) + 3])
def test_turns_are_those_of_64_bits(dtype, interleaved, start):
    """The angle is off by 2^-51 of the position (three roundings here and one in the oracle, each 2^-53 of it), sine
    and cosine by 2e-11 together with that of the oracle: a query is off by its roundings to fp32 and to its type and
    that much of its pair's size, and a key's code is the nearest but within that of the middle of two."""
    n = 120
    c = T.Rope(dtype, [start], n, 2, 3, 128, 128, 1024, interleaved=interleaved, scale=1.25, seed=9)
    q, pages = c.gpu()
    positions = start + np.arange(n)
    angle = 4e-11 + positions[:, None, None] * 2.0 ** -51
    ref, size = T.RP.rotate(c.qf[0].astype(np.float64), positions, c.inv, c.scale, interleaved)
    half = 2.0 ** -24 + (2.0 ** -8 if dtype == BF else 0.0)
    err = np.abs(q[0].double().cpu().numpy() - ref)
    assert (err <= half * np.abs(ref) + 1.01 * angle * size + 1e-44).all(), (err / (half * np.abs(ref) + angle * size)).max()
    inv = float(np.float32(1) / T.KS)
    ref, size = T.RP.rotate(c.kf[0].astype(np.float64), positions, c.inv, c.scale, interleaved)
    grid = T.KV.decode_f32(np.arange(127, dtype=np.uint8), np.float32(1.0)).astype(np.float64)
    grid = np.concatenate([-grid[:0:-1], grid])
    mid = (grid[1:] + grid[:-1]) / 2
    near = angle * size * inv + 2.0 ** -52 * np.abs(ref) * inv
    low, high = (grid[np.searchsorted(mid, ref * inv + s * near)] for s in (-1, 1))
    k = pages[0].cpu().numpy()
    for t in range(n):
        page, at = T.KC._slot(k, c.table, 0, start + t)
        got = T.KV.decode_f32(k[page, :, at], np.float32(1.0)).astype(np.float64)
        assert ((got == low[t]) | (got == high[t])).all(), t


# ----------------------------------------------------------------------------------------------- graphs


def every_call():
    """One call of each operator and form: (run, what it writes or NULL where it allocates that, how many of these count:
    a workspace behind them does not)."""
    made = []
    for dtype, nb, M, shape in ((BF, 2, 1, (2, 4, 128, 128)), (FP, 1, 9, (1, 2, 64, 64)), (BF, 1, 150, (1, 2, 128, 128)),
                                (FP, 2, 70, (1, 2, 64, 64)), (BF, 3, 70, (8, 48, 128, 128))):
        c = T.Delta(dtype, nb, M, *shape, seed=M)
        rows, kw = c.common()
        st, s, d = T.floats(c.states), T.ints(c.src), T.ints(c.dst)
        out = torch.empty_like(rows[2])
        need = T.B.load().nvfp4_delta_rule_workspace_bytes(nb, M, *shape, T.B.NVFP4_BF16 if dtype == BF else T.B.NVFP4_F32)
        ws = torch.empty((need,), dtype=torch.uint8, device=T.DEV) if need else None
        made.append((lambda rows=rows, st=st, s=s, d=d, out=out, ws=ws, kw=kw: T.B.nvfp4_delta_rule(
            *rows, st, s, d, out=out, workspace=ws, **kw), [out, st] + ([ws] if need else []), 2))
    c = T.Delta(FP, 2, 23, 1, 2, 64, 64, counts=[23, 0], seed=2)
    rows, kw = c.common()
    parent = T.ints(T.random_trees(np.random.default_rng(0), 2, 23))
    st, s, d = T.floats(c.states), T.ints(c.src), T.ints(c.dst)
    out, keys, updates = torch.empty_like(rows[2]), torch.empty((2, 23, 1, 64), device=T.DEV), torch.empty((2, 23, 2, 64), device=T.DEV)
    made.append((lambda: T.B.nvfp4_delta_tree(*rows, st, s, parent, out=out, keys=keys, updates=updates, **kw),
                 [out, keys, updates], 3))
    k2, u2 = torch.randn((1, 2, 23, 1, 64), device=T.DEV), torch.randn((1, 2, 23, 2, 64), device=T.DEV)
    cst, g, counts = T.floats(c.states)[None], T.floats(c.g)[None], T.ints([23, 0])
    result = T.ints([[0, 2, 0, 1, 4] + [-1] * 21, [0, 0, 0] + [-1] * 23])
    made.append((lambda: T.B.nvfp4_delta_commit(cst, k2, u2, g, result, s, d, counts=counts), [cst], 1))
    r = T.Rope(BF, [40, 7], 16, 4, 2, 128, 64, 16, tree=True)
    pages = [torch.from_numpy(x.copy()).to(T.DEV) for x in r.start]
    inv, ks, vs, tab, lens, par = (torch.from_numpy(r.inv).to(T.DEV), U.scalar(T.KS), U.scalar(T.VS), T.ints(r.table),
                                   T.ints(r.lens), T.ints(r.parent))
    q_out = torch.empty_like(r.q)
    made.append((lambda: T.B.nvfp4_kv_append_rope(r.q, r.k, r.v, inv, ks, vs, *pages, tab, lens, parent=par, q_out=q_out),
                 [q_out] + pages, 3))
    for M, N in ((16, 9001), (600, 3000)):
        z, tokens = T.typed(np.random.default_rng(3).standard_normal((M, N)) * 3, FP)[0], T.ints(np.arange(M))
        made.append((lambda z=z, tokens=tokens: T.B.nvfp4_token_logprobs(z, tokens, 20), None, 4))
    return made


def test_replays_write_every_output_anew():
    """Before each replay everything that a call writes holds what it starts from, or nothing of use."""
    runs = every_call()
    def begin(seed):
        g = torch.Generator(device=T.DEV).manual_seed(seed)
        for _, bufs, _ in runs:
            for x in bufs or []:
                if x.dtype is torch.uint8:
                    x.copy_(torch.randint(0, 256, x.shape, generator=g, device=T.DEV, dtype=torch.uint8))
                else:
                    x.copy_(torch.randn(x.shape, generator=g, device=T.DEV))

    def results(outs):
        return [[x.clone() for x in (bufs or out)[:n]] for (_, bufs, n), out in zip(runs, outs)]

    begin(0)
    for run, _, _ in runs:
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [run() for run, _, _ in runs]
    for seed in (1, 2, 1):
        begin(seed)
        want = results([run() for run, _, _ in runs])
        begin(seed)
        for (_, bufs, _), out in zip(runs, held):
            if bufs is None:
                for x in out:
                    x.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (got, ref) in enumerate(zip(results(held), want)):
            for x, y in zip(got, ref):
                assert torch.equal(x, y), (seed, i)
