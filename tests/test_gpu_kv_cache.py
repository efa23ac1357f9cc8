"""GPU parity of the paged FP8 KV cache against oracle/kvcache.py: appended and compacted bytes, page
tables, counts and free lists exactly; attention within a bound derived from its roundings.  Pages
"TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x Faster on Jetson AGX Thor",
sections on the FP8 KV cache, tree-based multi-token prediction and KV-cache reuse.

The bound.  u = 2^-24.  A score is a sum of D products in fp32, scaled once: it is off by at most ez =
(D + 8) u * sum|q k_hat| * sm_scale, plus 4 u |z| for the steps from the score to the exponent.  Each
probability is then off by a factor within 2 ez (its own error and the statistics'), and rounded for the
product: 2^-11 of itself in bf16 calls (f16), 2^-22 in fp32 calls, or, where it is tiny, by at most 2^-32
of the largest one.  Sums over N tokens in fp32 add N u in numerator and denominator.  The result is
rounded to its type by at most half a step of itself.  All of it scales the softmax's mean of |v_hat|."""
import numpy as np
import pytest
import torch

import gpu_util as U
from nvfp4_w4a4_block_amd import binding as B
from oracle import kvcache as C
from oracle import kvfp8 as KV

pytestmark = pytest.mark.gpu
DEV = U.DEV
KS, VS = np.float32(0.0123), np.float32(0.0171)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    U.require_gpu_lib()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def dtype_values(x, dtype):
    """(device tensor of dtype, its values as float32)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dtype)
    return t.to(DEV), t.float().numpy()


class Case:
    """A cache whose unseen bytes are NaN codes, with queries."""

    def __init__(self, dtype, lens, M, H, G, D, page, tree=False, counts=None, spare=3, seed=0, gain=1.5, width=None):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.M = np.asarray(lens), None if counts is None else np.asarray(counts), M
        nb = len(lens)
        need = [-(-(max(n, 0) + M) // page) for n in lens]
        P = sum(need) + spare
        order = rng.permutation(P)
        self.table = np.full((nb, width or max(1, max(need))), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k = np.full((P, H, page, D), 0x7F, dtype=np.uint8)
        self.v = np.full((P, H, page, D), 0xFF, dtype=np.uint8)
        for b, n in enumerate(lens):
            c = M if counts is None else min(M, counts[b])
            for t in range(max(n, 0) + c if n >= 0 else 0):
                p, s = self.table[b, t // page], t % page
                self.k[p, :, s] = KV.encode(rng.standard_normal((H, D)).astype(np.float32), KS)
                self.v[p, :, s] = KV.encode(rng.standard_normal((H, D)).astype(np.float32), VS)
        self.parent = None
        if tree:
            self.parent = np.array([[-1] + [int(rng.integers(max(0, v - 4), v)) for v in range(1, M)]
                                    for _ in range(nb)], dtype=np.int32)
        self.q, self.qf = dtype_values(rng.standard_normal((nb, M, H * G, D)) * gain, dtype)
        self.dtype, self.D = dtype, D

    def gpu(self, **kw):
        args = dict(parent=None if self.parent is None else ints(self.parent),
                    counts=None if self.counts is None else ints(self.counts), want_lse=True)
        pages = [torch.from_numpy(x).to(DEV) for x in (self.k, self.v)]
        q = kw.pop("q", self.q)
        args.update(kw)
        return B.nvfp4_kv_attention(q, U.scalar(KS), U.scalar(VS), *pages, ints(self.table), ints(self.lens), **args)

    def check(self, got, sm_scale=None):
        out, lse = (x.double().cpu().numpy() for x in got)
        ref, ref_lse, size = C.attention(self.qf, self.k, self.v, KS, VS, self.table, self.lens, self.parent,
                                         self.counts, sm_scale)
        u, D = 2.0 ** -24, self.D
        sm = 1 / np.sqrt(D) if sm_scale is None else abs(sm_scale)
        codes = C.F.decode_e4m3(np.where((self.k & 0x7F) == 0x7F, 0, self.k).astype(np.uint8)) * float(KS)
        qn = np.linalg.norm(self.qf.astype(np.float64), axis=-1)
        zmax = sm * qn * np.sqrt((codes ** 2).sum(-1).max())  # bounds sum|q k_hat| sm for every token
        ez = (D + 12) * u * zmax
        N = max(0, int(self.lens.max())) + self.M
        vmax = 448 * float(VS)
        half = torch.finfo(self.dtype).eps / 2
        rp = 2.0 ** -11 if self.dtype == torch.bfloat16 else 2.0 ** -22
        tol = half * np.abs(ref) + (2 * ez + rp + 2 * (N + 8) * u)[..., None] * size + N * 2.0 ** -32 * vmax
        empty = np.isneginf(ref_lse)
        assert np.array_equal(empty, np.isneginf(lse))
        assert not out[empty].any()
        err = np.abs(out - ref)
        assert np.isfinite(out).all() and (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
        tol = 2 * ez + 2 * (N + 8) * u + 4 * u * np.abs(np.where(empty, 0, ref_lse))
        assert (np.abs(lse[~empty] - ref_lse[~empty]) <= tol[~empty]).all()


BF, FP = torch.bfloat16, torch.float32


# ----------------------------------------------------------------------------------------------- append, compact


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B_,M,H,D,page,counts", [(1, 1, 1, 64, 16, None), (3, 5, 4, 128, 32, None),
                                                  (4, 37, 5, 256, 16, [0, 37, 9, 90]), (2, 700, 8, 128, 64, None)])
def test_append_matches_oracle(dtype, B_, M, H, D, page, counts):
    rng = np.random.default_rng(M)
    lens = rng.integers(0, 3 * page, B_)
    lens[-1] = -1 if B_ > 2 else lens[-1]
    W = -(-(3 * page + M) // page)
    P = B_ * W + 2
    table = rng.permutation(P)[: B_ * W].reshape(B_, W).astype(np.int32)
    start = [rng.integers(0, 256, (P, H, page, D), dtype=np.uint8) for _ in range(2)]
    x, xf = dtype_values(rng.standard_normal((2, B_, M, H, D)) * 3, dtype)
    pages = [torch.from_numpy(p).to(DEV) for p in start]
    B.nvfp4_kv_append(x[0], x[1], U.scalar(KS), U.scalar(VS), *pages, ints(table), ints(lens),
                      counts=None if counts is None else ints(counts))
    for got, x1, s, p in zip(pages, xf, (KS, VS), start):
        np.testing.assert_array_equal(got.cpu().numpy(), C.append(x1, s, p, table, lens, counts))


def test_append_takes_columns_of_a_projection_and_layers_of_a_pool():
    """k and v as column ranges of one [rows, (Hq + 2H) D] output; pages [P, L, 2, H, page, D]."""
    rng = np.random.default_rng(5)
    B_, M, Hq, H, D, page, P, L = 2, 3, 6, 2, 128, 16, 9, 3
    y, yf = dtype_values(rng.standard_normal((B_, M, (Hq + 2 * H) * D)), BF)
    k = y[..., Hq * D:(Hq + H) * D].view(B_, M, H, D)
    v = y[..., (Hq + H) * D:].view(B_, M, H, D)
    pool = torch.from_numpy(rng.integers(0, 256, (P, L, 2, H, page, D), dtype=np.uint8)).to(DEV)
    before = pool.cpu().numpy()
    table, lens = np.array([[4, 1], [8, 0]], dtype=np.int32), np.array([15, 3])
    B.nvfp4_kv_append(k, v, U.scalar(KS), U.scalar(VS), pool[:, 1, 0], pool[:, 1, 1], ints(table), ints(lens))
    got = pool.cpu().numpy()
    xf = yf.reshape(B_, M, Hq + 2 * H, D)
    np.testing.assert_array_equal(got[:, 1, 0], C.append(xf[:, :, Hq:Hq + H], KS, before[:, 1, 0], table, lens))
    np.testing.assert_array_equal(got[:, 1, 1], C.append(xf[:, :, Hq + H:], VS, before[:, 1, 1], table, lens))
    np.testing.assert_array_equal(got[:, [0, 2]], before[:, [0, 2]])


def test_append_leaves_out_tokens_without_a_page():
    rng = np.random.default_rng(6)
    table = np.array([[0, -1, 7], [2, 3, 1 << 20]], dtype=np.int32)  # P = 4
    lens = np.array([10, 44])                                        # the second runs past its table
    start = rng.integers(0, 256, (4, 2, 16, 64), dtype=np.uint8)
    x, xf = dtype_values(rng.standard_normal((2, 30, 2, 64)), FP)
    pages = [torch.from_numpy(start).to(DEV) for _ in range(2)]
    B.nvfp4_kv_append(x, x, U.scalar(KS), U.scalar(VS), *pages, ints(table), ints(lens))
    np.testing.assert_array_equal(pages[0].cpu().numpy(), C.append(xf, KS, start, table, lens))
    np.testing.assert_array_equal(pages[1].cpu().numpy(), C.append(xf, VS, start, table, lens))


@pytest.mark.parametrize("M,H,D,page,L", [(1, 2, 64, 16, 1), (16, 8, 128, 64, 3), (64, 3, 256, 32, 2),
                                          (33, 1, 128, 16, 5)])
def test_compact_matches_oracle(M, H, D, page, L):
    rng = np.random.default_rng(M + D)
    lens = np.array([0, 3 * page - 1, 17, -1, 2 * page])
    B_, W = len(lens), -(-(3 * page + M) // page)
    P = B_ * W
    table = rng.permutation(P).reshape(B_, W).astype(np.int32)
    result = np.full((B_, 3 + M), -1, dtype=np.int32)
    for b in range(B_):
        n = int(rng.integers(0, M))
        result[b, 1] = n
        result[b, 3:3 + n] = 1 + np.sort(rng.permutation(M - 1)[:n])
    start = rng.integers(0, 256, (2, L, P, H, page, D), dtype=np.uint8)
    pages = torch.from_numpy(start).to(DEV)
    old = ints(lens)
    new = B.nvfp4_kv_compact(pages[0], pages[1], ints(table), old, ints(result))
    want = [C.compact(p, table, lens, result) for p in start]
    np.testing.assert_array_equal(new.cpu().numpy(), want[0][1])
    np.testing.assert_array_equal(old.cpu().numpy(), lens)
    np.testing.assert_array_equal(pages.cpu().numpy(), np.stack([w[0] for w in want]))


def test_compact_passes_over_entries_that_name_no_node_and_pages_that_do_not_exist():
    rng = np.random.default_rng(8)
    table = np.array([[0, 9], [1, 2]], dtype=np.int32)  # P = 3
    lens = np.array([10, 12])
    result = np.array([[0, 5, 0, 3, 8, 9, 10, 11] + [-1] * 7, [0, 4, 0, 2, 50, -7, 6] + [-1] * 8], dtype=np.int32)
    start = rng.integers(0, 256, (2, 3, 1, 16, 64), dtype=np.uint8)
    pages = torch.from_numpy(start).to(DEV)
    B.nvfp4_kv_compact(pages, pages.clone(), ints(table), ints(lens), ints(result))
    np.testing.assert_array_equal(pages.cpu().numpy(), C.compact(start, table, lens, result)[0])


# ----------------------------------------------------------------------------------------------- page pool


def pool_tensors(pool):
    P = len(pool.refs)
    free = np.full(P + 1, -1, dtype=np.int32)
    free[0] = len(pool.free)
    free[1:1 + len(pool.free)] = pool.free
    return [ints(pool.table), ints(pool.held), ints(pool.refs), ints(free)]


def check_pool(t, pool):
    table, held, refs, free = (x.cpu().numpy() for x in t)
    np.testing.assert_array_equal(table, pool.table)
    np.testing.assert_array_equal(held, pool.held)
    np.testing.assert_array_equal(refs, pool.refs)
    assert free[0] == len(pool.free) and free[1:1 + free[0]].tolist() == pool.free


@pytest.mark.parametrize("seed,S,W,P,page,n", [(0, 7, 6, 23, 16, 4), (1, 1, 1, 1, 16, 2), (2, 40, 30, 500, 32, 17),
                                               (3, 1500, 9, 9000, 16, 1024), (4, 12, 400, 3000, 64, 12)])
def test_pool_steps_match_oracle(seed, S, W, P, page, n):
    rng = np.random.default_rng(seed)
    pool = C.Pool(S, W, P)
    t = list(B.kv_pool(S, W, P, DEV))
    check_pool(t, pool)
    start = rng.integers(0, 256, (2, 2, P, 1, page, 64), dtype=np.uint8) if P < 1000 else None
    pages = torch.zeros((2, 1, P, 1, page, 64), dtype=torch.uint8, device=DEV) if start is None else \
        torch.from_numpy(start).to(DEV)
    for step in range(16):
        m = int(rng.integers(0, n + 1)) if step else n
        a, b = rng.integers(-1, S + 1, m), rng.integers(-1, S + 1, m)
        tokens = rng.integers(-3, page * W + 2, m) // (1 if step % 3 else 4)
        if step % 2 == 0:
            want = pool.resize(page, a, tokens)
            got = B.nvfp4_kv_resize(*t, page, ints(a), ints(tokens))
        else:
            a = rng.integers(0, S, m)
            free = [s for s in range(S) if s not in set(a.tolist())] or [0]
            b = np.where(rng.random(m) < 0.8, rng.choice(free, m), b)
            tokens = np.minimum(tokens, np.where(rng.random(m) < 0.8, pool.held[a] * page, page * W))
            want, moves = pool.fork(page, a, b, tokens)
            got = B.nvfp4_kv_fork(*t, pages[0], pages[1], ints(a), ints(b), ints(tokens))
            if start is not None:
                start = np.stack([C.copy_slots(x, moves) for x in start])
        assert int(got) == want
        check_pool(t, pool)
    if start is not None:
        np.testing.assert_array_equal(pages.cpu().numpy(), start)


def test_a_short_free_list_changes_nothing():
    pool = C.Pool(4, 8, 10)
    pool.resize(16, [0], [100])
    t = pool_tensors(pool)
    pages = torch.zeros((1, 10, 1, 16, 64), dtype=torch.uint8, device=DEV)
    assert int(B.nvfp4_kv_resize(*t, 16, ints([1, 0]), ints([70, 0]))) == 2
    check_pool(t, pool)
    assert int(B.nvfp4_kv_fork(*t, pages, pages.clone(), ints([0] * 3), ints([1, 2, 3]), ints([3, 17, 99]))) == 0
    pool.fork(16, [0] * 3, [1, 2, 3], [3, 17, 99])
    check_pool(t, pool)
    assert int(B.nvfp4_kv_fork(*t, pages, pages.clone(), ints([0]), ints([1]), ints([4]))) == 1
    check_pool(t, pool)


# ----------------------------------------------------------------------------------------------- attention


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,M,H,G,D,page,tree,counts", [
    ([0], 1, 1, 1, 64, 16, False, None),
    ([1], 1, 2, 3, 128, 16, False, None),
    ([127], 1, 8, 5, 128, 64, False, None),
    ([128, 129, 0, 31], 1, 2, 8, 64, 16, False, None),
    ([700, -1, 15], 1, 3, 16, 128, 128, False, None),
    ([255], 16, 2, 5, 128, 64, True, None),
    ([100, 300, 0, 33], 16, 2, 4, 64, 32, True, [16, 0, 7, 40]),
    ([511], 64, 1, 8, 128, 256, True, None),
    ([77, -5], 13, 2, 3, 256, 16, True, [13, 13]),
    ([0, 40], 64, 2, 1, 256, 32, True, None),
    ([200], 7, 1, 12, 256, 1024, False, None),
    ([0], 150, 2, 2, 64, 16, False, None),
    ([333, 5], 90, 1, 5, 128, 32, False, [90, 41]),
    ([1000], 1, 1, 1, 256, 16, False, None),
    ([40] * 9, 2, 4, 2, 128, 16, True, None),
])
def test_attention_matches_oracle(dtype, lens, M, H, G, D, page, tree, counts):
    c = Case(dtype, lens, M, H, G, D, page, tree, counts, seed=sum(map(abs, lens)) + M)
    c.check(c.gpu())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_over_a_long_context(dtype):
    """The longest agent context of the pages, a 16-node tree at its end."""
    c = Case(dtype, [23536], 16, 2, 3, 128, 64, True, seed=3)
    c.check(c.gpu())


def test_attention_of_a_suffix_over_a_long_prefix():
    c = Case(BF, [2900], 130, 1, 5, 128, 64, seed=4)
    c.check(c.gpu())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_of_large_scores(dtype):
    """Scores of some thousands: the exponent's offset rounds, and every partial sum by its own."""
    c = Case(dtype, [1500, 700], 5, 2, 3, 64, 32, True, seed=19, gain=600.0)
    c.check(c.gpu())


@pytest.mark.parametrize("sm", [0.0, -0.3, 2.0])
def test_attention_scales(sm):
    c = Case(FP, [150, 20], 4, 2, 2, 64, 16, True, seed=9, gain=1.0)
    c.check(c.gpu(sm_scale=sm), sm)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_to_one_key_far_above_the_rest_at_the_end(dtype):
    """The running maximum rises late and by a lot: one of the last keys equals the query."""
    c = Case(dtype, [900], 3, 1, 2, 128, 16, seed=10, gain=0.02)
    p, s = c.table[0, 898 // 16], 898 % 16
    c.k[p, 0, s] = KV.encode(np.where(np.arange(128) % 2, 5.0, -5.0).astype(np.float32), KS)
    big, c.qf = dtype_values(np.broadcast_to(np.where(np.arange(128) % 2, 6.0, -6.0), c.qf.shape), dtype)
    c.q = big
    c.check(c.gpu())


def test_attention_of_strided_queries_and_layered_pages():
    c = Case(BF, [70, 300], 5, 2, 5, 128, 32, True, seed=11)
    B_, M, Hq, D = c.q.shape
    wide = torch.full((B_, M, (Hq + 4) * D), float("nan"), dtype=BF, device=DEV)
    wide[..., 2 * D:(Hq + 2) * D] = c.q.view(B_, M, Hq * D)
    q = wide[..., 2 * D:(Hq + 2) * D].view(B_, M, Hq, D)
    want = c.gpu()
    P, H, page, _ = c.k.shape
    pool = torch.full((P, 3, 2, H, page, D), 0x7F, dtype=torch.uint8, device=DEV)
    pool[:, 1, 0], pool[:, 1, 1] = torch.from_numpy(c.k).to(DEV), torch.from_numpy(c.v).to(DEV)
    got = B.nvfp4_kv_attention(q, U.scalar(KS), U.scalar(VS), pool[:, 1, 0], pool[:, 1, 1], ints(c.table),
                               ints(c.lens), parent=ints(c.parent), want_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(got)


def test_attention_passes_over_pages_that_do_not_exist():
    c = Case(BF, [400, 90], 6, 2, 4, 128, 16, True, seed=12)
    c.table[0, [3, 9, 10]] = [-1, c.k.shape[0], 1 << 30]
    c.table[1, :] = -1
    c.check(c.gpu())
    c = Case(FP, [50], 20, 1, 1, 64, 16, seed=13)
    c.table = c.table[:, :2].copy()  # the length runs past the table
    c.check(c.gpu())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_with_and_without_workspace(dtype):
    """Unsplit, split in a workspace full of NaN, in one too small: the same contract; each form
    gives the same bits every time."""
    c = Case(dtype, [3000, 10], 16, 2, 5, 128, 64, True, seed=14)
    need = B.load().nvfp4_kv_attention_workspace_bytes(2, 16, 10, 2, 128, 64, c.table.shape[1], B._dt(dtype))
    seen = []
    for size in (0, 16, need, need + 4096):
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        got = c.gpu(workspace=ws)
        c.check(got)
        again = c.gpu(workspace=ws.fill_(0x7F))
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
        seen.append(got)
    assert torch.equal(seen[2][0], seen[3][0])


def test_attention_writes_into_out_and_runs_on_a_side_stream():
    c = Case(BF, [500], 16, 2, 5, 128, 64, True, seed=15)
    want = c.gpu()[0]
    out = torch.full_like(c.q, float("nan"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.gpu(out=out, want_lse=False)
    torch.cuda.current_stream().wait_stream(s)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)


def test_pages_past_four_gigabytes():
    """Page offsets that pass 32 bits: the sequence's pages stand at the end of a 6 GB cache."""
    c = Case(BF, [100], 5, 1, 4, 128, 64, True, seed=16)
    P, H, page, D = c.k.shape
    far = 6_000_000_000 // (H * page * D)
    pages = [torch.zeros((far + P, H, page, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    for x, y in zip(pages, (c.k, c.v)):
        x[far:] = torch.from_numpy(y).to(DEV)
    table = np.where(c.table < 0, c.table, c.table + far)
    call = lambda: B.nvfp4_kv_attention(c.q, U.scalar(KS), U.scalar(VS), *pages, ints(table), ints(c.lens),  # noqa: E731
                                        parent=ints(c.parent), want_lse=True)
    c.check(call())
    x, xf = dtype_values(np.random.default_rng(1).standard_normal((1, 5, H, D)), BF)
    B.nvfp4_kv_append(x, x, U.scalar(KS), U.scalar(VS), *pages, ints(table), ints(c.lens))
    c.k, c.v = C.append(xf, KS, c.k, c.table, c.lens), C.append(xf, VS, c.v, c.table, c.lens)
    c.check(call())
    np.testing.assert_array_equal(pages[1][far:].cpu().numpy(), c.v)
    assert not pages[0][:far].any()
    result = np.array([[4, 2, 0, 2, 4, -1, -1, -1]])
    new = B.nvfp4_kv_compact(pages[0][None], pages[1][None], ints(table), ints(c.lens), ints(result))
    assert int(new) == 103
    np.testing.assert_array_equal(pages[0][far:].cpu().numpy(),
                                  C.compact(c.k[None], c.table, c.lens, result)[0][0])


# ----------------------------------------------------------------------------------------------- together


def step_tree(M):
    parent, chain = [-1], [0]
    while len(parent) < M:
        parent += [chain[-1], chain[-1]]
        chain.append(len(parent) - 2)
    return parent[:M]


def test_decode_steps_with_forks_match_oracle():
    """Two conversations over two layers: prompts, tree steps whose path is accepted, a fork, frees; pages,
    tables and outputs after every step."""
    rng = np.random.default_rng(20)
    S, W, P, L, H, G, D, page, M = 3, 12, 30, 2, 2, 4, 64, 16, 16
    pool, t = C.Pool(S, W, P), list(B.kv_pool(S, W, P, DEV))
    host = np.zeros((2, L, P, H, page, D), dtype=np.uint8)
    pages = torch.from_numpy(host).to(DEV)
    lens = np.array([0, 0, -1])
    parent = np.array([step_tree(M)] * S, dtype=np.int32)
    ids = ints([0, 1, 2])

    def layer_pass(rows, tree, counts):
        for l in range(L):
            x, xf = dtype_values(rng.standard_normal((2, S, rows, H, D)), BF)
            q, qf = dtype_values(rng.standard_normal((S, rows, H * G, D)), BF)
            B.nvfp4_kv_append(x[0], x[1], U.scalar(KS), U.scalar(VS), pages[0, l], pages[1, l], t[0], ints(lens),
                              counts=None if counts is None else ints(counts))
            got = B.nvfp4_kv_attention(q, U.scalar(KS), U.scalar(VS), pages[0, l], pages[1, l], t[0], ints(lens),
                                       parent=ints(parent) if tree else None, want_lse=True,
                                       counts=None if counts is None else ints(counts))
            for kv, s in ((0, KS), (1, VS)):
                host[kv, l] = C.append(xf[kv], s, host[kv, l], pool.table, lens, counts)
            c = Case.__new__(Case)
            c.qf, c.k, c.v, c.table, c.lens, c.M, c.D = qf, host[0, l], host[1, l], pool.table, lens, rows, D
            c.parent, c.counts, c.dtype = parent if tree else None, None if counts is None else np.asarray(counts), BF
            c.check(got)

    def resize(tokens):
        assert int(B.nvfp4_kv_resize(*t, page, ids, ints(tokens))) == pool.resize(page, [0, 1, 2], tokens) == 0
        check_pool(t, pool)

    counts = [50, 23, 0]  # the prompts
    resize(counts)
    layer_pass(50, False, counts)
    lens = np.array([50, 23, -1])
    for step in range(4):
        resize(np.maximum(lens, 0) + np.where(lens < 0, 0, M))
        layer_pass(M, True, None)
        drafts = rng.integers(0, 2, (S, M))
        greedy = rng.integers(0, 2, (S, M))
        result = torch.stack([B.nvfp4_tree_accept(ints(parent[b]), ints(drafts[b]), ints(greedy[b]))
                              for b in range(S)])
        new = B.nvfp4_kv_compact(pages[0], pages[1], t[0], ints(lens), result)
        r = result.cpu().numpy()
        both = [C.compact(host[kv], pool.table, lens, r) for kv in (0, 1)]
        host[0], host[1] = both[0][0], both[1][0]
        np.testing.assert_array_equal(new.cpu().numpy(), both[0][1])
        np.testing.assert_array_equal(pages.cpu().numpy(), host)
        lens = both[0][1]
        if step == 1:  # a third conversation starts from most of the first
            keep = int(lens[0]) - 3
            short = B.nvfp4_kv_fork(*t, pages[0], pages[1], ints([0]), ints([2]), ints([keep]))
            want, moves = pool.fork(page, [0], [2], [keep])
            host = np.stack([C.copy_slots(x, moves) for x in host])
            assert int(short) == want == 0
            check_pool(t, pool)
            lens[2] = keep
    resize([0, 0, 0])
    assert len(pool.free) == P


def test_a_captured_step_replays_with_new_lengths():
    """append, attention, acceptance and compaction in one graph; lengths advance on the device between
    replays, and every replay equals the eager step."""
    rng = np.random.default_rng(21)
    M, H, G, D, page, W, P, L = 16, 2, 5, 128, 64, 12, 40, 2
    parent = step_tree(M)
    x, _ = dtype_values(rng.standard_normal((2, 2, M, H, D)), BF)
    q, _ = dtype_values(rng.standard_normal((2, M, H * G, D)), BF)
    table = ints(rng.permutation(P)[: 2 * W].reshape(2, W))
    start = torch.from_numpy(KV.encode(rng.standard_normal((2, L, P, H, page, D)).astype(np.float32), KS)).to(DEV)
    par, par2 = ints(parent), ints([parent, parent])
    drafts, greedy = ints(rng.integers(0, 2, M)), ints(rng.integers(0, 2, M))
    ks, vs = U.scalar(KS), U.scalar(VS)
    state = dict(pages=start.clone(), lens=ints([70, 133]), out=torch.empty_like(q), new=ints([0, 0]))

    def step():
        for l in range(L):
            B.nvfp4_kv_append(x[0], x[1], ks, vs, state["pages"][0, l], state["pages"][1, l], table, state["lens"])
            B.nvfp4_kv_attention(q, ks, vs, state["pages"][0, l], state["pages"][1, l], table, state["lens"],
                                 parent=par2, out=state["out"])
        r = B.nvfp4_tree_accept(par, drafts, greedy)
        B.nvfp4_kv_compact(state["pages"][0], state["pages"][1], table, state["lens"], torch.stack([r, r]),
                           new_lens=state["new"])
        state["lens"].copy_(state["new"])

    def reset():
        state["pages"].copy_(start)
        state["lens"].copy_(ints([70, 133]))

    reset()
    want = []
    for _ in range(4):
        step()
        want.append([state[n].clone() for n in ("pages", "lens", "out")])
    torch.cuda.synchronize()
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    reset()
    for r, w in enumerate(want):
        g.replay()
        torch.cuda.synchronize()
        for name, y in zip(("pages", "lens", "out"), w):
            assert torch.equal(state[name].view(torch.uint8), y.view(torch.uint8)), (r, name)
        torch.zeros(1 << 20, device=DEV).add_(1)  # eager work between replays


def test_a_captured_resize_and_fork_replay():
    pool = C.Pool(4, 8, 20)
    pool.resize(16, [0, 1], [100, 30])
    t = pool_tensors(pool)
    pages = torch.randint(0, 256, (1, 20, 1, 16, 64), dtype=torch.uint8, device=DEV)
    src, dst, tok, ids, up, down = ints([0, 1]), ints([2, 3]), ints([37, 20]), ints([1, 0]), ints([60, 101]), ints([30, 100])
    shortage = ints([7])

    def step():
        B.nvfp4_kv_fork(*t, pages, pages, src, dst, tok, shortage=shortage)
        B.nvfp4_kv_resize(*t, 16, ids, up, shortage=shortage)
        B.nvfp4_kv_resize(*t, 16, ids, down, shortage=shortage)

    g = torch.cuda.CUDAGraph()
    saved = [x.clone() for x in t]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        step()
    for x, y in zip(t, saved):
        x.copy_(y)
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        pool.fork(16, [0, 1], [2, 3], [37, 20])
        pool.resize(16, [1, 0], [60, 101])
        pool.resize(16, [1, 0], [30, 100])
        check_pool(t, pool)
        assert int(shortage) == 0


# ----------------------------------------------------------------------------------------------- refusals


def test_binding_refuses_what_does_not_fit():
    c = Case(BF, [20], 3, 2, 2, 64, 16, True)
    pages = [torch.from_numpy(x).to(DEV) for x in (c.k, c.v)]
    ok = dict(q=c.q, k_scale=U.scalar(KS), v_scale=U.scalar(VS), k_pages=pages[0], v_pages=pages[1],
              table=ints(c.table), lens=ints(c.lens), parent=ints(c.parent))
    B.nvfp4_kv_attention(**ok)
    for bad in (dict(q=c.q.half()), dict(q=c.q[..., :32]), dict(q=c.q.transpose(1, 2)), dict(q=c.q[:, :, :3]),
                dict(table=ints(c.table).long()), dict(table=ints(c.table)[0]), dict(lens=ints([1, 2])),
                dict(parent=ints(c.parent)[:, :2]), dict(counts=ints([1, 1])), dict(k_scale=torch.ones(1)),
                dict(k_scale=torch.ones(2, device=DEV)), dict(v_pages=pages[1][:2]), dict(v_pages=pages[1].float()),
                dict(out=torch.empty_like(c.q, dtype=FP)), dict(out=c.q[:, :2]), dict(lens=ints(c.lens).cpu()),
                dict(k_pages=pages[0].transpose(1, 2), v_pages=pages[1].transpose(1, 2)),
                dict(workspace=torch.empty(64, device=DEV)), dict(k_pages=pages[0][:, :, :, :32],
                                                                  v_pages=pages[1][:, :, :, :32])):
        with pytest.raises((ValueError, TypeError)):
            B.nvfp4_kv_attention(**{**ok, **bad})
    with pytest.raises(B.NVFP4Error):
        B.nvfp4_kv_attention(**{**ok, "sm_scale": float("nan")})
    x = torch.zeros((1, 3, 2, 64), device=DEV)
    with pytest.raises(ValueError):
        B.nvfp4_kv_append(x, x[:, :2], ok["k_scale"], ok["v_scale"], *pages, ok["table"], ok["lens"])
    with pytest.raises(ValueError):
        B.nvfp4_kv_append(x, x.bfloat16(), ok["k_scale"], ok["v_scale"], *pages, ok["table"], ok["lens"])
    lens = ints([1])
    with pytest.raises(B.NVFP4Error):
        B.nvfp4_kv_compact(pages[0][None], pages[1][None], ok["table"], lens, ints([[0, 0, 0, -1]]), new_lens=lens)
    with pytest.raises(ValueError):
        B.nvfp4_kv_compact(pages[0], pages[1], ok["table"], lens, ints([[0, 0, 0, -1]]))


def test_empty_calls():
    pages = torch.zeros((2, 1, 16, 64), dtype=torch.uint8, device=DEV)
    s, none = U.scalar(KS), ints(np.zeros((0,)))
    q = torch.empty((0, 4, 2, 64), device=DEV)
    out, lse = B.nvfp4_kv_attention(q, s, s, pages, pages, ints(np.zeros((0, 3))), none, want_lse=True)
    assert out.shape == q.shape and lse.shape == (0, 4, 2)
    q = torch.empty((2, 0, 2, 64), device=DEV)
    assert B.nvfp4_kv_attention(q, s, s, pages, pages, ints(np.zeros((2, 3))), ints([1, 2])).shape == q.shape
    B.nvfp4_kv_append(q[:, :, :1], q[:, :, :1], s, s, pages, pages, ints(np.zeros((2, 3))), ints([1, 2]))
    t = B.kv_pool(2, 2, 2, DEV)
    assert int(B.nvfp4_kv_resize(*t, 16, none, none)) == 0
    assert int(B.nvfp4_kv_fork(*t, pages[None], pages[None].clone(), none, none, none)) == 0


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (256, BF), (128, FP)])
def test_nan_codes_reach_only_the_rows_that_see_them(D, dtype, tree):
    """A NaN among a node's values spoils one dimension, in the rows of its descendants; one among its
    keys, and one in a query, spoil whole rows.  The other rows are as they were without them."""
    c = Case(dtype, [70, 300], 12, 2, 3, D, 32, tree=tree, seed=D + tree)
    clean_out, clean_lse = (x.cpu().numpy() for x in (lambda r: (r[0].float(), r[1]))(c.gpu()))
    line = np.tri(12, dtype=bool) if not tree else C.ancestors(c.parent[1])

    def at(t):
        return c.table[1, t // 32], t % 32

    node_v, node_k = 5, 9
    p, s = at(300 + node_v)
    c.v[p, 1, s, 7] = 0xFF
    c.v[p, 1, s, D - 1] = 0x7F
    p, s = at(300 + node_k)
    c.k[p, 0, s, 3] = 0x7F
    q = c.q.clone()
    q[0, 4, 2, 1] = float("nan")
    out, lse = c.gpu(q=q)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    want_out, want_lse = clean_out.copy(), clean_lse.copy()
    for v in range(12):
        if line[v, node_v]:
            want_out[1, v, 3:, [7, D - 1]] = np.nan
        if line[v, node_k]:
            want_out[1, v, :3] = np.nan
            want_lse[1, v, :3] = np.nan
    want_out[0, 4, 2] = np.nan
    want_lse[0, 4, 2] = np.nan
    np.testing.assert_array_equal(out, want_out)
    np.testing.assert_array_equal(lse, want_lse)


def many_rows(D, dtype, most):
    return [pytest.param(D, dtype, n, id=f"{D}-{'bf16' if dtype == BF else 'f32'}-{n}") for n in most]


@pytest.mark.parametrize("D,dtype,tiles", many_rows(64, BF, [2, 5, 6, 7, 11, 13, 24, 25]) +
                         many_rows(128, BF, [2, 3, 4, 5, 8, 9, 16, 17]) + many_rows(256, BF, [1, 2, 3, 4, 5, 8, 9]) +
                         many_rows(64, FP, [1, 2, 3, 5, 8, 9]) + many_rows(128, FP, [2, 4, 7, 9]) +
                         many_rows(256, FP, [1, 2, 3, 4, 5]))
def test_attention_of_every_number_of_row_tiles(D, dtype, tiles):
    """Rows (3 query heads a KV head) that fill `tiles` tiles of 16, over sequences that are cut."""
    M = (16 * tiles - 1) // 3
    c = Case(dtype, [1150 - M, 40], M, 1, 3, D, 64, seed=D + tiles, width=20)
    c.check(c.gpu())


class Shared(Case):
    """Sequences whose tables name random pages of one small pool."""

    def __init__(self, dtype, lens, M, H, G, D, page, width, pages, seed, counts=None):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.M, self.parent, self.dtype, self.D = lens, counts, M, None, dtype, D
        self.table = rng.integers(0, pages, (len(lens), width)).astype(np.int32)
        self.k, self.v = (KV.encode(rng.standard_normal((pages, H, page, D)).astype(np.float32), s) for s in (KS, VS))
        self.q, self.qf = dtype_values(rng.standard_normal((len(lens), M, H * G, D)), dtype)


@pytest.mark.parametrize("dtype,B_,M,H", [(BF, 600, 1, 1), (FP, 350, 1, 2), (BF, 1100, 1, 1)])
def test_attention_of_more_sequences_than_workgroups(dtype, B_, M, H):
    """Ranges that hold several sequences, cut at places of their set-up as well, unused rows among them."""
    lens = np.random.default_rng(B_).integers(-60, 1290 - M, B_)
    c = Shared(dtype, lens, M, H, 2, 64, 64, 21, 50, B_)
    c.check(c.gpu())


@pytest.mark.parametrize("tree", [True, False])
def test_attention_of_nodes_behind_the_table(tree):
    """Nodes whose tokens have no place see the tokens that have one."""
    c = Case(BF, [60, 3000], 9, 2, 2, 64, 16, tree, seed=23)
    c.table = np.ascontiguousarray(c.table[:, :4])
    c.lens = np.array([60, 64])
    c.check(c.gpu())


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, give what they give alone."""
    cases = [Case(BF, [5000], 16, 2, 5, 128, 64, True, seed=24), Case(BF, [900, 2500, 40], 5, 2, 4, 64, 32, seed=25)]
    alone = [c.gpu() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cases[i].gpu())
    torch.cuda.synchronize()
    for i, want in enumerate(alone):
        for out, lse in got[i]:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_forks_of_one_sequence_and_pages_given_up_twice():
    """One source named many times; then its copies, which share every whole page, are freed in one call."""
    pool = C.Pool(12, 8, 60)
    pool.resize(16, [0, 1], [100, 40])
    t = pool_tensors(pool)
    start = np.random.default_rng(26).integers(0, 256, (2, 3, 60, 2, 16, 64), dtype=np.uint8)
    pages = torch.from_numpy(start).to(DEV)
    src, dst, tokens = [0] * 9, [2, 3, 4, 5, 6, 7, 8, 9, 1], [100, 96, 95, 1, 16, 0, 81, 100, 33]
    short, moves = pool.fork(16, src, dst, tokens)
    assert int(B.nvfp4_kv_fork(*t, pages[0], pages[1], ints(src), ints(dst), ints(tokens))) == short == 0
    check_pool(t, pool)
    np.testing.assert_array_equal(pages.cpu().numpy(), np.stack([C.copy_slots(x, moves) for x in start]))
    seqs = [9, 3, 0, 0, 8, 2, 1, 6]
    assert pool.resize(16, seqs, [0] * 8) == 0
    assert int(B.nvfp4_kv_resize(*t, 16, ints(seqs), ints([0] * 8))) == 0
    check_pool(t, pool)


@pytest.mark.parametrize("D,dtype,tiles", many_rows(64, BF, [13, 24]) + many_rows(128, BF, [9, 13, 16]) +
                         many_rows(256, BF, [5, 8]) + many_rows(64, FP, [5, 8]) + many_rows(256, FP, [3, 4]))
def test_attention_of_many_rows_under_a_wide_table(D, dtype, tiles):
    """A table that covers a cache of more than 256 MB, of which the sequences use little."""
    M = (16 * tiles - 1) // 3
    c = Case(dtype, [1150 - M, 40], M, 1, 3, D, 64, seed=D + tiles, width=(1 << 30) // (2 * 2 * D * 64))
    c.check(c.gpu())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_nans_reach_their_rows_through_split_sequences(dtype):
    """NaN codes in a long prefix (every row sees them) and in one node, and a NaN with payload in a query."""
    c = Case(dtype, [3000, 2000], 5, 2, 2, 128, 64, tree=False, seed=41)
    clean_out, clean_lse = [x.float().cpu().numpy() for x in c.gpu()]
    p, s = c.table[0, 1700 // 64], 1700 % 64
    c.v[p, 0, s, 100] = 0x7F
    p, s = c.table[1, 2003 // 64], 2003 % 64
    c.k[p, 1, s, 127] = 0xFF
    q = c.q.clone()
    raw = q.view(torch.int16 if dtype == BF else torch.int32)
    raw[0, 2, 3, 5] = 0x7FFF if dtype == BF else 0x7FFFFFFF
    out, lse = [x.float().cpu().numpy() for x in c.gpu(q=q)]
    clean_out[0, :, :2, 100] = np.nan
    clean_out[1, 3:, 2:], clean_lse[1, 3:, 2:] = np.nan, np.nan
    clean_out[0, 2, 3], clean_lse[0, 2, 3] = np.nan, np.nan
    np.testing.assert_array_equal(out, clean_out)
    np.testing.assert_array_equal(lse, clean_lse)


def test_attention_of_scores_far_below_zero():
    """All scores near -2.6e32: the offset follows them, the weights are those of their differences."""
    c = Case(BF, [40], 2, 1, 2, 64, 16, seed=43)
    c.k[:] = np.where((c.k & 0x7F) == 0x7F, c.k, 0x40)             # every seen key the same: equal scores
    c.q, c.qf = dtype_values(np.full(c.qf.shape, -2.0 ** 110), BF)  # z = -64 * 2 * 0.0123 * 2^110 / 8
    out, lse = c.gpu()
    ref, ref_lse, size = C.attention(c.qf, c.k, c.v, KS, VS, c.table, c.lens)
    # equal scores give equal weights exactly; what is left are the f16 weights, the sums and the result's rounding
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 100 * 2.0 ** -24) * size
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() / ref_lse - 1) <= 200 * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_appended_nans_reach_the_rows_that_see_them(dtype):
    """NaN, infinities and scales that make NaN: append stores the codec's bytes, and attention carries a
    NaN key or value to the nodes that see it and to no other."""
    rng = np.random.default_rng(51)
    M, H, G, D, page = 6, 2, 2, 64, 16
    c = Case(dtype, [20], M, H, G, D, page, seed=51)
    x, xf = dtype_values(rng.standard_normal((2, 1, M, H, D)), dtype)
    x[0, 0, 4, 1, 9], xf[0, 0, 4, 1, 9] = float("nan"), np.nan    # a key of node 4
    x[1, 0, 2, 0, 3], xf[1, 0, 2, 0, 3] = float("nan"), np.nan    # a value of node 2
    x[1, 0, 1, 1, 5], xf[1, 0, 1, 1, 5] = float("inf"), np.inf
    x[0, 0, 0, 0, 7], xf[0, 0, 0, 0, 7] = float("-inf"), -np.inf
    table, lens = ints(c.table), ints(c.lens)
    for ks, vs in ((KS, VS), (np.float32(0), VS), (KS, np.float32(1e-39))):
        pages = [torch.from_numpy(p).to(DEV) for p in (c.k, c.v)]
        B.nvfp4_kv_append(x[0], x[1], U.scalar(ks), U.scalar(vs), *pages, table, lens)
        for got, x1, s, p in zip(pages, xf, (ks, vs), (c.k, c.v)):
            with np.errstate(invalid="ignore"):
                want = C.append(x1, s, p, c.table, c.lens)
            got = got.cpu().numpy()
            nan = (want & 0x7F) == 0x7F
            np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan)
            np.testing.assert_array_equal(got[~nan], want[~nan])
    pages = [torch.from_numpy(p).to(DEV) for p in (c.k, c.v)]
    B.nvfp4_kv_append(x[0], x[1], U.scalar(KS), U.scalar(VS), *pages, table, lens)
    out = B.nvfp4_kv_attention(c.q, U.scalar(KS), U.scalar(VS), *pages, table, lens).float().cpu().numpy()
    want = np.zeros((1, M, H * G, D), dtype=bool)
    want[0, 4:, G:] = True        # head 1, from node 4 on
    want[0, 2:, :G, 3] = True     # head 0, one dimension, from node 2 on
    np.testing.assert_array_equal(np.isnan(out), want)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("split", [True, False])
def test_scales_that_are_no_number_reach_every_row_that_sees_something(dtype, split, bad):
    """A NaN or infinite k_scale: NaN out and lse.  A NaN v_scale: NaN out, lse as it was.  Rows that see
    nothing (an unused sequence, nodes behind counts, a table without pages) stay zero and -infinity."""
    c = Case(dtype, [2500, 40, -1, 30], 5, 2, 3, 64, 32, tree=True, counts=[5, 3, 5, 5], seed=53)
    c.table[3] = -1
    pages = [torch.from_numpy(x).to(DEV) for x in (c.k, c.v)]

    def call(ks, vs):
        ws = None if split else torch.empty(0, dtype=torch.uint8, device=DEV)
        out, lse = B.nvfp4_kv_attention(c.q, U.scalar(np.float32(ks)), U.scalar(np.float32(vs)), *pages, ints(c.table),
                                        ints(c.lens), parent=ints(c.parent), counts=ints(c.counts), want_lse=True,
                                        workspace=ws)
        return out.float().cpu().numpy(), lse.cpu().numpy()

    clean = call(KS, VS)
    sees = np.isfinite(clean[1])
    assert sees[0].all() and sees[1, :3].all() and not sees[1, 3:].any() and not sees[2:].any()
    out, lse = call(bad, VS)
    assert np.isnan(out[sees]).all() and np.isnan(lse[sees]).all()
    assert not out[~sees].any() and np.isneginf(lse[~sees]).all()
    if np.isnan(bad):
        out, lse = call(KS, bad)
        assert np.isnan(out[sees]).all() and not out[~sees].any()
        np.testing.assert_array_equal(lse, clean[1])


def far_check(c, got, rows, sm):
    """Rows [B, M] whose best key leads by more than the scores' rounding can hide: its value is the
    result.  The bound: a score is off by ez (module docstring) and, on the way to the exponent, by 8 u of
    itself; beyond that and 200 powers of two nothing else weighs in fp32.  The one weight is rounded (2^-11,
    2^-22), then a few products."""
    out, lse = (x.double().cpu().numpy() for x in got)
    ref, ref_lse, _ = C.attention(c.qf, c.k, c.v, KS, VS, c.table, c.lens, c.parent, c.counts, sm)
    u, B_, M = 2.0 ** -24, len(c.lens), c.M
    H, page, D = c.k.shape[1:]
    G = c.qf.shape[2] // H
    half = torch.finfo(c.dtype).eps / 2
    rp = 2.0 ** -11 if c.dtype == BF else 2.0 ** -22
    for b in range(B_):
        n = int(c.lens[b]) + M
        at = [(int(c.table[b, t // page]), t % page) for t in range(n)]
        line = np.tri(M, dtype=bool) if c.parent is None else C.ancestors(c.parent[b])
        for j in range(H * G):
            k = C.F.decode_e4m3(np.array([c.k[p, j // G, s] for p, s in at])) * float(KS)
            for v in np.nonzero(rows[b])[0]:
                see = np.concatenate([np.ones(n - M, dtype=bool), line[v]])
                q = c.qf[b, v, j].astype(np.float64)
                z = abs(sm) * (k[see] @ q) * np.sign(sm)
                ez = (D + 12) * u * abs(sm) * (np.abs(k[see]) @ np.abs(q)).max() + 8 * u * np.abs(z).max()
                second, first = np.sort(z)[-2:]
                assert first - second > 2 * ez + 200, "the case does not say which key wins"
                assert (np.abs(out[b, v, j] - ref[b, v, j]) <= (half + rp + 16 * u) * np.abs(ref[b, v, j])).all()
                assert abs(lse[b, v, j] - ref_lse[b, v, j]) <= ez + 8 * u * abs(ref_lse[b, v, j])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sm", [1e8, -3e9, 7e13, 1.1e30])
def test_attention_of_scores_past_the_exponents_precision(dtype, D, sm):
    """Scores from 1e9 to 1e31, of either sign: one key takes all, and its value comes out."""
    c = Case(dtype, [1500, 30], 5, 2, 3, D, 32, tree=True, seed=57 + D)
    every = np.ones((2, 5), dtype=bool)
    far_check(c, c.gpu(sm_scale=sm), every, float(np.float32(sm)))
    far_check(c, c.gpu(sm_scale=sm, workspace=torch.empty(0, dtype=torch.uint8, device=DEV)), every,
              float(np.float32(sm)))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_far_scores_beside_ordinary_ones(dtype, sign):
    """Nodes whose queries are 1e9 times as large share their row tiles with ordinary ones, and the keys of
    the first 1,400 tokens are zero: their rows' scores move from 0 to +-1e10 in the middle of the walk."""
    c = Case(dtype, [1500, 40], 6, 1, 2, 64, 32, seed=61)
    for t in range(1400):
        c.k[c.table[0, t // 32], :, t % 32] = 0
    q = c.qf.copy()
    q[:, 1::2] *= sign * 1e9
    c.q, c.qf = dtype_values(q, dtype)
    got = c.gpu()
    rows = np.zeros((2, 6), dtype=bool)
    rows[:, 1::2] = True
    far_check(c, got, rows, 1 / 8.0)
    near = Case.__new__(Case)
    near.__dict__.update(c.__dict__)
    for b in range(2):  # the ordinary rows by themselves, under the usual bound
        for v in range(0, 6, 2):
            near.qf, near.M = c.qf[b:b + 1, v:v + 1], 1
            near.lens, near.table = np.array([c.lens[b] + v]), c.table[b:b + 1]
            near.check([x[b:b + 1, v:v + 1] for x in got])


def test_a_sequence_cut_back_into_a_shared_page_goes_on_as_a_fork():
    """Sequence 0's 96 tokens are shared whole with sequence 1; 0 is cut back to 40, in the middle of a shared
    page, and goes on as its fork 2: 1 keeps its bytes, and both attend to what is theirs."""
    rng = np.random.default_rng(71)
    S, W, P, L, H, G, D, page, M = 3, 8, 30, 2, 2, 3, 64, 16, 12
    pool, t = C.Pool(S, W, P), list(B.kv_pool(S, W, P, DEV))
    host = np.zeros((2, L, P, H, page, D), dtype=np.uint8)
    pages = torch.from_numpy(host).to(DEV)

    def resize(seqs, tokens):
        assert int(B.nvfp4_kv_resize(*t, page, ints(seqs), ints(tokens))) == pool.resize(page, seqs, tokens) == 0
        check_pool(t, pool)

    def fork(src, dst, tokens):
        nonlocal host
        short, moves = pool.fork(page, [src], [dst], [tokens])
        assert int(B.nvfp4_kv_fork(*t, pages[0], pages[1], ints([src]), ints([dst]), ints([tokens]))) == short == 0
        host = np.stack([C.copy_slots(x, moves) for x in host])
        check_pool(t, pool)

    def append(rows, lens):
        x, xf = dtype_values(rng.standard_normal((2, S, rows, H, D)), BF)
        for l in range(L):
            B.nvfp4_kv_append(x[0], x[1], U.scalar(KS), U.scalar(VS), pages[0, l], pages[1, l], t[0], ints(lens))
            for kv, s in ((0, KS), (1, VS)):
                host[kv, l] = C.append(xf[kv], s, host[kv, l], pool.table, np.asarray(lens))
        np.testing.assert_array_equal(pages.cpu().numpy(), host)

    resize([0], [96])
    append(96, [0, -1, -1])
    fork(0, 1, 96)
    resize([0], [40])
    assert not pool.writable(0, page, 40, 41)  # its page is sequence 1's, too
    fork(0, 2, 40)
    resize([0, 2], [0, 40 + M])
    assert pool.writable(2, page, 40, 40 + M)
    before = host[:, :, pool.table[1, :6]].copy()
    append(M, [-1, -1, 40])
    np.testing.assert_array_equal(host[:, :, pool.table[1, :6]], before)
    c = Case.__new__(Case)
    c.q, c.qf = dtype_values(rng.standard_normal((S, M, H * G, D)), BF)
    c.k, c.v, c.table, c.lens, c.M, c.D = host[0, 1], host[1, 1], pool.table, np.array([-1, 84, 40]), M, D
    c.parent, c.counts, c.dtype = None, None, BF
    c.check(c.gpu())
