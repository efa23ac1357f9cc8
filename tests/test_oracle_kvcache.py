"""Pins of the paged-cache oracle (oracle/kvcache.py): closed forms and exhaustive invariants, no
GPU.  Pages "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x Faster on Jetson
AGX Thor", sections on tree-based multi-token prediction and KV-cache reuse."""
import numpy as np
import pytest

from oracle import kvcache as C
from oracle import kvfp8 as KV

F32 = np.float32


def cache(rng, P, H, page, D):
    return KV.encode(rng.standard_normal((P, H, page, D)).astype(F32), F32(0.02))


def test_one_visible_token_returns_its_value():
    rng = np.random.default_rng(0)
    k, v = cache(rng, 3, 2, 16, 64), cache(rng, 3, 2, 16, 64)
    table, lens = np.array([[2, 0]]), np.array([0])
    q = rng.standard_normal((1, 1, 4, 64)).astype(F32)
    out, lse, _ = C.attention(q, k, v, F32(0.02), F32(0.02), table, lens)
    want = KV.decode_f32(v[2, :, 0], F32(0.02))
    np.testing.assert_allclose(out[0, 0], np.repeat(want, 2, axis=0), rtol=1e-6)
    z = (KV.decode_f32(k[2, :, 0], F32(0.02)).astype(np.float64).repeat(2, axis=0) * q[0, 0]).sum(-1) / 8
    np.testing.assert_allclose(lse[0, 0], z, rtol=1e-6, atol=1e-6)


def test_zero_queries_average_what_is_seen():
    rng = np.random.default_rng(1)
    k, v = cache(rng, 4, 1, 16, 64), cache(rng, 4, 1, 16, 64)
    table, lens = np.array([[3, 1, 0]]), np.array([20])
    parent = np.array([[-1, 0, 0, 1]])
    q = np.zeros((1, 4, 1, 64), F32)
    out, lse, _ = C.attention(q, k, v, 1.0, 1.0, table, lens, parent)
    x = KV.decode_f32(np.concatenate([v[3, 0], v[1, 0]]), F32(1)).astype(np.float64)
    for node, line in enumerate(([0], [0, 1], [0, 2], [0, 1, 3])):
        rows = list(range(20)) + [20 + u for u in line]
        np.testing.assert_allclose(out[0, node, 0], x[rows].mean(0), atol=1e-12)
        np.testing.assert_allclose(lse[0, node, 0], np.log(len(rows)))


def test_a_chain_is_the_tree_of_a_chain_and_counts_cut_it():
    rng = np.random.default_rng(2)
    k, v = cache(rng, 5, 2, 16, 64), cache(rng, 5, 2, 16, 64)
    table, lens = np.array([[0, 1], [2, 4]]), np.array([11, -1])
    q = rng.standard_normal((2, 6, 2, 64)).astype(F32)
    chain = np.tile(np.arange(-1, 5), (2, 1))
    a = C.attention(q, k, v, 0.02, 0.02, table, lens)
    b = C.attention(q, k, v, 0.02, 0.02, table, lens, chain)
    cut = C.attention(q, k, v, 0.02, 0.02, table, lens, counts=np.array([4, 6]))
    np.testing.assert_array_equal(a[0], b[0])
    np.testing.assert_array_equal(a[0][0, :4], cut[0][0, :4])
    assert not cut[0][0, 4:].any() and np.isneginf(cut[1][0, 4:]).all()
    assert not a[0][1].any() and np.isneginf(a[1][1]).all()


def test_ancestors():
    assert C.ancestors([-1, 0, 0, 2, 7]).astype(int).tolist() == [
        [1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0], [0, 0, 0, 0, 1]]


def test_append_then_compact_keeps_the_path():
    rng = np.random.default_rng(3)
    pages = cache(rng, 4, 2, 16, 64)
    table, lens = np.array([[1, 3, 0]]), np.array([13])
    x = rng.standard_normal((1, 6, 2, 64)).astype(F32)
    one = C.append(x, F32(0.02), pages, table, lens)
    result = np.array([[5, 2, 9, 2, 5, -1, -1, -1, -1]])
    out, new = C.compact(one[None], table, lens, result)
    assert new.tolist() == [16]
    path = KV.encode(x[0, [0, 2, 5]], F32(0.02))
    got = np.stack([out[0, 1, :, 13], out[0, 1, :, 14], out[0, 1, :, 15]])
    np.testing.assert_array_equal(got, path)
    np.testing.assert_array_equal(out[0, 2], pages[2])


def check_pool(pool):
    held = [int(p) for row, n in zip(pool.table, pool.held) for p in row[:n]]
    assert (np.bincount(held, minlength=len(pool.refs)) == pool.refs).all()
    assert sorted(pool.free) == np.nonzero(pool.refs == 0)[0].tolist()
    for row, n in zip(pool.table, pool.held):
        assert (row[n:] == -1).all() and len(set(row[:n].tolist())) == n


@pytest.mark.parametrize("seed", range(20))
def test_pool_invariants_hold_over_random_steps(seed):
    rng = np.random.default_rng(seed)
    S, W, P, page = 7, 6, 23, 16
    pool = C.Pool(S, W, P)
    short = 0
    for _ in range(60):
        n = int(rng.integers(1, 5))
        a, b = rng.integers(-1, S + 1, n), rng.integers(-1, S + 1, n)
        tokens = rng.integers(-3, page * (W + 1), n)
        before = (pool.table.copy(), pool.held.copy(), pool.refs.copy(), list(pool.free))
        if rng.random() < 0.5:
            got = pool.resize(page, a, tokens)
        else:
            got, moves = pool.fork(page, a, b, tokens)
            for x, y, used in moves:
                assert x != y and 0 < used < page and pool.refs[y] == 1
        check_pool(pool)
        if got:
            short += 1
            assert all(np.array_equal(x, y) for x, y in zip(before, (pool.table, pool.held, pool.refs, pool.free)))
    assert seed or short


def test_fork_shares_whole_pages_and_copies_the_rest():
    pool = C.Pool(3, 4, 10)
    assert pool.resize(16, [0], [40]) == 0
    short, moves = pool.fork(16, [0], [2], [37])
    assert short == 0 and moves == [(2, 3, 5)]
    assert pool.table[2].tolist() == [0, 1, 3, -1] and pool.refs[:5].tolist() == [2, 2, 1, 1, 0]
    pool.resize(16, [0], [0])
    assert pool.refs[:4].tolist() == [1, 1, 0, 1] and pool.free[-1] == 2


@pytest.mark.parametrize("seed", range(20))
def test_only_a_cut_back_leads_onto_a_shared_page_and_a_fork_leads_off_it(seed):
    """What the header says of shared pages: while sequences grow and are forked from committed tokens, the
    tokens that any of them writes next lie on pages of its own; one cut back into a shared page would
    write another's tokens, and its fork does not."""
    rng = np.random.default_rng(seed)
    S, W, page = 6, 8, 16
    pool, lens, cut = C.Pool(S, W, 60), np.zeros(S, dtype=np.int64), 0
    for _ in range(400):
        s, d = rng.permutation(S)[:2]
        what = rng.integers(0, 4)
        if what <= 1:  # a step: pages for its nodes, the nodes, some of them accepted
            n = int(min(lens[s] + rng.integers(1, 40), page * W))
            if pool.resize(page, [s], [n]):
                continue
            assert pool.writable(s, page, int(lens[s]), n)
            lens[s] = rng.integers(lens[s], n + 1)
        elif what == 2:  # a turn from committed tokens
            n = int(lens[s] - rng.integers(0, min(lens[s], 20) + 1))
            if pool.fork(page, [s], [d], [n])[0] == 0:
                lens[d] = n
        else:  # a cut back, continued as the header says
            n = int(rng.integers(0, lens[s] + 1))
            pool.resize(page, [s], [n])
            if n % page and not pool.writable(s, page, n, n + 1):
                cut += 1
                if pool.fork(page, [s], [d], [n])[0] == 0:
                    pool.resize(page, [s], [0])
                    lens[d], lens[s] = n, 0
                    assert pool.writable(d, page, n, n + 1)
                else:
                    pool.resize(page, [s], [0])
                    lens[s] = 0
            else:
                lens[s] = n
        check_pool(pool)
    assert cut
