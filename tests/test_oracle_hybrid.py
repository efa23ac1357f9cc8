"""Pins of oracle/delta.py, oracle/rope.py and oracle/logprobs.py (CPU): closed forms, block forms and brute force; and
of the frequency tables that the binding makes."""
import numpy as np
import pytest

from nvfp4_w4a4_block_amd import binding as B
from oracle import delta as DR
from oracle import logprobs as LP
from oracle import rope as RP


def step(rng, nb=1, M=6, Hk=1, H=2, Dk=8, Dv=5, slots=3):
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    q, k, v, states = f(nb, M, Hk, Dk), f(nb, M, Hk, Dk), f(nb, M, H, Dv), f(slots, H, Dv, Dk)
    return q, k, v, -np.abs(f(nb, M, H)), 1 / (1 + np.exp(-f(nb, M, H))), states


def test_a_full_rate_stores_the_value_and_reads_it_back():
    rng = np.random.default_rng(0)
    q, k, v, g, beta, states = step(rng)
    g[:], beta[:] = 0.0, 1.0
    out, tol, after, off, big = DR.chain(k, k, v, g, beta, states, [0], [1], scale=1.0, eps=0.0)
    assert np.allclose(out[0], v[0])  # S k = v right after k was written
    assert (tol > 0).all() and (off[1] > 0).all() and not off[2].any()
    assert np.array_equal(after[0], states[0]) and (big[1] >= np.abs(after[1]) - 1e-12).all()


def test_hand_worked_tokens():
    one = lambda *x: np.array(x, dtype=np.float32).reshape(1, 2, 1, -1)  # noqa: E731
    k, q, v = one(1, 0, 0, 2), one(1, 0, 1, 1), one(6, 10)
    g, beta = np.log(np.array([[[0.5], [0.25]]])), np.array([[[0.5], [1.0]]])
    out, _, after, _, _ = DR.chain(q, k, v, g, beta, np.array([[[[4.0, 8.0]]]]), [0], [0], scale=1.0)
    # S = [2, 4], u = .5 (6 - 2) = 2, S = [4, 4], o = 4; S = [1, 1], u = 10 - 2 = 8, S = [1, 17], o = 18
    assert np.allclose(out.ravel(), [4, 18]) and np.allclose(after.ravel(), [1, 17])


@pytest.mark.parametrize("seed", range(4))
def test_tree_is_the_triangular_system_and_lines_are_chains(seed):
    rng = np.random.default_rng(seed)
    M = 9
    q, k, v, g, beta, states = step(rng, M=M, Hk=2, H=4)
    parent = np.array([[-1] + [int(rng.integers(-1, t)) for t in range(1, M)]])
    out, _, keys, upd, _ = DR.tree(q, k, v, g, beta, states, [2], parent, eps=1e-6)
    qn, kn = (np.repeat(DR.normalised(x, 1e-6), 2, axis=2) for x in (q, k))
    for h in range(4):
        line = np.zeros((M, M), bool)
        for t in range(M):
            u = t
            while u >= 0:
                line[t, u] = True
                u = parent[0, u]
        G = line @ g[0, :, h]
        decay = np.where(line, np.exp(G[:, None] - G[None]), 0)
        A = np.tril(beta[0, :, h, None] * decay * (kn[0, :, h] @ kn[0, :, h].T), -1)
        S = states[2, h].astype(np.float64)
        u = np.linalg.solve(np.eye(M) + A, beta[0, :, h, None] * (v[0, :, h] - np.exp(G)[:, None] * (kn[0, :, h] @ S.T)))
        o = np.exp(G)[:, None] * (qn[0, :, h] @ S.T) + (decay * (qn[0, :, h] @ kn[0, :, h].T)) @ u
        assert np.allclose(upd[0, :, h], u) and np.allclose(out[0, :, h], o / np.sqrt(8))
    assert np.allclose(keys, DR.normalised(k, 1e-6))
    lines = np.arange(M)[None] - 1
    a, b = DR.tree(q, k, v, g, beta, states, [0], lines), DR.chain(q, k, v, g, beta, states, [0], [1])
    assert np.allclose(a[0], b[0])
    result = np.array([[M - 1, M - 1, 0] + list(range(1, M)) + [-1]])
    after, size = DR.commit(states[None], a[2][None], a[3][None], g[None], result, [0], [1])
    assert np.allclose(after[0], b[2]) and (size >= np.abs(after) - 1e-12).all()


def test_slots_counts_and_pieces():
    rng = np.random.default_rng(5)
    q, k, v, g, beta, states = step(rng, nb=2, slots=5)
    out, _, after, _, _ = DR.chain(q, k, v, g, beta, states, [0, -1], [1, 3], counts=[4, 0])
    assert not out[0, 4:].any() and not out[1].any() and not after[3].any()
    assert np.array_equal(after[[0, 2, 4]], states[[0, 2, 4]])
    part = DR.chain(q[:1, :2], k[:1, :2], v[:1, :2], g[:1, :2], beta[:1, :2], states, [0], [0])[2]
    assert np.allclose(DR.chain(q[:1, 2:4], k[:1, 2:4], v[:1, 2:4], g[:1, 2:4], beta[:1, 2:4], part, [0], [1])[2][1],
                       after[1])
    src, dst = [0, 1, 2, 3, -2, 9], [4, 4, 3, 5, 6, 7]
    assert [DR.slot_written(src, dst, 8, b) for b in range(6)] == [4, -1, -1, 5, -1, -1]


def test_rope_keeps_lengths_and_depends_on_distance():
    rng = np.random.default_rng(1)
    inv = 10000.0 ** (-np.arange(0, 16, 2) / 16)
    x, y = rng.standard_normal((2, 1, 1, 24))
    for inter in (False, True):
        a, _ = RP.rotate(x, np.array([7]), inv, interleaved=inter)
        assert np.allclose((a ** 2).sum(), (x ** 2).sum()) and np.array_equal(a[..., 16:], x[..., 16:])
        dot = lambda p, r: (RP.rotate(x, np.array([p]), inv, 1.0, inter)[0] *  # noqa: E731
                            RP.rotate(y, np.array([r]), inv, 1.0, inter)[0]).sum()
        assert np.isclose(dot(1000, 990), dot(30, 20))
    one, _ = RP.rotate(np.array([[[1.0, 0.0]]]), np.array([1]), np.array([np.pi / 2]), 2.0)
    assert np.allclose(one, [[[0, 2]]])
    assert RP.depths([-1, 0, 0, 2, 5, 4]).tolist() == [0, 1, 1, 2, 0, 1]


def test_frequency_tables():
    plain, one = B.rope_frequencies(64)
    assert one == 1.0 and np.allclose(plain.numpy(), 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-15)
    linear, _ = B.rope_frequencies(64, scaling="linear", factor=4.0)
    assert np.allclose(linear.numpy() * 4, plain.numpy(), rtol=1e-15)
    ntk, _ = B.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1].item() * 4, plain[-1].item())
    yarn, scale = B.rope_frequencies(64, scaling="yarn", factor=4.0, trained=4096)
    turns = 4096 * plain.numpy() / (2 * np.pi)
    ratio = yarn.numpy() / plain.numpy()
    assert np.isclose(scale, 0.1 * np.log(4.0) + 1) and (np.diff(ratio) <= 1e-12).all()
    assert np.allclose(ratio[turns > 34 * 1.4], 1) and np.allclose(ratio[turns < 0.7], 0.25)
    for bad in (dict(rotary=24), dict(rotary=0), dict(rotary=32, base=1.0), dict(rotary=32, factor=0.5),
                dict(rotary=32, scaling="other"), dict(rotary=32, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            B.rope_frequencies(**bad)


def test_logprobs_by_brute_force_and_closed_forms():
    rng = np.random.default_rng(2)
    z = rng.standard_normal(40)
    p = np.exp(z) / np.exp(z).sum()
    lp, ent, best, ids = LP.row(z, 7, 40)
    assert np.isclose(lp, np.log(p[7])) and np.isclose(ent, -(p * np.log(p)).sum())
    assert np.allclose(best, np.log(np.sort(p)[::-1])) and np.allclose(p[ids], np.sort(p)[::-1])
    lp, ent, best, ids = LP.row(np.zeros(1000), 3, 4)
    assert np.isclose(ent, np.log(1000)) and ids.tolist() == [0, 1, 2, 3] and np.isclose(lp, -np.log(1000))
    z = np.array([-0.0, 0.0, -np.inf, 0.0])
    lp, ent, best, ids = LP.row(z, 2, 4)
    assert lp == -np.inf and ids.tolist() == [1, 3, 0, 2] and np.isclose(ent, np.log(3)) and best[3] == -np.inf
    for bad in ([np.nan, 1.0], [np.inf, 1.0], [-np.inf, -np.inf]):
        assert np.isnan(LP.row(np.array(bad), 0, 1)[1]) and LP.row(np.array(bad), 0, 1)[3].tolist() == [-1]
    assert np.isnan(LP.row(np.zeros(3), 3, 0)[0]) and np.isnan(LP.row(np.zeros(3), -1, 0)[0])
    lp, ent, _, _ = LP.row(np.array([0.0, 100.0]), 1, 0)
    assert np.isclose(lp, -np.exp(-100.0), rtol=1e-12) and np.isclose(ent, 101 * np.exp(-100.0), rtol=1e-12)
