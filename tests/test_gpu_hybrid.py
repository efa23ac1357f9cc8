"""GPU parity of the gated delta rule, the rotary append and the token log probabilities against oracle/.  Pages
"TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x Faster on Jetson AGX Thor", sections on KV-cache
reuse (a hybrid's recurrent states are kept with its pages) and tree-based multi-token prediction.

Bounds.  Delta rule: oracle/delta.py follows how far a state may be off, with u = 2^-22 for the factors of a state and
(Dk + 80) of them for its sums (Dk products, a block of at most 64 tokens, the scalars); an output adds the half step of
its type, and in bf16 calls three factors rounded to f16 (2^-11 each: q and the state, or the score and u).  Four times
that bound is granted, because a block's u come from the inverse of a triangular matrix, whose own rounding the
recurrence does not follow.  Rope: angles are off by 2^-26 turns (2 pi 2^-26 < 2^-23 rad) and their sine and cosine by
2^-23, the two products and their sum by 3 * 2^-24: 2^-21 of |x| + |y|.  Log probabilities: a sum of N terms in fp32,
each off by 2^-22 (its argument's rounding in an exponent of up to |z - m|), is off by (N / 64 + 64) 2^-24 at most as it is
summed in at least 64 lanes."""
import numpy as np
import pytest
import torch

import gpu_util as U
from nvfp4_w4a4_block_amd import binding as B
from oracle import delta as DR
from oracle import kvcache as KC
from oracle import kvfp8 as KV
from oracle import logprobs as LP
from oracle import rope as RP
from oracle import tree as TR

pytestmark = pytest.mark.gpu
DEV = U.DEV
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    U.require_gpu_lib()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def floats(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV)


def typed(x, dtype):
    """(device tensor of dtype, its values as float32)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dtype)
    return t.to(DEV), t.float().numpy()


def random_trees(rng, nb, M):
    return np.array([[-1] + [int(rng.integers(max(0, v - 4), v)) for v in range(1, M)] for _ in range(nb)],
                    dtype=np.int32).reshape(nb, M)


class Delta:
    """A step's rows and states: keys share a direction, some decays are strong."""

    def __init__(self, dtype, nb, M, Hk, H, Dk, Dv, norm=True, counts=None, slots=None, src=None, dst=None, seed=0,
                 wide=False, decay=3.0):
        rng = np.random.default_rng(seed)
        k = rng.standard_normal((nb, M, Hk, Dk)) + 0.5 * rng.standard_normal((nb, 1, Hk, Dk))
        q = rng.standard_normal((nb, M, Hk, Dk))
        if not norm:
            q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
        v = rng.standard_normal((nb, M, H, Dv))
        if counts is not None:  # what rows that are no tokens hold is not read
            for b, c in enumerate(counts):
                for x in (q, k, v):
                    x[b, max(0, c):] = np.nan
        self.dtype, self.dims = dtype, (nb, M, Hk, H, Dk, Dv)
        if wide:  # column ranges of one projection's output
            n = 2 * Hk * Dk + H * Dv
            both = np.full((nb, M, n + 16), 77.0)
            parts, at = [], 0
            for x in (q, k, v):
                w = x.shape[2] * x.shape[3]
                both[:, :, at:at + w] = x.reshape(nb, M, w)
                parts.append((at, w, x.shape[2:]))
                at += w
            t, f = typed(both, dtype)
            (self.q, self.qf), (self.k, self.kf), (self.v, self.vf) = (
                (t[:, :, a:a + w].unflatten(2, s), f[:, :, a:a + w].reshape((nb, M) + s)) for a, w, s in parts)
        else:
            (self.q, self.qf), (self.k, self.kf), (self.v, self.vf) = (typed(x, dtype) for x in (q, k, v))
        self.g = -np.exp(1.5 * rng.standard_normal((nb, M, H)) - decay).astype(np.float32)
        self.beta = (1 / (1 + np.exp(-1.5 * rng.standard_normal((nb, M, H))))).astype(np.float32)
        slots = 2 * nb + 1 if slots is None else slots
        self.states = (rng.standard_normal((slots, H, Dv, Dk)) * 2 / np.sqrt(Dk)).astype(np.float32)
        order = rng.permutation(slots)
        self.src = np.asarray(order[:nb] if src is None else src, dtype=np.int32)
        self.dst = np.asarray(order[nb:2 * nb] if dst is None else dst, dtype=np.int32)
        self.counts, self.eps, self.scale = counts, 1e-6 if norm else None, None
        self.rounded = 2.0 ** -11 if dtype == BF else 0.0

    def common(self):
        kw = dict(counts=None if self.counts is None else ints(self.counts), norm_eps=self.eps, scale=self.scale)
        return (self.q, self.k, self.v, floats(self.g), floats(self.beta)), kw

    def chain(self, states=None, **more):
        rows, kw = self.common()
        states = floats(self.states) if states is None else states
        kw.update(more)
        return B.nvfp4_delta_rule(*rows, states, ints(self.src), ints(self.dst), **kw), states

    def chain_ref(self):
        return DR.chain(self.qf, self.kf, self.vf, self.g, self.beta, self.states, self.src, self.dst, self.counts,
                        self.scale, self.eps, self.rounded)

    def near(self, got, ref, tol, what):
        half = torch.finfo(self.dtype).eps / 2
        tol = 4 * tol + half * (np.abs(ref) + 4 * tol)
        got = got.double().cpu().numpy()
        err = np.abs(got - ref)
        assert np.isfinite(got).all() and (err <= tol).all(), (what, (err / np.maximum(tol, 1e-300)).max())

    def check_chain(self, out, states):
        ref, tol, after, off, big = self.chain_ref()
        self.near(out, ref, tol, "out")
        got = states.double().cpu().numpy()
        err = np.sqrt(((got - after) ** 2).sum(-1))
        tol = 4 * off + 2.0 ** -23 * np.sqrt((after ** 2).sum(-1)) * (off > 0)
        assert np.isfinite(got).all() and (err <= tol).all(), ("states", (err / np.maximum(tol, 1e-300)).max())
        # roundings of either sign: as a whole a state is off by the root of their number, not by it
        whole = np.sqrt((err ** 2).sum(-1)), 2 * np.sqrt(self.dims[4] + 80) * DR.U * np.sqrt((big ** 2).sum((-1, -2)))
        assert (whole[0] <= whole[1]).all(), ("a whole state", (whole[0] / np.maximum(whole[1], 1e-300)).max())


SHAPES = [(1, 1, 64, 64), (2, 2, 64, 128), (1, 3, 128, 64), (4, 8, 128, 128), (2, 6, 256, 64), (1, 2, 64, 256),
          (1, 1, 256, 256)]


# ----------------------------------------------------------------------------------------------- delta rule, chain


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 64, 65, 130])
def test_chain_matches_oracle(dtype, M):
    for i, (Hk, H, Dk, Dv) in enumerate(SHAPES[M % 2::2]):
        c = Delta(dtype, 1 + i, M, Hk, H, Dk, Dv, norm=i % 2 == 0, seed=M + i, wide=i == 1)
        c.check_chain(*c.chain())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,shape", [(257, (1, 3, 128, 128)), (512, (2, 2, 128, 64)), (777, (1, 1, 64, 64)),
                                     (320, (1, 2, 256, 64)), (1300, (1, 1, 64, 64))])
def test_long_chains(dtype, M, shape):
    c = Delta(dtype, 2, M, *shape, seed=M, decay=5.0)
    c.check_chain(*c.chain())


@pytest.mark.parametrize("M,shape,dtype", [(2300, (1, 1, 128, 64), BF), (2200, (1, 2, 64, 64), BF),
                                           (2113, (1, 1, 64, 128), FP), (2500, (1, 1, 128, 64), FP)])
def test_chains_of_more_than_32_blocks(M, shape, dtype):
    """Sequences that end in the first block, between and at the end, new ones and ones without tokens."""
    counts = [M, 2112, 63, 0, 2049, 1]
    c = Delta(dtype, 6, M, *shape, counts=counts, slots=13, src=[0, -1, 2, 3, 4, 5], dst=[6, 7, 8, 9, 4, 11], seed=M,
              decay=5.0)
    out, states = c.chain()
    c.check_chain(out, states)
    assert not out[2, 63:].any() and not out[3].any() and not out[5, 1:].any()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [3, 12, 70, 200])
def test_ragged_chains_new_and_unused(dtype, M):
    counts = [M, 0, -4, M + 9, 1, M // 2, M - 1]
    src = [-1, 3, 4, 0, -2, 2, 99]
    dst = [5, 6, -1, 0, 1, 12, 7]
    c = Delta(dtype, 7, M, 2, 4, 64, 64, counts=counts, slots=12, src=src, dst=dst, seed=M)
    out, states = c.chain()
    c.check_chain(out, states)
    assert not out[1].any() and not out[4].any() and not out[6].any() and not out[5, M // 2:].any()
    after = states.cpu().numpy()
    assert np.array_equal(after[6], c.states[3])  # no tokens: the state is copied
    for s in (1, 2, 3, 4, 7, 8, 9, 10, 11):  # slots of unused sequences, sources and the others
        assert np.array_equal(after[s], c.states[s]), s


@pytest.mark.parametrize("nb,M,dtype", [(900, 130, FP), (1900, 70, FP), (1200, 200, BF)])
def test_calls_that_take_several_rounds(nb, M, dtype):
    """What is prepared of a block of so many sequences is past a round's workspace: states are carried from one
    round to the next, and the sequences themselves taken in turns."""
    counts = np.full(nb, M)
    counts[::7] = 65
    c = Delta(dtype, nb, M, 1, 1, 64, 64, slots=nb, src=np.arange(nb), dst=np.arange(nb), seed=21)
    c.counts = counts
    need = B.load().nvfp4_delta_rule_workspace_bytes(nb, M, 1, 1, 64, 64, B.NVFP4_F32 if dtype == FP else B.NVFP4_BF16)
    assert 64 << 20 < need < 256 << 20
    out, states = c.chain()
    some = np.random.default_rng(0).permutation(nb)[:24]
    some = np.concatenate([some, [0, 7, nb - 1]])
    for name in ("qf", "kf", "vf", "g", "beta", "states"):
        setattr(c, name, getattr(c, name)[some])
    c.counts, c.src, c.dst, n = counts[some], np.arange(len(some)), np.arange(len(some)), len(some)
    c.dims = (n,) + c.dims[1:]
    c.check_chain(out[torch.from_numpy(some).to(DEV)], states[torch.from_numpy(some).to(DEV)])


@pytest.mark.parametrize("M", [1, 20, 100])
def test_slots_that_two_sequences_name(M):
    # 0 and 1: the first goes into 5, the second nowhere; 2's dst is 3's src; 4 and 5 share a src, 4 stays in place
    src, dst = [0, 1, 2, 3, 4, 4, -1], [5, 5, 3, 6, 4, 7, 7]
    c = Delta(BF, 7, M, 1, 2, 64, 64, slots=9, src=src, dst=dst, seed=3)
    out, states = c.chain()
    c.check_chain(out, states)
    after = states.cpu().numpy()
    for s in (0, 1, 2, 3, 4, 8):  # 4 is the src of sequence 5 too
        assert np.array_equal(after[s], c.states[s]), s
    assert not np.array_equal(after[5], c.states[5]) and not np.array_equal(after[7], c.states[7])


@pytest.mark.parametrize("M", [1, 7, 40, 150])
def test_in_place_and_many_sequences(M):
    n = 70 if M < 40 else 5
    slots = np.random.default_rng(0).permutation(n)
    c = Delta(BF, n, M, 1, 1, 64, 64, slots=n, src=slots, dst=slots, seed=9)
    c.check_chain(*c.chain())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [2, 18, 90])
def test_decays_and_rates_at_their_ends(dtype, M):
    rng = np.random.default_rng(M)
    c = Delta(dtype, 2, M, 1, 4, 64, 64, seed=M)
    c.g[:, :, 0] = 0.0  # nothing is forgotten
    c.g[:, rng.permutation(M)[: M // 2], 1] = -np.inf  # all is, now and then
    c.g[:, :, 2] = -np.float32(80) * rng.random((2, M))
    c.g[:, :, 3] *= 1e-4
    c.beta[:, :, 0] = 1.0
    c.beta[:, :, 1] = np.where(rng.random((2, M)) < 0.5, 0.0, 1.0)
    c.beta[0, :, 3] = 0.0
    c.check_chain(*c.chain())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [1, 24, 100])
def test_equal_keys_and_large_states(dtype, M):
    """One key again and again (the triangular system is at its worst), states of 1e20 and of 1e-20."""
    c = Delta(dtype, 1, M, 1, 3, 128, 64, seed=M)
    c.k[:] = c.k[:, :1]
    c.kf[:] = c.kf[:, :1]
    c.beta[:, :, 0], c.g[:, :, 0] = 1.0, 0.0
    c.states[:, 1] *= 1e20
    c.states[:, 2] *= 1e-20
    c.check_chain(*c.chain())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [1, 30, 129])
def test_zero_and_tiny_and_huge_rows(dtype, M):
    """Zero keys, keys and queries of very different lengths, values that reach 1e30."""
    rng = np.random.default_rng(M)
    c = Delta(dtype, 1, M, 2, 2, 64, 64, seed=M)
    gain = torch.from_numpy(2.0 ** rng.integers(-40, 40, (1, M, 2, 1))).to(DEV)
    c.q.mul_(gain.to(dtype))
    c.k.mul_(gain.flip(1).to(dtype))
    c.k[:, M // 2] = 0
    c.v[:, :, 1] *= 1e30
    c.qf, c.kf, c.vf = (x.float().cpu().numpy() for x in (c.q, c.k, c.v))
    c.check_chain(*c.chain())


@pytest.mark.parametrize("M", [2, 20, 100])
def test_scale_argument_and_given_buffers(M):
    c = Delta(FP, 2, M, 1, 2, 64, 128, seed=1)
    c.scale = -2.5
    out = torch.full((2, M, 2, 128), 9.0, device=DEV)
    need = B.load().nvfp4_delta_rule_workspace_bytes(2, M, 1, 2, 64, 128, B.NVFP4_F32)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    got, states = c.chain(out=out, workspace=ws)
    assert got is out
    c.check_chain(out, states)
    assert (ws[need:] == 255).all()
    none, _ = c.chain(workspace=ws[:0])  # too little: one token after the other
    c.near(none, *c.chain_ref()[:2], "out")


@pytest.mark.parametrize("M", [1, 5, 33, 140])
def test_a_nan_stays_in_its_sequence_and_head(M):
    c = Delta(BF, 3, M, 2, 4, 64, 64, seed=5)
    ref, ref_states = (x.clone() for x in c.chain())
    c.v[1, M // 2, 1, 3] = float("nan")
    c.k[2, M - 1, 0, 0] = float("inf")
    out, states = c.chain()
    assert torch.equal(out[0], ref[0]) and torch.equal(states[c.dst[0]], ref_states[c.dst[0]])
    assert torch.equal(out[1, :, [0, 2, 3]], ref[1, :, [0, 2, 3]])
    assert out[1, M // 2, 1, 3].isnan() and states[c.dst[1], 1, 3].isnan().any()
    assert torch.equal(out[2, :, 2:], ref[2, :, 2:]) and out[2, M - 1, :2].isnan().all()


def test_a_chain_in_pieces_is_the_chain():
    c = Delta(FP, 2, 200, 1, 2, 64, 64, src=[0, 1], dst=[2, 3], slots=4, seed=8)
    whole, states = c.chain()
    pieces, at = [], 0
    st = floats(c.states)
    for n in (1, 3, 16, 64, 100, 16):
        s = ints(c.src if at == 0 else c.dst)
        pieces.append(B.nvfp4_delta_rule(*(x[:, at:at + n].contiguous() for x in c.common()[0]), st, s, ints(c.dst),
                                         norm_eps=1e-6))
        at += n
    c.check_chain(torch.cat(pieces, 1), st)
    c.check_chain(whole, states)


def test_no_rows_copy_the_states():
    c = Delta(BF, 2, 0, 1, 2, 64, 64, src=[0, -1], dst=[2, 3], slots=4)
    out, states = c.chain()
    assert out.shape == (2, 0, 2, 64) and torch.equal(states[2], states[0]) and not states[3].any()


# ----------------------------------------------------------------------------------------------- delta rule, trees


def run_tree(c, parent, **more):
    rows, kw = c.common()
    kw.update(more)
    states = floats(c.states)
    got = B.nvfp4_delta_tree(*rows, states, ints(c.src), ints(parent), **kw)
    assert torch.equal(states, floats(c.states))
    return got


def check_tree(c, parent, got):
    out, keys, updates = got
    ref, tol, kref, uref, utol = DR.tree(c.qf, c.kf, c.vf, c.g, c.beta, c.states, c.src, parent, c.counts, c.scale,
                                         c.eps, c.rounded)
    c.near(out, ref, tol, "out")
    Dk = c.dims[4]
    assert np.abs(keys.cpu().numpy() - kref).max(initial=0) <= (Dk + 4) * 2.0 ** -24 * np.abs(kref).max(initial=0)
    err = np.abs(updates.double().cpu().numpy() - uref)
    assert (err <= 4 * utol + 2.0 ** -23 * np.abs(uref)).all(), (err / np.maximum(utol, 1e-300)).max()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M", [1, 2, 5, 15, 16, 17, 32, 33, 48, 49, 63, 64])
def test_tree_matches_oracle(dtype, M):
    rng = np.random.default_rng(M)
    for i, (Hk, H, Dk, Dv) in enumerate(SHAPES[M % 3::3]):
        c = Delta(dtype, 1 + i, M, Hk, H, Dk, Dv, norm=i != 1, seed=M, wide=i == 0)
        parent = random_trees(rng, 1 + i, M)
        check_tree(c, parent, run_tree(c, parent))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_ragged_trees_roots_and_unused(dtype):
    M, rng = 21, np.random.default_rng(1)
    c = Delta(dtype, 6, M, 2, 4, 128, 64, counts=[M, 0, 7, 90, 3, 5], slots=4, src=[0, 1, -1, 3, 4, -7], seed=2)
    parent = random_trees(rng, 6, M)
    parent[0, 5], parent[0, 9], parent[2, 3], parent[3, 1:] = 5, 40, -9, -1  # more roots
    got = run_tree(c, parent)
    check_tree(c, parent, got)
    for x in got:
        assert not x[1].any() and not x[2, 7:].any() and not x[4:].any()


def test_a_line_is_a_chain_and_its_commit_the_chains_state():
    M = 40
    c = Delta(FP, 1, M, 1, 2, 128, 128, src=[0], dst=[1], slots=2, seed=4)
    line = np.arange(M, dtype=np.int32)[None] - 1
    got = run_tree(c, line)
    check_tree(c, line, got)
    out, states = c.chain()
    ref, tol = c.chain_ref()[:2]
    c.near(got[0], ref, tol, "out")
    st = floats(c.states)
    result = ints([[M - 1, M - 1, 0] + list(range(1, M)) + [-1]])
    B.nvfp4_delta_commit(st[None], got[1][None], got[2][None], floats(c.g)[None], result, ints([0]), ints([1]))
    c.check_chain(out, st)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_tree_decays_at_their_ends(dtype):
    M, rng = 37, np.random.default_rng(2)
    c = Delta(dtype, 1, M, 1, 3, 64, 64, seed=6)
    c.g[:, ::5, 0] = -np.inf
    c.g[:, :, 1] = 0.0
    c.beta[:, :, 1] = 1.0
    c.g[:, :, 2] *= 500
    parent = random_trees(rng, 1, M)
    check_tree(c, parent, run_tree(c, parent))


# ----------------------------------------------------------------------------------------------- delta rule, commit


@pytest.mark.parametrize("L,nb,M,Hk,H,Dk,Dv", [(1, 1, 1, 1, 1, 64, 64), (3, 2, 16, 2, 6, 128, 128),
                                               (2, 5, 33, 1, 2, 64, 256), (1, 2, 64, 2, 2, 256, 64)])
def test_commit_matches_oracle(L, nb, M, Hk, H, Dk, Dv):
    rng = np.random.default_rng(M)
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    states, keys, updates = f32(L, 2 * nb + 1, H, Dv, Dk), f32(L, nb, M, Hk, Dk), f32(L, nb, M, H, Dv)
    g = -np.exp(f32(L, nb, M, H) - 2)
    g[:, :, M // 3::7, 0] = -np.inf
    result = np.full((nb, 3 + M), -1, dtype=np.int32)
    for b in range(nb):
        n = [M - 1, 0, M // 2, M + 5, -3][b % 5]
        result[b, :3] = 0, n, 7
        path = np.sort(rng.permutation(np.arange(1, M))[: max(0, min(n, M - 1))])
        result[b, 3:3 + len(path)] = path
        if len(path) > 3:
            result[b, 4], result[b, 5] = -1, M  # passed over
    src, dst = rng.permutation(2 * nb)[:nb].astype(np.int32), np.arange(nb, dtype=np.int32)
    dst[:] = src  # in place
    if nb > 1:
        src[0], dst[1] = -1, 2 * nb  # from zeros, and into the slot that no other names
        dst[0] = src[1] if nb < 3 else dst[0]  # another's src: not written
    got = floats(states)
    B.nvfp4_delta_commit(got, floats(keys), floats(updates), floats(g), ints(result), ints(src), ints(dst))
    ref, size = DR.commit(states, keys, updates, g, result, src, dst)
    err = np.abs(got.double().cpu().numpy() - ref)
    # up to 65 products summed, each factor e^x off by 2^-23 (1 + |x|), and x at most 88 where it is not zero
    tol = (66 * 2.0 ** -24 + 90 * 2.0 ** -23) * size
    changed = (ref != states).any((0, 2, 3, 4))
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    assert torch.equal(got[:, ~torch.from_numpy(changed)].cpu(), torch.from_numpy(states[:, ~changed]))


def test_commit_slots_that_two_sequences_name():
    rng = np.random.default_rng(0)
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    states, keys, updates = f32(2, 6, 1, 64, 64), f32(2, 4, 2, 1, 64), f32(2, 4, 2, 1, 64)
    g, result = -np.abs(f32(2, 4, 2, 1)), np.tile(np.array([0, 0, 0, -1, -1], dtype=np.int32), (4, 1))
    src, dst = [0, 1, 2, -5], [4, 4, 0, 5]  # 1: an earlier dst; 2: a src; 3: not in use
    got = floats(states)
    B.nvfp4_delta_commit(got, floats(keys), floats(updates), floats(g), ints(result), ints(src), ints(dst))
    same = [0, 1, 2, 3, 5]
    assert torch.equal(got[:, same].cpu(), torch.from_numpy(states[:, same]))
    ref, _ = DR.commit(states, keys, updates, g, result, src, dst)
    assert np.abs(got.cpu().numpy() - ref).max() < 1e-5


# ----------------------------------------------------------------------------------------------- rotary append

KS, VS = np.float32(0.0123), np.float32(0.0171)


class Rope:
    def __init__(self, dtype, lens, M, Hq, H, D, R, page, tree=False, counts=None, interleaved=False, scale=1.0,
                 seed=0, wide=False, base=10000.0):
        rng = np.random.default_rng(seed)
        nb = len(lens)
        self.lens, self.counts, self.M, self.dtype = np.asarray(lens), counts, M, dtype
        self.W = -(-(max(max(lens), 0) + M) // page)
        P = nb * (M // page + 2) + 2
        order = rng.permutation(P)
        self.table = np.full((nb, self.W), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(lens):
            for w in range(max(n, 0) // page, -(-(max(n, 0) + M) // page)):
                self.table[b, w] = order[at]
                at += 1
        self.parent = random_trees(rng, nb, M) if tree else None
        self.inv = base ** (-np.arange(0, R, 2) / R)
        self.scale, self.interleaved = scale, interleaved
        if wide:
            t, f = typed(rng.standard_normal((nb, M, (Hq + 2 * H) * D)) * 2, dtype)
            cut = np.cumsum([0, Hq * D, H * D, H * D])
            (self.q, self.qf), (self.k, self.kf), (self.v, self.vf) = (
                (t[:, :, a:e].unflatten(2, (-1, D)), f[:, :, a:e].reshape(nb, M, -1, D)) for a, e in zip(cut, cut[1:]))
        else:
            (self.q, self.qf), (self.k, self.kf), (self.v, self.vf) = (
                typed(rng.standard_normal((nb, M, h, D)) * 2, dtype) for h in (Hq, H, H))
        self.start = [rng.integers(0, 256, (P, H, page, D), dtype=np.uint8) for _ in range(2)]

    def gpu(self, **kw):
        pages = [torch.from_numpy(x.copy()).to(DEV) for x in self.start]
        args = dict(parent=None if self.parent is None else ints(self.parent),
                    counts=None if self.counts is None else ints(self.counts), interleaved=self.interleaved,
                    rope_scale=self.scale)
        args.update(kw)
        q = B.nvfp4_kv_append_rope(self.q, self.k, self.v, torch.from_numpy(self.inv).to(DEV), U.scalar(KS),
                                   U.scalar(VS), *pages, ints(self.table), ints(self.lens), **args)
        return q, pages

    def check(self, q, pages):
        q, k, v = q.double().cpu().numpy(), pages[0].cpu().numpy(), pages[1].cpu().numpy()
        want_v = KC.append(self.vf, VS, self.start[1], self.table, self.lens, self.counts)
        assert np.array_equal(v, want_v)
        grid = KV.decode_f32(np.arange(127, dtype=np.uint8), np.float32(1.0)).astype(np.float64)
        grid = np.concatenate([-grid[:0:-1], grid])
        mid = (grid[1:] + grid[:-1]) / 2
        half = torch.finfo(self.dtype).eps / 2
        rest = np.ones(k.shape, dtype=bool)
        for b, n in enumerate(self.lens):
            c = 0 if n < 0 else self.M if self.counts is None else max(0, min(self.M, self.counts[b]))
            depth = np.arange(c) if self.parent is None else RP.depths(self.parent[b].tolist())[:c]
            ref, size = RP.rotate(self.qf[b, :c].astype(np.float64), n + depth, self.inv, self.scale, self.interleaved)
            tol = half * np.abs(ref) + 2.0 ** -21 * (1 + half) * size
            assert (np.abs(q[b, :c] - ref) <= tol).all(), (np.abs(q[b, :c] - ref) / np.maximum(tol, 1e-300)).max()
            assert not q[b, c:].any()
            ref, size = RP.rotate(self.kf[b, :c].astype(np.float64), n + depth, self.inv, self.scale, self.interleaved)
            inv = float(np.float32(1) / KS)
            y, tol = ref * inv, (2.0 ** -21 * size + 2.0 ** -23 * np.abs(ref)) * inv
            for t in range(c):
                at = KC._slot(k, self.table, b, int(n) + t)
                if at is None:
                    continue
                rest[at[0], :, at[1]] = False
                got = KV.decode_f32(k[at[0], :, at[1]], np.float32(1.0)).astype(np.float64)
                # rounding keeps order: the byte's value lies between those of the bound's two ends
                low = grid[np.searchsorted(mid, y[t] - tol[t], side="left")]
                high = grid[np.searchsorted(mid, y[t] + tol[t], side="right")]
                assert ((low <= got) & (got <= high)).all()
        assert np.array_equal(k[rest], self.start[0][rest])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,M,Hq,H,D,R,page,tree,counts", [
    ([0], 1, 1, 1, 64, 16, 16, False, None), ([5, 131], 16, 10, 2, 128, 64, 64, True, None),
    ([3, -1, 40, 0, 7], 9, 4, 4, 64, 64, 16, False, [9, 9, 0, 30, 4]), ([17, 1], 64, 3, 1, 256, 96, 32, True, [64, 11]),
    ([1000], 130, 5, 5, 128, 128, 128, False, None), ([2], 7, 6, 3, 128, 112, 16, False, None)])
def test_rope_matches_oracle(dtype, interleaved, lens, M, Hq, H, D, R, page, tree, counts):
    for wide in (False, True):
        c = Rope(dtype, lens, M, Hq, H, D, R, page, tree, counts, interleaved, scale=1.0 if wide else 1.21, seed=M,
                 wide=wide)
        c.check(*c.gpu())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("start", [1 << 20, (1 << 24) + 1, (1 << 27) - 40])
def test_rope_far_positions(dtype, start):
    c = Rope(dtype, [start], 33, 2, 1, 64, 64, 1024, seed=1)
    c.check(*c.gpu())


def test_rope_tokens_without_a_page():
    c = Rope(BF, [30, 2], 40, 2, 2, 64, 32, 16, seed=2)
    c.table[0, 2], c.table[1, 0] = -1, 1 << 20
    c.check(*c.gpu())
    c.table = np.ascontiguousarray(c.table[:, :3])  # tokens behind the table
    c.check(*c.gpu())


def test_rope_in_place_and_trees_with_more_roots():
    c = Rope(BF, [50, 9], 12, 4, 2, 128, 128, 16, tree=True, seed=3)
    c.parent[0, 4], c.parent[1, 11] = 4, -3
    c.check(*c.gpu())
    q = c.q.clone()
    got, pages = c.q, [torch.from_numpy(x.copy()).to(DEV) for x in c.start]
    c.q = q
    out, pages = c.gpu(q_out=q)
    assert out is q
    c.check(out, pages)
    c.q = got


def test_rope_without_turning_is_append():
    c = Rope(BF, [7, 90], 20, 3, 2, 64, 64, 16, seed=4)
    c.inv[:] = 0.0
    q, pages = c.gpu()
    assert torch.equal(q, c.q)
    assert np.array_equal(pages[0].cpu().numpy(), KC.append(c.kf, KS, c.start[0], c.table, c.lens))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
def test_turned_codes_are_the_nearest(dtype, interleaved):
    """A turned key times fl32(1 / scale) is rounded once.  Up to position 60,500 the angle is off by no more than
    2^-52 * 60,500 + 2e-11, so a value within 4e-11 of its pair's size from the middle of two codes may go to either."""
    c = Rope(dtype, [60000], 500, 1, 4, 128, 128, 64, interleaved=interleaved, scale=1.25, seed=9)
    q, pages = c.gpu()
    ref, size = RP.rotate(c.kf[0].astype(np.float64), 60000 + np.arange(500), c.inv, c.scale, interleaved)
    y, near = ref * float(np.float32(1) / KS), 4e-11 * size * float(np.float32(1) / KS)
    grid = KV.decode_f32(np.arange(127, dtype=np.uint8), np.float32(1.0)).astype(np.float64)
    grid = np.concatenate([-grid[:0:-1], grid])
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = (grid[np.searchsorted(mid, y + s * near)] for s in (-1, 1))
    k = pages[0].cpu().numpy()
    for t in range(500):
        page, at = KC._slot(k, c.table, 0, 60000 + t)
        got = KV.decode_f32(k[page, :, at], np.float32(1.0)).astype(np.float64)
        assert ((got == low[t]) | (got == high[t])).all(), t


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_nan_and_saturates_infinities(dtype, interleaved):
    c = Rope(dtype, [5, 20], 4, 2, 2, 64, 32, 16, interleaved=interleaved, seed=10)
    for x in (c.q, c.k):
        x[0, 1, 0, 3], x[0, 2, 1, 40], x[1, 0, 1, 2], x[1, 3, 0, 50] = (float("nan"), float("nan"), float("inf"),
                                                                       -float("inf"))
    q, pages = c.gpu()
    other = (lambda d: d ^ 1) if interleaved else (lambda d: d ^ 16)
    bad = np.zeros((2, 4, 2, 64), dtype=bool)
    bad[0, 1, 0, [3, other(3)]] = bad[0, 2, 1, 40] = True
    got = q.float().cpu().numpy()
    assert np.array_equal(np.isnan(got), bad)
    big = np.zeros_like(bad)
    big[1, 0, 1, [2, other(2)]] = big[1, 3, 0, 50] = True
    assert np.array_equal(np.isinf(got), big)
    k = pages[0].cpu().numpy()
    for b in range(2):
        for t in range(4):
            page, at = KC._slot(k, c.table, b, int(c.lens[b]) + t)
            code = k[page, :, at] & 127
            assert np.array_equal(code == 127, bad[b, t])
            assert (code[big[b, t]] == 126).all()


# ----------------------------------------------------------------------------------------------- log probabilities


def check_logprobs(z, tokens, top, got):
    lp, ent, best, ids = (x.cpu().numpy() for x in got)
    N = z.shape[1]
    for i in range(len(z)):
        a, e, b, o = LP.row(z[i].astype(np.float64), int(tokens[i]), top)
        assert np.array_equal(ids[i], o), (i, ids[i], o)
        if np.isnan(e):
            assert np.isnan(ent[i]) and np.isnan(lp[i]) and np.isnan(best[i]).all()
            continue
        live = z[i][np.isfinite(z[i])].astype(np.float64)
        span = min(104.0, float(live.max() - live.min()))
        # every e^(z - m): z - m is rounded once, e^x by 2^-23; sums as the docstring has them
        rel = (span + 2) * 2.0 ** -23 + (N / 64 + 64) * 2.0 ** -24
        # log1p(a) is off by rel a / (1 + a) at most, and a / (1 + a) = 1 - e^(the best's log p)
        small = -np.expm1(b[0]) if top else 1.0
        assert abs(ent[i] - e) <= 2 * rel * (e + small) + 2.0 ** -22 * e + 1e-37, (i, ent[i], e)
        for x, y in [(lp[i], a)] + list(zip(best[i], b)):
            if not np.isfinite(y):
                assert np.array_equal(np.float64(x), y, equal_nan=True), (i, x, y)
            else:
                assert abs(x - y) <= rel * small + 2.0 ** -23 * abs(y) + 1e-37, (i, x, y)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,N,top", [(1, 1, 1), (3, 2, 0), (5, 63, 63), (2, 1000, 64), (4, 4097, 20), (1, 151936, 20),
                                     (2, 50257, 5), (33, 333, 7), (1, 8191, 64), (300, 64, 3)])
def test_logprobs_match_oracle(dtype, M, N, top):
    rng = np.random.default_rng(N)
    z = rng.standard_normal((M, N)) * 3
    z[:, rng.integers(0, N, min(N, 4))] += 9
    t, z = typed(z, dtype)
    tokens = rng.integers(0, N, M)
    check_logprobs(z, tokens, top, B.nvfp4_token_logprobs(t, ints(tokens), top))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N", [5, 1000, 5000])
def test_logprobs_masks_and_rows_without_a_distribution(dtype, N):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((9, N)).astype(np.float32)
    low = torch.finfo(dtype).min
    z[0] = -np.inf
    z[1, N // 2] = np.nan
    z[2, 0] = np.inf
    z[3, 1:] = -np.inf  # one token is left
    z[4, ::2] = -np.inf
    z[5, 1:] = low  # masked by the type's lowest value
    z[6] = low
    z[7] = 1e30 if dtype == FP else 2.0 ** 100
    z[8, :] = 0.0
    z[8, 1::2] = -0.0
    t, z = typed(z, dtype)
    tokens = np.array([0, 0, 0, 0, 1, 2, 3, 4, -1])
    tokens[4] = 0
    got = B.nvfp4_token_logprobs(t, ints(tokens), 5)
    check_logprobs(z, tokens, 5, got)
    assert got[3][0].tolist() == [-1] * 5 and got[0][3] == 0.0 and got[1][3] == 0.0
    assert B.nvfp4_token_logprobs(t, ints(np.full(9, N)), 0)[0].isnan().all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("order", ["up", "down", "equal", "two values", "steps"])
def test_logprobs_orders_and_ties(dtype, order):
    N, top = 20000, 64
    n = np.arange(N, dtype=np.float32)
    z = {"up": n / 1000, "down": -n / 1000, "equal": np.zeros(N), "two values": (n % 7 == 3) * 4.0,
         "steps": np.floor(n / 100) % 13}[order]
    t, z = typed(np.stack([z, z[::-1]]), dtype)
    check_logprobs(z, [5, N - 1], top, B.nvfp4_token_logprobs(t, ints([5, N - 1]), top))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_logprobs_of_a_sure_row_keep_their_digits(dtype):
    z = np.zeros((3, 3000), dtype=np.float32)
    z[0, 100], z[1, 2999], z[2, 0] = 30.0, 60.0, 100.0
    t, z = typed(z, dtype)
    got = B.nvfp4_token_logprobs(t, ints([100, 2999, 0]), 2)
    check_logprobs(z, [100, 2999, 0], 2, got)
    want = -2999 * np.exp(-30.0)  # the other columns
    assert abs(got[0][0].item() - want) < 1e-4 * abs(want)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("first,stride", [(0, 1003), (1, 1003), (3, 1017), (7, 2000)])
def test_logprobs_of_spaced_and_unaligned_rows(dtype, first, stride):
    rng = np.random.default_rng(first)
    base, f = typed(rng.standard_normal((6, stride)), dtype)
    t, z = base.reshape(-1)[first:first + 5 * stride].view(5, stride)[:, :1000], \
        f.reshape(-1)[first:first + 5 * stride].reshape(5, stride)[:, :1000]
    check_logprobs(z, [1, 2, 3, 4, 999], 9, B.nvfp4_token_logprobs(t, ints([1, 2, 3, 4, 999]), 9))


# ----------------------------------------------------------------------------------------------- streams, graphs, steps


def calls():
    """One call of each operator on buffers of its own, as (run, results) pairs."""
    d1, d2, d3 = Delta(BF, 2, 1, 2, 4, 128, 128), Delta(BF, 1, 150, 1, 2, 128, 128), Delta(FP, 2, 23, 1, 2, 64, 64)
    tree = random_trees(np.random.default_rng(0), 2, 23)
    r = Rope(BF, [40, 7], 16, 4, 2, 128, 64, 16, tree=True)
    z, tokens = typed(np.random.default_rng(3).standard_normal((16, 9001)) * 3, FP)[0], ints(np.arange(16))
    made = []
    for d in (d1, d2):
        rows, kw = d.common()
        st, first, s, t = floats(d.states), floats(d.states), ints(d.src), ints(d.dst)
        def run(rows=rows, kw=kw, st=st, first=first, s=s, t=t):
            st.copy_(first)
            return [B.nvfp4_delta_rule(*rows, st, s, t, **kw), st]
        made.append(run)
    rows, kw = d3.common()
    st, s, par = floats(d3.states), ints(d3.src), ints(tree)
    made.append(lambda: list(B.nvfp4_delta_tree(*rows, st, s, par, **kw)))
    pages = [torch.from_numpy(x.copy()).to(DEV) for x in r.start]
    inv, ks, vs, tab, lens, rp = (torch.from_numpy(r.inv).to(DEV), U.scalar(KS), U.scalar(VS), ints(r.table),
                                  ints(r.lens), ints(r.parent))
    made.append(lambda: [B.nvfp4_kv_append_rope(r.q, r.k, r.v, inv, ks, vs, *pages, tab, lens, parent=rp)] + pages)
    made.append(lambda: list(B.nvfp4_token_logprobs(z, tokens, 20)))
    cst, g = floats(d3.states)[None], floats(d3.g)[None]
    keys, updates = B.nvfp4_delta_tree(*rows, st, s, par, **kw)[1:]
    result, dst = ints([[0, 2, 0, 1, 4] + [-1] * 21, [0, 0, 0] + [-1] * 23]), ints(d3.dst)

    def commit():
        B.nvfp4_delta_commit(cst, keys[None], updates[None], g, result, s, dst)
        return [cst]
    made.append(commit)
    return made


def test_two_runs_give_the_same_bits():
    for run in calls():
        first = [x.clone() for x in run()]
        for x, y in zip(first, run()):
            assert torch.equal(x, y)


def test_graphs_replay_to_the_eager_result():
    runs = calls()
    want = [[x.clone() for x in run()] for run in runs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [run() for run in runs]
    other = calls()
    for _ in range(3):
        for outs in got[:-1]:  # the commit's only result holds what it starts from
            outs[0].zero_()
        for run in other:  # eager work between the replays
            run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for outs, ref in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(outs, ref))


def test_calls_on_two_streams_at_once():
    a, b = calls(), calls()
    want = [[x.clone() for x in run()] for run in a]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for i in range(len(a)):
        for s, runs, outs in zip(streams, (a, b), got):
            with torch.cuda.stream(s):
                outs.append([x.clone() for x in runs[i]()])
    torch.cuda.synchronize()
    for outs in got:
        for x, y in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_a_decode_step_of_a_hybrid_model():
    """A tree's nodes through a recurrent layer and an attention layer; the LM head's rows accepted and scored; the
    accepted path put into pages and states; then the next token from there."""
    rng = np.random.default_rng(11)
    M, Hk, H, D, page, Hq, Hkv, N = 12, 2, 4, 64, 16, 4, 2, 512
    n0 = 37
    parent = random_trees(rng, 1, M)
    d = Delta(BF, 1, M, Hk, H, D, D, src=[1], dst=[1], slots=3, seed=12)
    out, keys, updates = run_tree(d, parent)
    check_tree(d, parent, (out, keys, updates))
    # attention layer
    r = Rope(BF, [n0], M, Hq, Hkv, D, 32, page, seed=13)
    r.parent = parent
    W = -(-(n0 + M + 1) // page)
    r.table = np.arange(W, dtype=np.int32)[None] + 1
    r.start = [KV.encode(rng.standard_normal((W + 2, Hkv, page, D)).astype(np.float32), s) for s in (KS, VS)]
    q, pages = r.gpu()
    r.check(q, pages)
    att, lse = B.nvfp4_kv_attention(q, U.scalar(KS), U.scalar(VS), *pages, ints(r.table), ints(r.lens),
                                    parent=ints(parent), want_lse=True)
    k_ref, v_ref = (x.cpu().numpy() for x in pages)
    ref, ref_lse, _ = KC.attention(q.float().cpu().numpy(), k_ref, v_ref, KS, VS, r.table, r.lens, parent)
    assert np.abs(att.float().cpu().numpy() - ref).max() < 2.0 ** -7 * np.abs(ref).max()
    # the rows' logits: the accepted path follows their argmax
    z = rng.standard_normal((M, N)).astype(np.float32)
    greedy = z.argmax(-1).astype(np.int32)
    draft = np.array([0] + [int(greedy[parent[0, v]]) if rng.random() < 0.7 else -1 for v in range(1, M)], np.int32)
    result = B.nvfp4_tree_accept(ints(parent[0]), ints(draft), ints(greedy))[None]
    row = result[0].tolist()
    path = [0] + row[3:3 + row[1]]
    assert (row[0], path[1:], row[2]) == TR.accept(parent[0], draft, greedy)
    lp = B.nvfp4_token_logprobs(floats(z), ints(greedy), 3)
    check_logprobs(z, greedy, 3, lp)
    assert lp[3][:, 0].tolist() == greedy.tolist()
    lens = B.nvfp4_kv_compact(pages[0][None], pages[1][None], ints(r.table), ints(r.lens), result)
    assert lens.tolist() == [n0 + len(path)]
    st = floats(d.states)
    B.nvfp4_delta_commit(st[None], keys[None], updates[None], floats(d.g)[None], result, ints([1]), ints([1]))
    # the chain of the path's tokens leaves the same state
    c = Delta(BF, 1, M, Hk, H, D, D, src=[1], dst=[1], slots=3, seed=12)
    for name in ("q", "k", "v", "qf", "kf", "vf", "g", "beta"):
        setattr(c, name, getattr(c, name)[:, path])
    for name in ("q", "k", "v"):
        setattr(c, name, getattr(c, name).contiguous())
    c.dims = (1, len(path)) + c.dims[2:]
    after, off = c.chain_ref()[2:4]
    err = np.sqrt(((st.double().cpu().numpy() - after) ** 2).sum(-1))
    # the tree's u are off by their bound (as large as a state's), the path's sums by 90 * 2^-23 of what they add up
    assert (err <= 4 * off + 100 * 2.0 ** -23 * np.sqrt((after ** 2).sum(-1) + (c.states ** 2).sum(-1))).all()
    nxt = Delta(BF, 1, 1, Hk, H, D, D, src=[1], dst=[2], slots=3, seed=14)
    nxt.states = st.cpu().numpy()
    nxt.check_chain(*nxt.chain())
