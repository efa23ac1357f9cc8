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
