"""Host-side rules of the gated delta rule, the rotary append and the token log probabilities at their ends (CPU only:
sizes, and calls that are refused or empty before any HIP call)."""
import pytest

from nvfp4_w4a4_block_amd import binding as B

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return B.load()


@pytest.mark.parametrize("dt", [B.NVFP4_BF16, B.NVFP4_F32])
@pytest.mark.parametrize("seqs,nodes,key_heads,heads,dk,dv", [
    (64, 200, 16, 48, 128, 128), (80, 130, 16, 48, 128, 128), (300, 130, 1, 16, 256, 256), (4, 2047, 16, 48, 128, 128),
    (1, 65535, 16, 48, 128, 128), (256, 65535, 16, 48, 128, 128), (65535, 256, 1, 1, 64, 64), (3, 4099, 4, 8, 64, 128),
    (40, 1000, 16, 48, 256, 256), (1000, 66, 16, 32, 128, 64)])
def test_prepared_blocks_and_carried_states_stay_within_a_round(lib, seqs, nodes, key_heads, heads, dk, dv, dt):
    """Half the Infinity Cache holds what a round prepares and hands to the next."""
    assert 0 < lib.nvfp4_delta_rule_workspace_bytes(seqs, nodes, key_heads, heads, dk, dv, dt) <= 128 * MB


def test_no_state_is_carried_where_a_sequence_fits(lib):
    """130 tokens are three blocks: what 80 sequences need is a multiple of three blocks of one, without states."""
    size = lambda n, m: lib.nvfp4_delta_rule_workspace_bytes(n, m, 16, 48, 128, 128, B.NVFP4_BF16)  # noqa: E731
    many = size(80, 130)
    state, block = 48 * 128 * 128 * 4, (many // 3) / 1.0
    assert many % 3 == 0 and many < 128 * MB and block % state != 0
    one = size(2, 65)  # two blocks of two sequences, more columns a workgroup
    assert one % 4 == 0 and many % (one // 4) == 0


def test_a_block_of_the_largest_shape_is_the_least(lib):
    """1,024 key and value heads of 256 in fp32: one block is past a round, and is taken nevertheless."""
    one = lib.nvfp4_delta_rule_workspace_bytes(1, 64 + 1, 1024, 1024, 256, 256, B.NVFP4_F32)
    assert 128 * MB < one < 512 * MB and one == lib.nvfp4_delta_rule_workspace_bytes(1, 65535, 1024, 1024, 256, 256, B.NVFP4_F32)


@pytest.mark.parametrize("seqs", [2, 3, 7, 100])
def test_sequences_whose_blocks_and_states_do_not_fit_come_in_turns(lib, seqs):
    assert 0 < lib.nvfp4_delta_rule_workspace_bytes(seqs, 430, 4, 1024, 64, 64, B.NVFP4_F32) <= 128 * MB


# ----------------------------------------------------------------------------------------------- refusals

A = 0x100000  # a fake, aligned address: never dereferenced by a rejected call


def test_commit_with_counts_refuses_as_without(lib):
    ok = dict(L=2, B=2, M=3, Hk=2, H=4, Dk=64, Dv=128, S=5, states=16 * A, keys=A, updates=2 * A, g=3 * A, result=4 * A,
              src=4 * A, dst=4 * A, counts=4 * A, stream=None)
    call = lambda **new: lib.nvfp4_delta_commit_counts(*{**ok, **new}.values())  # noqa: E731
    for bad in (dict(M=0), dict(M=65), dict(L=-1), dict(Hk=3), dict(Dk=96), dict(S=0)):
        assert call(**bad) == B.NVFP4_ERR_SHAPE
    for name in ("states", "keys", "updates", "g", "result", "src", "dst"):
        assert call(**{name: None}) == B.NVFP4_ERR_NULL
        assert call(**{name: ok[name] + 1}) == B.NVFP4_ERR_ALIGN
    assert call(counts=A + 1) == B.NVFP4_ERR_ALIGN
    assert call(B=0) == call(L=0, counts=None) == B.NVFP4_OK
