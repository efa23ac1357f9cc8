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


# Arrays a megabyte or more apart, every size below that.
FAR = 1 << 28


def places(*names):
    return {name: FAR * (i + 1) for i, name in enumerate(names)}


RULE = dict(B=2, M=70, Hk=2, H=4, Dk=64, Dv=128, S=5, **places("q", "k", "v"), dt=B.NVFP4_BF16, qs=128, ks=128, vs=512,
            g=8 * FAR, beta=9 * FAR, scale=0.125, eps=1e-6, states=10 * FAR, src=11 * FAR, dst=12 * FAR, counts=13 * FAR,
            out=14 * FAR, ws=15 * FAR, wsb=1 << 24, stream=None)
TREE = dict(B=2, M=3, Hk=2, H=4, Dk=64, Dv=128, S=5, **places("q", "k", "v"), dt=B.NVFP4_BF16, qs=128, ks=128, vs=512,
            g=8 * FAR, beta=9 * FAR, scale=0.125, eps=1e-6, states=10 * FAR, src=11 * FAR, parent=12 * FAR,
            counts=13 * FAR, out=14 * FAR, keys=15 * FAR, updates=16 * FAR, stream=None)
COMMIT = dict(L=2, B=2, M=3, Hk=2, H=4, Dk=64, Dv=128, S=5, states=FAR, keys=2 * FAR, updates=3 * FAR, g=4 * FAR,
              result=5 * FAR, src=6 * FAR, dst=7 * FAR, counts=8 * FAR, stream=None)
ROPE = dict(B=2, M=3, Hq=8, H=4, D=64, R=32, page=16, P=8, W=5, **places("q", "k", "v"), dt=B.NVFP4_BF16, qs=520,
            ks=256, vs=256, inv=8 * FAR, rope=1.0, inter=0, k_scale=9 * FAR, v_scale=10 * FAR, kp=11 * FAR, vp=12 * FAR,
            stride=4 * 16 * 64, table=13 * FAR, lens=14 * FAR, parent=15 * FAR, counts=16 * FAR, q_out=17 * FAR,
            stream=None)
PROBS = dict(M=3, N=1000, top=5, logits=FAR, dt=B.NVFP4_BF16, stride=1000, tokens=2 * FAR, lp=3 * FAR, ent=4 * FAR,
             best=5 * FAR, ids=6 * FAR, ws=7 * FAR, wsb=1 << 20, stream=None)
CALLS = [("nvfp4_delta_rule", RULE, ("out", "ws"), ("q", "k", "v", "g", "beta", "states", "src", "dst", "counts")),
         ("nvfp4_delta_tree", TREE, ("out", "keys", "updates"),
          ("q", "k", "v", "g", "beta", "states", "src", "parent", "counts")),
         ("nvfp4_delta_commit_counts", COMMIT, ("states",), ("keys", "updates", "g", "result", "src", "dst", "counts")),
         ("nvfp4_kv_append_rope", ROPE, ("q_out",),
          ("q", "k", "v", "inv", "k_scale", "v_scale", "kp", "vp", "table", "lens", "parent", "counts")),
         ("nvfp4_token_logprobs", PROBS, ("lp", "ent", "best", "ids", "ws"), ("logits", "tokens"))]


@pytest.mark.parametrize("call,args,outs,others", CALLS)
def test_outputs_that_share_bytes_with_another_array(lib, call, args, outs, others):
    for out in outs:
        for other in others + tuple(o for o in outs if o != out):
            # its first bytes are the other's first ones; the other's are its first ones
            for moved, at in ((out, args[other]), (other, args[out])):
                assert getattr(lib, call)(*{**args, moved: at}.values()) == B.NVFP4_ERR_SHAPE, (out, other)


def test_an_output_that_ends_in_another_array(lib):
    """The last 16 bytes of each are the first of another's."""
    sizes = [("nvfp4_delta_rule", RULE, "out", 2 * 70 * 512 * 2, "beta"), ("nvfp4_delta_rule", RULE, "g", 2 * 70 * 16, "out"),
             ("nvfp4_delta_rule", RULE, "ws", 1 << 24, "states"), ("nvfp4_delta_tree", TREE, "updates", 6 * 512 * 4, "g"),
             ("nvfp4_delta_tree", TREE, "beta", 6 * 16, "keys"), ("nvfp4_delta_commit_counts", COMMIT, "g", 2 * 6 * 16, "states"),
             ("nvfp4_delta_commit_counts", COMMIT, "states", 2 * 5 * 4 * 64 * 128 * 4, "updates"),
             ("nvfp4_kv_append_rope", ROPE, "vp", 8 * 4096, "q_out"), ("nvfp4_kv_append_rope", ROPE, "q_out", 6 * 1024, "kp"),
             ("nvfp4_token_logprobs", PROBS, "logits", 6000 // 16 * 16, "best")]
    for call, args, name, size, other in sizes:
        assert getattr(lib, call)(*{**args, name: args[other] - size + 16}.values()) == B.NVFP4_ERR_SHAPE, (call, name)


def test_states_of_the_largest_counts_are_compared_as_they_are(lib):
    """Their bytes do not fit 64 bits: an array behind them shares theirs."""
    many = dict(L=4096, H=1024, Hk=1, Dk=256, Dv=256, S=(1 << 31) - 1, B=1, M=1)
    assert lib.nvfp4_delta_commit_counts(*{**COMMIT, **many}.values()) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(base=x) for x in (float("nan"), float("inf"))] +
                         [dict(factor=x, scaling=s) for x in (float("nan"), float("inf")) for s in ("linear", "ntk", "yarn")] +
                         [dict(trained=float("nan"), scaling="yarn"), dict(trained=float("inf"), scaling="yarn"),
                          dict(fast=float("inf"), scaling="yarn"), dict(slow=float("nan"), scaling="yarn")])
def test_frequencies_of_numbers_that_are_not_finite(bad):
    with pytest.raises(ValueError):
        B.rope_frequencies(32, **bad)
