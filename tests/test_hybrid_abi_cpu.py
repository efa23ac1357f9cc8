"""Host-side refusals of the gated delta rule, the rotary append and the token log probabilities (CPU only: every call
is rejected, or empty, before any HIP call) and of their Python binding."""
import pytest
import torch

from nvfp4_w4a4_block_amd import binding as B

A = 0x100000  # a fake, aligned address: never dereferenced by a rejected call


@pytest.fixture(scope="module")
def lib():
    return B.load()


def changed(args, **new):
    args = dict(args)
    for name in new:
        assert name in args
    args.update(new)
    return list(args.values())


ROWS = dict(q=A, k=A, v=A, dt=B.NVFP4_BF16, qs=128, ks=128, vs=512, g=A, beta=A, scale=0.125, eps=1e-6)
RULE = dict(B=2, M=3, Hk=2, H=4, Dk=64, Dv=128, S=5, **ROWS, states=A, src=A, dst=A, counts=None, out=16 * A, ws=None,
            wsb=0, stream=None)
TREE = dict(B=2, M=3, Hk=2, H=4, Dk=64, Dv=128, S=5, **ROWS, states=A, src=A, parent=A, counts=None, out=16 * A,
            keys=A, updates=A, stream=None)
COMMIT = dict(L=2, B=2, M=3, Hk=2, H=4, Dk=64, Dv=128, S=5, states=A, keys=A, updates=A, g=A, result=A, src=A, dst=A,
              stream=None)
ROPE = dict(B=2, M=3, Hq=8, H=4, D=64, R=32, page=16, P=8, W=5, q=A, k=A, v=A, dt=B.NVFP4_BF16, qs=512, ks=256, vs=256,
            inv=A, rope=1.0, inter=0, k_scale=A, v_scale=A, kp=A, vp=2 * A, stride=4 * 16 * 64, table=A, lens=A,
            parent=A, counts=None, q_out=16 * A, stream=None)
PROBS = dict(M=3, N=1000, top=5, logits=A, dt=B.NVFP4_BF16, stride=1000, tokens=A, lp=A, ent=A, best=A, ids=A, ws=A,
             wsb=1 << 20, stream=None)
NAN, INF = float("nan"), float("inf")
SHAPES = [dict(B=-1), dict(B=65536), dict(M=-1), dict(Hk=0), dict(Hk=3), dict(H=0), dict(H=1026, Hk=1), dict(Dk=96),
          dict(Dv=32), dict(Dk=512), dict(S=0), dict(S=1 << 31)]
VALUES = [dict(qs=127), dict(ks=64), dict(vs=504), dict(vs=516), dict(qs=1 << 31), dict(scale=NAN), dict(scale=INF),
          dict(eps=NAN), dict(eps=INF)]


@pytest.mark.parametrize("bad", SHAPES + VALUES + [dict(M=65536), dict(B=4096, M=8192), dict(wsb=-1), dict(out=A),
                                                   dict(out=A + 1280), dict(v=16 * A + 2048 * 2)])
def test_rule_refuses_shapes(lib, bad):
    assert lib.nvfp4_delta_rule(*changed(RULE, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", SHAPES + VALUES + [dict(M=65), dict(out=A)])
def test_tree_refuses_shapes(lib, bad):
    assert lib.nvfp4_delta_tree(*changed(TREE, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(states=16 * A + 4000), dict(states=16 * A - 4 * 5 * 4 * 64 * 128 + 16)])
def test_rule_refuses_outputs_in_the_states(lib, bad):
    assert lib.nvfp4_delta_rule(*changed(RULE, **bad)) == B.NVFP4_ERR_SHAPE
    assert lib.nvfp4_delta_tree(*changed(TREE, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("name", ["q", "k", "v", "states", "out", "updates"])
def test_tree_refuses_outputs_that_share_bytes(lib, name):
    apart = changed(TREE, q=A, k=2 * A, v=3 * A, states=8 * A, out=4 * A, keys=5 * A, updates=6 * A)
    apart = dict(zip(TREE, apart))
    assert lib.nvfp4_delta_tree(*changed(apart, keys=apart[name] + 16)) == B.NVFP4_ERR_SHAPE
    other = "keys" if name == "updates" else name
    assert lib.nvfp4_delta_tree(*changed(apart, updates=apart[other] + 16)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", SHAPES + [dict(M=0), dict(M=65), dict(L=-1), dict(L=4097)])
def test_commit_refuses_shapes(lib, bad):
    assert lib.nvfp4_delta_commit(*changed(COMMIT, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(M=-1), dict(M=65), dict(H=0), dict(Hq=0), dict(D=96), dict(R=0), dict(R=8), dict(R=40),
    dict(R=80), dict(page=8), dict(page=24), dict(page=2048), dict(P=0), dict(W=0), dict(W=1 << 27), dict(stride=4080),
    dict(stride=4 * 16 * 64 + 8), dict(qs=504), dict(ks=255), dict(vs=260), dict(rope=NAN), dict(rope=-INF),
    dict(vp=A), dict(q_out=A), dict(q_out=A + 6000), dict(q=16 * A, qs=520), dict(parent=None, B=4096, M=8192)])
def test_rope_refuses_shapes(lib, bad):
    assert lib.nvfp4_kv_append_rope(*changed(ROPE, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(M=-1), dict(M=65536), dict(N=0), dict(N=1 << 24), dict(top=-1), dict(top=65),
                                 dict(top=6, N=5, stride=5), dict(stride=999), dict(stride=1 << 31), dict(wsb=8)])
def test_logprobs_refuses_shapes(lib, bad):
    assert lib.nvfp4_token_logprobs(*changed(PROBS, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("call,args,optional", [
    ("nvfp4_delta_rule", RULE, ("counts", "ws")), ("nvfp4_delta_tree", TREE, ("counts",)),
    ("nvfp4_delta_commit", COMMIT, ()), ("nvfp4_kv_append_rope", ROPE, ("parent", "counts")),
    ("nvfp4_token_logprobs", PROBS, ())])
def test_null_and_misaligned_pointers(lib, call, args, optional):
    for name, value in args.items():
        if not isinstance(value, int) or value < A or name == "wsb":
            continue
        if name not in optional:
            assert getattr(lib, call)(*changed(args, **{name: None})) == B.NVFP4_ERR_NULL, name
        assert getattr(lib, call)(*changed(args, **{name: value + 1})) == B.NVFP4_ERR_ALIGN, name


def test_alignment_of_a_value(lib):
    for name in ("q", "k", "v", "out", "states"):
        assert lib.nvfp4_delta_rule(*changed(RULE, **{name: 32 * A + 8})) == B.NVFP4_ERR_ALIGN, name
    assert lib.nvfp4_kv_append_rope(*changed(ROPE, inv=A + 4)) == B.NVFP4_ERR_ALIGN
    assert lib.nvfp4_token_logprobs(*changed(PROBS, logits=A + 1)) == B.NVFP4_ERR_ALIGN
    assert lib.nvfp4_token_logprobs(*changed(PROBS, logits=A + 2, dt=B.NVFP4_F32)) == B.NVFP4_ERR_ALIGN


def test_dtypes_and_workspaces(lib):
    assert lib.nvfp4_delta_rule(*changed(RULE, dt=2)) == B.NVFP4_ERR_DTYPE
    assert lib.nvfp4_delta_tree(*changed(TREE, dt=-1)) == B.NVFP4_ERR_DTYPE
    assert lib.nvfp4_kv_append_rope(*changed(ROPE, dt=7)) == B.NVFP4_ERR_DTYPE
    assert lib.nvfp4_token_logprobs(*changed(PROBS, dt=3)) == B.NVFP4_ERR_DTYPE
    assert lib.nvfp4_delta_rule(*changed(RULE, wsb=64)) == B.NVFP4_ERR_NULL
    assert lib.nvfp4_delta_rule(*changed(RULE, ws=A + 8, wsb=64)) == B.NVFP4_ERR_ALIGN
    size = lib.nvfp4_delta_rule_workspace_bytes
    assert size(0, 512, 2, 4, 64, 64, B.NVFP4_BF16) == size(1, 512, 3, 4, 64, 64, B.NVFP4_BF16) == 0
    assert size(1, 512, 2, 4, 64, 64, 5) == size(1, 512, 2, 4, 64, 65, B.NVFP4_BF16) == 0
    size = lib.nvfp4_token_logprobs_workspace_bytes
    assert size(0, 10, 1, B.NVFP4_F32) == size(1, 10, 11, B.NVFP4_F32) == size(1, 10, 1, 9) == 0
    assert size(2, 1000, 5, B.NVFP4_F32) > 0 and size(2, 1000, 5, B.NVFP4_F32) % 8 == 0


def test_empty_calls_need_no_pointers(lib):
    none = {n: None for n in ("q", "k", "v", "g", "beta", "states", "src", "dst", "out")}
    assert lib.nvfp4_delta_rule(*changed(RULE, B=0, **none)) == B.NVFP4_OK
    none = {n: None for n in ("q", "k", "v", "g", "beta", "states", "src", "parent", "out", "keys", "updates")}
    assert lib.nvfp4_delta_tree(*changed(TREE, B=0, **none)) == B.NVFP4_OK
    assert lib.nvfp4_delta_tree(*changed(TREE, M=0, **none)) == B.NVFP4_OK
    none = {n: None for n in ("states", "keys", "updates", "g", "result", "src", "dst")}
    assert lib.nvfp4_delta_commit(*changed(COMMIT, B=0, **none)) == B.NVFP4_OK
    assert lib.nvfp4_delta_commit(*changed(COMMIT, L=0, **none)) == B.NVFP4_OK
    none = {n: None for n in ("q", "k", "v", "inv", "kp", "vp", "table", "lens", "q_out", "k_scale", "v_scale")}
    assert lib.nvfp4_kv_append_rope(*changed(ROPE, B=0, **none)) == B.NVFP4_OK
    assert lib.nvfp4_kv_append_rope(*changed(ROPE, M=0, **none)) == B.NVFP4_OK
    none = {n: None for n in ("logits", "tokens", "lp", "ent", "best", "ids", "ws")}
    assert lib.nvfp4_token_logprobs(*changed(PROBS, M=0, **none)) == B.NVFP4_OK


def test_binding_refuses_cpu_tensors():
    f, i = torch.zeros, torch.zeros((1,), dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        B.nvfp4_delta_rule(f(1, 1, 1, 64), f(1, 1, 1, 64), f(1, 1, 1, 64), f(1, 1, 1), f(1, 1, 1), f(1, 1, 64, 64), i, i)
    with pytest.raises(ValueError, match="on a GPU"):
        B.nvfp4_delta_tree(f(1, 1, 1, 64), f(1, 1, 1, 64), f(1, 1, 1, 64), f(1, 1, 1), f(1, 1, 1), f(1, 1, 64, 64), i,
                           i[None])
    with pytest.raises(ValueError, match="on a GPU"):
        B.nvfp4_delta_commit(f(1, 1, 1, 64, 64), f(1, 1, 1, 1, 64), f(1, 1, 1, 1, 64), f(1, 1, 1, 1), i[None], i, i)
    with pytest.raises(ValueError, match="on one GPU"):
        pages = torch.zeros((4, 1, 16, 64), dtype=torch.uint8)
        B.nvfp4_kv_append_rope(f(1, 1, 1, 64), f(1, 1, 1, 64), f(1, 1, 1, 64), f(32).double(), f(1), f(1), pages, pages,
                               i[None], i)
    with pytest.raises(ValueError, match="on a GPU"):
        B.nvfp4_token_logprobs(f(1, 10), i, 2)
