"""Host-side refusals of the paged KV-cache entry points (CPU only: every call is rejected, or
empty, before any HIP call) and of their Python binding."""
import ctypes

import pytest
import torch

from nvfp4_w4a4_block_amd import binding as B

A = 0x10000  # a fake, aligned address: never dereferenced by a rejected call


@pytest.fixture(scope="module")
def lib():
    return B.load()


def changed(args, **new):
    args = dict(args)
    for name in new:
        assert name in args
    args.update(new)
    return list(args.values())


APPEND = dict(B=2, M=3, H=4, D=64, page=16, P=8, W=5, k=A, v=A, dt=B.NVFP4_BF16, ks=256, vs=256, k_scale=A, v_scale=A,
              kp=A, vp=A, stride=4 * 16 * 64, table=A, lens=A, counts=None, stream=None)
ATTEND = dict(B=2, M=3, Hq=8, H=4, D=64, page=16, P=8, W=5, q=16 * A, dt=B.NVFP4_BF16, qs=512, sm=0.125, k_scale=A,
              v_scale=A, kp=A, vp=A, stride=4 * 16 * 64, table=A, lens=A, parent=A, counts=None, out=A, lse=A, ws=None,
              wsb=0, stream=None)
COMPACT = dict(L=2, B=2, M=3, H=4, D=64, page=16, P=8, W=5, kp=A, vp=A, layer=8 * 4096, stride=4096, table=A, lens=A,
               result=A, new=A + 64, stream=None)
RESIZE = dict(n=2, S=3, W=5, P=8, page=16, table=A, held=A, refs=A, free=A, seqs=A, tokens=A, short=A, stream=None)
FORK = dict(n=2, S=3, W=5, P=8, page=16, table=A, held=A, refs=A, free=A, src=A, dst=A, tokens=A, short=A, moves=A,
            L=2, H=4, D=64, kp=A, vp=A, layer=8 * 4096, stride=4096, stream=None)

SHAPES = [dict(H=0), dict(D=96), dict(D=512), dict(page=8), dict(page=24), dict(page=2048), dict(P=0),
          dict(P=1 << 31), dict(W=0), dict(W=1 << 27), dict(stride=4 * 16 * 64 - 16), dict(stride=4 * 16 * 64 + 8),
          dict(stride=1 << 31)]


@pytest.mark.parametrize("bad", SHAPES + [dict(B=-1), dict(B=65536), dict(M=-1), dict(M=65536), dict(ks=255),
                                          dict(vs=248), dict(ks=260), dict(B=4096, M=8192), dict(H=1025)])
def test_append_refuses_shapes(lib, bad):
    assert lib.nvfp4_kv_append(*changed(APPEND, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", SHAPES + [dict(B=-1), dict(M=65), dict(Hq=6), dict(Hq=0), dict(Hq=4 * 257, qs=4 * 257 * 64), dict(qs=504), dict(qs=516),
                                          dict(sm=float("inf")), dict(sm=float("nan")), dict(wsb=-1), dict(out=16 * A), dict(out=16 * A + 6000), dict(q=A),
                                          dict(B=65535, H=1024, Hq=1024, M=1, qs=65536, stride=1 << 20),
                                          dict(parent=None, B=4096, M=8192)])
def test_attention_refuses_shapes(lib, bad):
    assert lib.nvfp4_kv_attention(*changed(ATTEND, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", SHAPES + [dict(L=0), dict(L=4097), dict(B=-1), dict(M=0), dict(M=65), dict(layer=-16),
                                          dict(layer=8), dict(B=4096, L=4096, H=1), dict(new=A), dict(new=A + 4), dict(new=A - 4)])
def test_compact_refuses_shapes(lib, bad):
    assert lib.nvfp4_kv_compact(*changed(COMPACT, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n=1025), dict(S=0), dict(W=0), dict(P=0), dict(page=0), dict(page=17),
                                 dict(S=65536), dict(S=60000, W=10000)])
def test_pool_refuses_shapes(lib, bad):
    assert lib.nvfp4_kv_resize(*changed(RESIZE, **bad)) == B.NVFP4_ERR_SHAPE
    assert lib.nvfp4_kv_fork(*changed(FORK, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(H=0), dict(D=65), dict(stride=4080), dict(layer=8), dict(L=-1)])
def test_fork_refuses_pages(lib, bad):
    assert lib.nvfp4_kv_fork(*changed(FORK, **bad)) == B.NVFP4_ERR_SHAPE


@pytest.mark.parametrize("call,args,optional", [
    ("nvfp4_kv_append", APPEND, ("counts",)), ("nvfp4_kv_attention", ATTEND, ("parent", "counts", "lse", "ws")),
    ("nvfp4_kv_compact", COMPACT, ()), ("nvfp4_kv_resize", RESIZE, ()), ("nvfp4_kv_fork", FORK, ())])
def test_null_and_misaligned_pointers(lib, call, args, optional):
    for name, value in args.items():
        if not isinstance(value, int) or value < A or name in ("layer", "stride"):
            continue
        if name not in optional:
            assert getattr(lib, call)(*changed(args, **{name: None})) == B.NVFP4_ERR_NULL, name
        assert getattr(lib, call)(*changed(args, **{name: value + 2})) == B.NVFP4_ERR_ALIGN, name


@pytest.mark.parametrize("call,args", [("nvfp4_kv_compact", COMPACT), ("nvfp4_kv_fork", FORK)])
def test_layers_that_overlap_are_refused(lib, call, args):
    for bad in (dict(layer=0), dict(layer=4096), dict(layer=8 * 4096 - 16), dict(layer=4096, stride=2 * 4096 - 16),
                dict(layer=4080, stride=3 * 4096)):
        assert getattr(lib, call)(*changed(args, **bad)) == B.NVFP4_ERR_SHAPE, bad
    for good in (dict(layer=8 * 4096 - 4096), dict(layer=4096, stride=2 * 4096), dict(layer=2 * 4096, stride=3 * 4096),
                 dict(L=1, layer=0)):  # past the shapes: the missing table is what is refused
        if good.get("layer") == 7 * 4096:
            good["P"] = 7
        assert getattr(lib, call)(*changed(args, **good, table=None)) == B.NVFP4_ERR_NULL, good


def test_one_array_for_keys_and_values_is_not_written(lib):
    assert lib.nvfp4_kv_append(*changed(APPEND, v=A + 64)) == B.NVFP4_ERR_SHAPE
    assert lib.nvfp4_kv_compact(*changed(COMPACT)) == B.NVFP4_ERR_SHAPE


def test_dtypes_and_workspace(lib):
    assert lib.nvfp4_kv_append(*changed(APPEND, dt=2)) == B.NVFP4_ERR_DTYPE
    assert lib.nvfp4_kv_attention(*changed(ATTEND, dt=-1)) == B.NVFP4_ERR_DTYPE
    assert lib.nvfp4_kv_attention(*changed(ATTEND, wsb=64)) == B.NVFP4_ERR_NULL
    assert lib.nvfp4_kv_attention(*changed(ATTEND, ws=A + 8, wsb=64)) == B.NVFP4_ERR_ALIGN
    assert lib.nvfp4_kv_attention_workspace_bytes(2, 3, 7, 4, 64, 16, 5, B.NVFP4_BF16) == 0
    assert lib.nvfp4_kv_attention_workspace_bytes(0, 3, 8, 4, 64, 16, 5, B.NVFP4_BF16) == 0


def test_empty_calls_need_no_pointers(lib):
    none = {n: None for n in ("k", "v", "k_scale", "v_scale", "kp", "vp", "table", "lens")}
    assert lib.nvfp4_kv_append(*changed(APPEND, B=0, **none)) == B.NVFP4_OK
    assert lib.nvfp4_kv_append(*changed(APPEND, M=0, **none)) == B.NVFP4_OK
    none = {n: None for n in ("q", "k_scale", "v_scale", "kp", "vp", "table", "lens", "out", "lse", "parent")}
    assert lib.nvfp4_kv_attention(*changed(ATTEND, B=0, **none)) == B.NVFP4_OK
    none = {n: None for n in ("kp", "vp", "table", "lens", "result", "new")}
    assert lib.nvfp4_kv_compact(*changed(COMPACT, B=0, **none)) == B.NVFP4_OK


def test_binding_refuses_cpu_tensors_and_wrong_types():
    pages = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    ints = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="one GPU"):
        B.nvfp4_kv_append(torch.zeros(1, 1, 2, 64), torch.zeros(1, 1, 2, 64), torch.ones(1), torch.ones(1), pages,
                          pages, ints, ints[0, :1])
    with pytest.raises(ValueError, match="one GPU"):
        B.nvfp4_kv_attention(torch.zeros(1, 1, 2, 64), torch.ones(1), torch.ones(1), pages.float(), pages, ints,
                             ints[0, :1])
    with pytest.raises(ValueError, match="one GPU"):
        B.nvfp4_kv_compact(pages[None], pages[None], ints, ints[0, :1], ints)
    pool = B.kv_pool(3, 2, 4, "cpu")
    assert [tuple(t.shape) for t in pool] == [(3, 2), (3,), (4,), (5,)] and pool[3].tolist() == [4, 3, 2, 1, 0]
    with pytest.raises(ValueError, match="on a GPU"):
        B.nvfp4_kv_resize(*pool, 16, ints[0], ints[0])
    with pytest.raises(ValueError, match="on a GPU"):
        B.nvfp4_kv_fork(*pool, pages[None], pages[None], ints[0], ints[0], ints[0])
