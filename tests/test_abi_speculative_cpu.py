"""Host checks of the speculative-decoding calls: bad sizes, nulls, alignment and overlaps are refused
before the device is touched, in the C ABI and in the Python binding."""
import ctypes

import pytest
import torch

import fp8_blockwise_w8a8_b200 as fq
from fp8_blockwise_w8a8_b200 import _lib, build

FAKE = 1 << 20          # a 16-byte aligned non-null address; never dereferenced on these paths
MB = 1 << 20
SHAPE, ARG, ALIGN, NULL, OK = (_lib.FP8Q_ERR_SHAPE, _lib.FP8Q_ERR_ARG, _lib.FP8Q_ERR_ALIGN,
                               _lib.FP8Q_ERR_NULL, _lib.FP8Q_OK)


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def _no_device(status):
    """What valid arguments give: without a GPU, FP8Q_ERR_ARCH."""
    if not torch.cuda.is_available():
        assert status() == _lib.FP8Q_ERR_ARCH


def test_paged_batch_tables(L):
    ok = dict(ctx=FAKE, new=FAKE + MB, B=8, bs=16, bt=FAKE + 2 * MB, maxb=4, fb=FAKE + 3 * MB, nf=9,
              fc=FAKE + 4 * MB, fl=FAKE + 5 * MB, mt=64, cu=FAKE + 6 * MB, sl=FAKE + 7 * MB,
              slots=FAKE + 8 * MB, pos=FAKE + 9 * MB)

    def call(**kw):
        a = dict(ok, **kw)
        return L.fp8q_paged_batch_tables(*(a[k] for k in ok), None)
    for kw in (dict(B=-1), dict(B=16385), dict(bs=0), dict(maxb=-1), dict(maxb=2 ** 28), dict(nf=-1),
               dict(mt=-1), dict(mt=2 ** 31), dict(nf=2 ** 31)):
        assert call(**kw) == SHAPE, kw
    for name in ("ctx", "new", "bt", "fb", "fc", "fl", "cu", "sl", "slots", "pos"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ok[name] + 2}) == ALIGN, name
    assert call(slots=ok["slots"] + 4) == ALIGN
    for kw in (dict(fl=ok["fc"]), dict(sl=ok["ctx"]), dict(sl=ok["new"]), dict(cu=ok["ctx"] + 28),
               dict(sl=ok["ctx"] - 28), dict(fl=ok["new"] + 4)):
        assert call(**kw) == ARG, kw
    _no_device(call)
    _no_device(lambda: call(B=0, ctx=None, new=None, sl=None, bt=None))
    _no_device(lambda: call(sl=ok["ctx"] + 32))                   # adjacent is not overlapping


def test_tree_mask(L):
    ok = dict(par=FAKE, cu=FAKE, ctx=FAKE, B=2, total=100, maxn=65, mask=FAKE, ldm=2, pos=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return L.fp8q_tree_mask(*(a[k] for k in ok), None)
    for kw in (dict(B=-1), dict(total=-1), dict(maxn=1025, ldm=99), dict(maxn=-1), dict(ldm=1)):
        assert call(**kw) == SHAPE, kw
    for name in ("par", "cu", "mask"):
        assert call(**{name: None}) == NULL, name
    for kw in (dict(par=FAKE + 2), dict(cu=FAKE + 2), dict(ctx=FAKE + 2), dict(mask=FAKE + 4),
               dict(pos=FAKE + 4)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(B=0), dict(total=0), dict(maxn=0)):
        assert call(par=None, cu=None, mask=None, **kw) == OK
    _no_device(call)
    _no_device(lambda: call(ctx=None, pos=None))


def test_tree_mask_batch_limit(L):
    call = lambda B: L.fp8q_tree_mask(FAKE, FAKE, None, B, 100, 64, FAKE, 1, None, None)
    assert call(65536) == SHAPE
    _no_device(lambda: call(65535))


def test_attention_tree(L):
    q = L.fp8q_attention_tree_workspace_bytes
    b = ctypes.c_int64(-1)
    for args in ((2, 8, 2, 96, 16, 300), (2, 9, 2, 128, 16, 300), (2, 258, 2, 128, 16, 300),
                 (65536, 8, 2, 128, 16, 300), (2, 8, 2, 128, 1025, 300), (2, 8, 0, 128, 16, 300),
                 (2, 8, 2, 128, 16, -1), (-1, 8, 2, 128, 16, 300)):
        assert q(*args, ctypes.byref(b)) == SHAPE, args
    assert q(2, 8, 2, 128, 16, 300, None) == NULL
    assert q(2, 8, 2, 128, 16, 300, ctypes.byref(b)) == OK and b.value > 0
    ok = dict(q=FAKE, ldq=1024, k=FAKE, v=FAKE, slots=64, s3=FAKE, bt=FAKE, maxb=4, ctx=FAKE,
              cu=FAKE, mask=FAKE, ldm=1, B=2, total=8, Hq=8, Hkv=2, D=128, bs=16, maxn=16,
              maxlen=64, sm=0.088, out=FAKE, ldo=1024, ws=FAKE, wsb=1 << 40)

    def call(**kw):
        a = dict(ok, **kw)
        return L.fp8q_attention_tree(*(a[k] for k in ok), None)
    for kw in (dict(D=32), dict(D=256), dict(Hq=7), dict(maxlen=65), dict(ldq=1008), dict(ldo=1016),
               dict(ldm=0), dict(maxn=65), dict(maxn=1025, ldm=17), dict(slots=2 ** 31),
               dict(total=-1), dict(bs=0), dict(B=65536), dict(wsb=15), dict(maxb=-1)):
        assert call(**kw) == SHAPE, kw
    for name in ("q", "k", "v", "s3", "bt", "ctx", "cu", "out", "ws"):
        assert call(**{name: None}) == NULL, name
    for kw in (dict(q=FAKE + 8), dict(ldq=1032), dict(k=FAKE + 8), dict(v=FAKE + 8),
               dict(out=FAKE + 8), dict(ldo=1028), dict(mask=FAKE + 4), dict(ctx=FAKE + 2),
               dict(cu=FAKE + 1), dict(bt=FAKE + 2), dict(s3=FAKE + 2), dict(ws=FAKE + 8)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(B=0), dict(total=0), dict(maxn=0)):
        assert call(q=None, out=None, ws=None, **kw) == OK
    _no_device(call)
    _no_device(lambda: call(mask=None, ldm=0))


def test_kv_cache_accept(L):
    ok = dict(k=FAKE, v=FAKE, slots=64, layers=3, stride=64 * 256, row=256, bt=FAKE + MB, maxb=4,
              bs=16, ctx=FAKE + 2 * MB, cu=FAKE + 3 * MB, path=FAKE + 4 * MB, maxp=5,
              plen=FAKE + 5 * MB, B=4, out=FAKE + 6 * MB)

    def call(**kw):
        a = dict(ok, **kw)
        return L.fp8q_kv_cache_accept(*(a[k] for k in ok), None)
    for kw in (dict(row=24), dict(row=0), dict(stride=64 * 256 - 16), dict(layers=65536),
               dict(maxp=1025), dict(bs=0), dict(maxb=2 ** 28), dict(B=-1), dict(slots=-1),
               dict(slots=2 ** 31)):
        assert call(**kw) == SHAPE, kw
    for name in ("k", "v", "bt", "ctx", "cu", "path", "plen", "out"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ok[name] + 2}) == ALIGN, name
    assert call(stride=64 * 256 + 8) == ALIGN
    for name in ("ctx", "cu", "path", "plen", "bt"):
        assert call(out=ok[name] + 4) == ARG, name
    assert call(B=0, k=None, ctx=None) == OK and call(layers=0, k=None) == OK
    _no_device(call)


def test_binding_refuses_other_types_shapes_and_devices():
    i32 = dict(dtype=torch.int32)
    z = torch.zeros
    ctx, cu, table = z(2, **i32), z(3, **i32), z((2, 4), **i32)
    with pytest.raises(ValueError, match="CUDA"):                 # tensors of the host
        fq.paged_batch_tables(ctx, ctx, table, z(9, **i32), z(1, **i32), 16, 8)
    with pytest.raises(ValueError, match="new_lens"):
        fq.paged_batch_tables(ctx, z(2, dtype=torch.int64), table, z(9, **i32), z(1, **i32), 16, 8)
    with pytest.raises(ValueError, match="block_table"):
        fq.paged_batch_tables(ctx, ctx, z((2, 8), **i32)[:, ::2], z(9, **i32), z(1, **i32), 16, 8)
    with pytest.raises(ValueError, match="cu_nodes"):
        fq.tree_mask(z(5, **i32), z(3), 4)
    with pytest.raises(ValueError, match="ctx_lens"):
        fq.tree_mask(z(5, **i32), cu, 4, ctx_lens=z(3, **i32))
    k = z((64, 256), dtype=torch.uint8)
    s3, q = z(3), z((5, 1024), dtype=torch.uint8)
    mask = z((5, 1), dtype=torch.int64)
    with pytest.raises(ValueError, match="v_cache"):
        fq.attention_tree(q, k, k[:32], s3, table, ctx, cu, mask, 8, 2, 16, 4, 64)
    with pytest.raises(ValueError, match="q_codes"):
        fq.attention_tree(q[:, :512], k, k, s3, table, ctx, cu, mask, 8, 2, 16, 4, 64)
    with pytest.raises(ValueError, match="mask"):
        fq.attention_tree(q, k, k, s3, table, ctx, cu, mask[:4], 8, 2, 16, 4, 64)
    with pytest.raises(ValueError, match="mask"):
        fq.attention_tree(q, k, k, s3, table, ctx, cu, mask, 8, 2, 16, 65, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fq.attention_tree(q, k, k, s3, table, ctx, cu, mask, 8, 2, 16, 4, 64)
    with pytest.raises(ValueError, match="path_lens"):
        fq.kv_cache_accept(k, k, table, ctx, cu, z((2, 3), **i32), z(3, **i32), 16)
    with pytest.raises(ValueError, match="v_cache"):
        fq.kv_cache_accept(k, k.view(1, 64, 256), table, ctx, cu, z((2, 3), **i32), ctx, 16)


def test_paged_batch_tables_held(L):
    ok = dict(ctx=FAKE, new=FAKE + MB, B=8, bs=16, bt=FAKE + 2 * MB, maxb=4, fb=FAKE + 3 * MB, nf=9,
              fc=FAKE + 4 * MB, fl=FAKE + 5 * MB, held=FAKE + 10 * MB, hout=FAKE + 11 * MB, mt=64,
              cu=FAKE + 6 * MB, sl=FAKE + 7 * MB, slots=FAKE + 8 * MB, pos=FAKE + 9 * MB)

    def call(**kw):
        a = dict(ok, **kw)
        return L.fp8q_paged_batch_tables_held(*(a[k] for k in ok), None)
    for name in ("held", "hout"):                                 # one without the other
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ok[name] + 2}) == ALIGN, name
    for kw in (dict(hout=ok["held"]), dict(hout=ok["held"] + 28), dict(hout=ok["ctx"]),
               dict(hout=ok["fc"] - 4), dict(sl=ok["held"] + 4), dict(fl=ok["held"]),
               dict(cu=ok["held"] - 32)):
        assert call(**kw) == ARG, kw
    assert call(B=-1) == SHAPE
    _no_device(call)
    _no_device(lambda: call(held=None, hout=None))
    _no_device(lambda: call(hout=ok["held"] + 32))
    _no_device(lambda: call(B=0, held=None))


def test_binding_of_held_blocks_refuses():
    i32 = dict(dtype=torch.int32)
    z = torch.zeros
    args = (z(2, **i32), z(2, **i32), z((2, 4), **i32), z(9, **i32), z(1, **i32), 16, 8)
    for held in (z(3, **i32), z(2), z(4, **i32)[::2]):
        with pytest.raises(ValueError, match="held_blocks"):
            fq.paged_batch_tables(*args, held_blocks=held)
    five = (z(3, **i32), z(2, **i32), z(8, dtype=torch.int64), z(8, dtype=torch.int64), z(1, **i32))
    with pytest.raises(ValueError, match="sixth"):
        fq.paged_batch_tables(*args, held_blocks=z(2, **i32), out=five)
    with pytest.raises(ValueError, match="held_out"):
        fq.paged_batch_tables(*args, held_blocks=z(2, **i32), out=(*five, z(3, **i32)))
    with pytest.raises(ValueError, match="CUDA"):
        fq.paged_batch_tables(*args, held_blocks=z(2, **i32), out=(*five, z(2, **i32)))


def test_accept_without_a_layer_is_refused_by_the_binding():
    """The C call does nothing then, and the binding would return lengths that nothing has written."""
    i32 = dict(dtype=torch.int32)
    z = torch.zeros
    ctx, cu, table = z(2, **i32), z(3, **i32), z((2, 4), **i32)
    k = z((0, 64, 256), dtype=torch.uint8)
    for out in (None, z(2, **i32)):
        with pytest.raises(ValueError, match="layer"):
            fq.kv_cache_accept(k, k, table, ctx, cu, z((2, 3), **i32), ctx, 16, out_lens=out)


def test_selftest_attention_tree(L):
    """The limit's range, then the ordinary call's checks."""
    def call(polls, B=2, D=128, ws=FAKE):
        return L.fp8q_selftest_attention_tree(polls, FAKE, 1024, FAKE, FAKE, 64, FAKE, FAKE, 4, FAKE,
                                              FAKE, None, 0, B, 8, 8, 2, D, 16, 16, 64, 0.088, FAKE,
                                              1024, ws, 1 << 40, None)
    for polls in (0, -1, (1 << 18) + 1):
        assert call(polls) == ARG
    assert call(1, D=96) == SHAPE and call(1, ws=None) == NULL and call(1, B=0) == OK
    _no_device(lambda: call(1))
    _no_device(lambda: call(1 << 18))


def test_accept_of_overlapping_caches_is_refused_by_the_binding():
    """Rows of K and V move at the same time: one of them would read what the other has moved."""
    i32 = dict(dtype=torch.int32)
    z = torch.zeros
    ctx, cu, table = z(2, **i32), z(3, **i32), z((2, 4), **i32)
    both = z((100, 256), dtype=torch.uint8)
    for k, v in ((both, both), (both[:64], both[36:]), (both[36:], both[:64])):
        with pytest.raises(ValueError, match="overlap"):
            fq.kv_cache_accept(k, v, table, ctx, cu, z((2, 3), **i32), ctx, 16)
    with pytest.raises(ValueError, match="CUDA"):                 # adjacent is not overlapping
        fq.kv_cache_accept(both[:50], both[50:], table, ctx, cu, z((2, 3), **i32), ctx, 16)
