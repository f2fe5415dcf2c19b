"""The cache and tree entry points without a GPU: bad arguments are refused on the
host, before any CUDA call, with the documented status; the binding refuses what
the C side cannot see."""
import ctypes

import pytest
import torch

import draft_selection_gb300 as dfl2
from draft_selection_gb300 import build as dbuild
from draft_selection_gb300 import _CacheStruct

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
A = 0x10000  # an aligned stand-in address: never dereferenced by these tests


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dfl2.load()


def cache(**kw):
    c = dict(k=A, v=A, dtype=1, layers=2, pages=10, kv_heads=4, page_size=16, head_dim=128,
             layer_stride=81920, page_stride=8192, head_stride=2048, slot_stride=128, table=A,
             rows=3, cols=5, refs=A, free_bits=A)
    c.update(kw)
    return ctypes.byref(_CacheStruct(**c))


S3 = ctypes.c_int64 * 3
S4 = ctypes.c_int64 * 4
QS = S3(4096, 1024, 128)


def attn(lib, c=None, q=A, qs=QS, layer=0, B=2, T=4, hq=8, length=A, out=A, os_=QS, scale=0.1,
         ws=A, n=1 << 40, mask=A, lse=A):
    return lib.dfl2_tree_attn(q, qs, c or cache(), layer, B, T, hq, None, length, None, mask, scale,
                              out, os_, lse, ws, n, None)


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=A + 8), INVALID),
    (dict(table=None), INVALID), (dict(table=A + 2), INVALID), (dict(refs=None), INVALID),
    (dict(free_bits=None), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(layers=0), INVALID),
    (dict(pages=0), INVALID), (dict(kv_heads=0), INVALID), (dict(rows=0), INVALID),
    (dict(cols=-1), INVALID), (dict(page_size=12), UNSUPPORTED), (dict(page_size=4), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(head_dim=100), UNSUPPORTED),
    (dict(kv_heads=1024), UNSUPPORTED), (dict(slot_stride=130), INVALID),
    (dict(page_stride=-8), INVALID)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_call_checks_its_cache(lib, bad, status):
    c = cache(**bad)
    assert attn(lib, c) == status
    assert lib.dfl2_cache_reserve(c, 1, 4, None, A, None, A, None) == status
    assert lib.dfl2_cache_write(c, 0, 1, A, A, S4(0, 0, 0, 0), 1, 4, None, A, None, None) == status
    assert lib.dfl2_cache_compact(c, 1, 4, None, A, None, A, A, A, None) == status
    assert lib.dfl2_cache_fork(c, 1, A, A, A, A, None) == status
    assert lib.dfl2_cache_free(c, 1, A, None) == status
    assert dfl2.dfl2_last_error()


def test_no_cache(lib):
    assert lib.dfl2_cache_free(None, 1, A, None) == INVALID


def test_attention_refuses(lib):
    for kw, status in [
            (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(hq=0), INVALID),
            (dict(hq=6), INVALID), (dict(T=257), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
            (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(q=None), INVALID),
            (dict(q=A + 8), INVALID), (dict(length=None), INVALID), (dict(length=A + 1), INVALID),
            (dict(out=None), INVALID), (dict(out=A + 4), INVALID), (dict(mask=A + 2), INVALID),
            (dict(lse=A + 2), INVALID), (dict(qs=S3(4096, 1028, 128)), INVALID),
            (dict(os_=S3(4096, -1024, 128)), INVALID), (dict(scale=float("nan")), INVALID),
            (dict(scale=float("inf")), INVALID), (dict(c=cache(dtype=0)), UNSUPPORTED),
            (dict(c=cache(head_dim=96)), UNSUPPORTED), (dict(qs=None), INVALID)]:
        assert attn(lib, **kw) == status, kw


def test_bookkeeping_refuses(lib):
    c = cache()
    r = lib.dfl2_cache_reserve
    assert r(c, 0, 4, None, A, None, A, None) == INVALID
    assert r(c, 4097, 4, None, A, None, A, None) == UNSUPPORTED
    assert r(c, 1, -1, None, A, None, A, None) == INVALID
    assert r(c, 1, 4, None, None, None, A, None) == INVALID
    assert r(c, 1, 4, None, A, None, None, None) == INVALID
    assert r(c, 1, 4, A + 2, A, None, A, None) == INVALID
    w = lib.dfl2_cache_write
    ok = S4(0, 0, 512, 128)
    assert w(c, 0, 3, A, A, ok, 1, 4, None, A, None, None) == INVALID      # three layers of two
    assert w(c, -1, 1, A, A, ok, 1, 4, None, A, None, None) == INVALID
    assert w(c, 0, 0, A, A, ok, 1, 4, None, A, None, None) == INVALID
    assert w(c, 0, 1, None, A, ok, 1, 4, None, A, None, None) == INVALID
    assert w(c, 0, 1, A, A + 8, ok, 1, 4, None, A, None, None) == INVALID
    assert w(c, 0, 1, A, A, None, 1, 4, None, A, None, None) == INVALID
    assert w(c, 0, 1, A, A, S4(0, 0, 100, 128), 1, 4, None, A, None, None) == INVALID
    p = lib.dfl2_cache_compact
    assert p(c, 1, 257, None, A, None, A, A, A, None) == UNSUPPORTED
    assert p(c, 1, 4, None, A, None, None, A, A, None) == INVALID
    assert p(c, 1, 4, None, A, None, A, None, A, None) == INVALID
    assert p(c, 1, 4, None, A, None, A, A, None, None) == INVALID
    f = lib.dfl2_cache_fork
    assert f(c, 0, A, A, A, A, None) == INVALID
    assert f(c, 1, None, A, A, A, None) == INVALID
    assert f(c, 1, A, None, A, A, None) == INVALID
    assert f(c, 1, A, A, None, A, None) == INVALID
    assert f(c, 1, A, A, A, None, None) == INVALID
    assert lib.dfl2_cache_free(c, 1, None, None) == INVALID


def test_needs_that_32_bits_do_not_count_are_refused(lib):
    c = cache(cols=1 << 20)
    r = lib.dfl2_cache_reserve
    assert r(c, 2048, 1 << 30, None, A, A, A, None) == UNSUPPORTED      # 2^31 entries
    assert r(c, 2048, 16 << 20, None, A, None, A, None) == UNSUPPORTED
    # (what is in range fails later, for want of a device or of its memory)
    assert r(c, 2047, 1 << 30, None, A, A, A, None) not in (0, UNSUPPORTED)
    assert r(c, 4096, 1 << 20, None, A, None, A, None) not in (0, UNSUPPORTED)


def test_no_rows_to_write_need_no_address(lib):
    w = lib.dfl2_cache_write
    st = S4(0, 0, 0, 0)
    args = 0, 1, None, None, st, 1, 0, None, A, None, None
    assert w(cache(), *args) != 0                    # for want of a device, or A is not its memory
    assert "k_new" not in dfl2.dfl2_last_error() and "v_new" not in dfl2.dfl2_last_error()
    assert w(cache(), 0, 1, None, A, st, 1, 1, None, A, None, None) == INVALID
    assert "k_new" in dfl2.dfl2_last_error()


def test_trees_refuse(lib):
    m, t = lib.dfl2_tree_mask, lib.dfl2_tree_accept
    assert m(None, 1, 4, None, A, None, None) == INVALID
    assert m(A, 1, 4, None, None, None, None) == INVALID
    assert m(A, 1, 0, None, A, None, None) == INVALID
    assert m(A, 1, 257, None, A, None, None) == UNSUPPORTED
    assert m(A + 2, 1, 4, None, A, None, None) == INVALID
    for i in range(6):
        args = [A] * 6
        args[i] = None
        assert t(args[0], args[1], args[2], 1, 4, None, *args[3:], None) == INVALID
    assert t(A, A, A, 0, 4, None, A, A, A, None) == INVALID
    assert t(A, A, A, 1, 300, None, A, A, A, None) == UNSUPPORTED


def test_workspace_size_of_a_refused_shape_is_zero(lib):
    for bad in [(0, 1, 8, 8, 128, 1), (1, 0, 8, 8, 128, 1), (1, 1, 7, 2, 128, 1),
                (1, 1, 8, 8, 96, 1), (1, 1, 8, 8, 128, 0), (1, 257, 8, 8, 128, 1)]:
        assert dfl2.dfl2_tree_attn_workspace_size(*bad) == 0


def test_binding_refuses_types_and_shapes():
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    assert c.free_bits.tolist() == [15] and c._s.page_stride == 2 * 16 * 64
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        dfl2.dfl2_cache_reserve(c, i.long(), 4, i)
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_reserve(c, i, 4, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_reserve(c, torch.zeros(4, dtype=torch.int32)[::2], 4, i)
    new = torch.zeros(2, 5, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_write(c, new.bfloat16(), new.bfloat16(), i)
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_write(c, new, new[:, :4], i)
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_write(c, new[:, :, :1], new[:, :, :1], i)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_attn(q.float(), c, 0, i, None, q.float(), i)
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_attn(q, c, 0, i, None, q, i, lse=torch.zeros(2, 3, 4, dtype=torch.float16))
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_attn(q, c, 0, i, torch.zeros(2, 3, 2, dtype=torch.int32), q, i)
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_compact(c, i, 4, torch.zeros(2, 3, dtype=torch.int32), i, i)
    with pytest.raises(TypeError):
        dfl2.Cache(c.k.int(), c.v.int(), c.table, c.refs, c.free_bits)
    with pytest.raises(ValueError):
        dfl2.Cache(c.k, c.v.transpose(2, 3).contiguous().transpose(2, 3), c.table, c.refs,
                   c.free_bits)
    with pytest.raises(ValueError):
        dfl2.Cache(c.k, c.v, c.table, c.refs[:2], c.free_bits)


def test_binding_refuses_what_is_no_tensor_or_number():
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    ij = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(TypeError):
        dfl2.dfl2_cache_reserve(c, [0, 0], 4, i)
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_reserve(c, ij, 4, i)
    with pytest.raises(OverflowError):
        dfl2.dfl2_cache_reserve(c, i, 1 << 31, i)
    with pytest.raises(AttributeError):
        dfl2.dfl2_cache_free(None, i)
    with pytest.raises(TypeError):
        dfl2.dfl2_cache_fork(c, i, i, i, i.numpy())
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_mask(ij, ij)                      # mask [2, 3, 1]
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_accept(ij, ij.t(), ij, ij, i, i)
    new = torch.zeros(2, 5, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_write(c, new[0], new[0], i)      # three dimensions
    with pytest.raises(ValueError):
        dfl2.dfl2_cache_write(c, new, new.transpose(0, 1).contiguous().transpose(0, 1), i)
    with pytest.raises(TypeError):
        dfl2.dfl2_cache_write(c, new, new, i, layer="0")
    q = torch.zeros(2, 3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_attn(q[0], c, 0, i, None, q[0], i)
    with pytest.raises(TypeError):
        dfl2.dfl2_tree_attn(q, c, 0, i, None, q, i, scale="1")
    with pytest.raises(ValueError):
        dfl2.dfl2_tree_attn(q.transpose(2, 3), c, 0, i, None, q.transpose(2, 3), i)


def test_binding_passes_the_c_sides_refusals_on():
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: dfl2.dfl2_cache_free(c, i, stream=1),              # no device memory
                 lambda: dfl2.dfl2_cache_reserve(c, i, 4, None, stream=1),  # no served
                 lambda: dfl2.dfl2_cache_reserve(c, i, -1, i, stream=1)):
        with pytest.raises(dfl2.Dfl2Error) as e:
            call()
        assert e.value.status != 0 and e.value.message


def test_calls_that_take_no_pages_have_the_attentions_batch(lib):
    """More than 4096 sequences are not refused (the call fails later, for want of a device or
    of its memory), more than 65535 are."""
    c = cache()
    st = S4(0, 0, 512, 128)
    calls = [lambda B: lib.dfl2_cache_write(c, 0, 1, A, A, st, B, 4, None, A, None, None),
             lambda B: lib.dfl2_cache_compact(c, B, 4, None, A, None, A, A, A, None),
             lambda B: lib.dfl2_cache_free(c, B, A, None)]
    for call in calls:
        assert call(4097) not in (0, UNSUPPORTED) and call(65535) not in (0, UNSUPPORTED)
        assert call(65536) == UNSUPPORTED
    assert lib.dfl2_cache_fork(c, 4097, A, A, A, A, None) == UNSUPPORTED


def test_binding_refuses_a_reserve_without_a_count():
    c = dfl2.cache(1, 4, 2, 16, 64, 2, 3, torch.float16, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="count"):
        dfl2.dfl2_cache_reserve(c, i, None, i, stream=1)
