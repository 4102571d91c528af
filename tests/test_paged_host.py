"""Host-side checks of the paged-cache calls: what is refused, before anything is launched,
and the workspace sizes. Only invalid arguments (or empty calls) reach the library here."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # never dereferenced: every call below returns from validation


@pytest.fixture(scope="module")
def gdn():
    from linear_attention_decode_gdn_gb300 import build
    build.build()
    import linear_attention_decode_gdn_gb300 as g
    return g


def cache(gdn, **kw):
    d = dict(k=FAKE, v=FAKE, k_strides=(8192, 512, 128), v_strides=(8192, 512, 128), num_pages=4, page_size=16,
             num_kv_heads=4, dk=128, dv=128)
    d.update(kw)
    kv = gdn._abi.PagedKV()
    for name, value in d.items():
        setattr(kv, name, (ctypes.c_int64 * 3)(*value) if name.endswith("strides") else value)
    return kv


def latent(gdn, **kw):
    return cache(gdn, **{**dict(v=None, num_kv_heads=1, dk=576, dv=512), **kw})


def attn(gdn, **kw):
    d = dict(batch=2, num_tokens=1, num_heads=8, max_pages=4, window=0, scale=1.0, q=FAKE, q_strides=(1024, 1024, 128),
             block_table=FAKE, kv_len=FAKE, o=FAKE, lse=None)
    d.update(kw)
    a = gdn._abi.Attn()
    for name, value in d.items():
        setattr(a, name, (ctypes.c_int64 * 3)(*value) if name.endswith("strides") else value)
    return a


def attend(gdn, kv, a, size=1 << 40, workspace=FAKE, name="gdn_attn_decode"):
    by = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return getattr(gdn._abi.load(), name)(by(kv), by(a), workspace, size, None, None)


BAD, NO = 1, 2  # GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), BAD), (dict(num_pages=0), BAD), (dict(page_size=0), BAD), (dict(num_kv_heads=0), BAD),
    (dict(dk=0), BAD), (dict(dv=-8), BAD), (dict(dk=100), NO), (dict(dk=584), NO), (dict(dv=520), NO),
    (dict(k=FAKE + 8), NO), (dict(v=FAKE + 2), NO), (dict(k_strides=(8192, 512, 4)), NO),
    (dict(v_strides=(8192, -512, 128)), NO), (dict(v=None), BAD),
])
def test_cache_is_checked(gdn, kw, code):
    kv = cache(gdn, **kw)
    assert attend(gdn, kv, attn(gdn)) == code
    size = ctypes.c_size_t()
    assert gdn._abi.load().gdn_attn_workspace(ctypes.byref(kv), 1, 1, 8, ctypes.byref(size)) == code
    s2 = (ctypes.c_int64 * 2)(512, 128)
    assert gdn._abi.load().gdn_kv_append(ctypes.byref(kv), 3, FAKE, s2, FAKE, s2, FAKE, gdn.QKV_BF16, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(num_tokens=0), BAD), (dict(num_heads=0), BAD), (dict(num_heads=6), BAD),
    (dict(max_pages=0), BAD), (dict(window=-1), BAD), (dict(max_pages=1 << 28), BAD), (dict(num_tokens=2049), NO),
    (dict(batch=1 << 28, num_heads=16), BAD), (dict(q=None), BAD), (dict(block_table=None), BAD),
    (dict(kv_len=None), BAD), (dict(o=None), BAD), (dict(q=FAKE + 8), NO), (dict(o=FAKE + 4), NO),
    (dict(q_strides=(1024, 1024, 100)), NO), (dict(q_strides=(-1024, 1024, 128)), NO),
])
def test_attention_arguments_are_checked(gdn, kw, code):
    assert attend(gdn, cache(gdn), attn(gdn, **kw)) == code
    assert gdn._abi.load().gdn_last_error()


def test_attention_cache_kinds_and_workspace(gdn):
    lib = gdn._abi.load()
    assert attend(gdn, None, attn(gdn)) == BAD
    assert attend(gdn, cache(gdn), None) == BAD
    assert attend(gdn, cache(gdn), attn(gdn), workspace=None) == BAD
    assert attend(gdn, cache(gdn), attn(gdn), workspace=FAKE + 8) == NO
    assert attend(gdn, cache(gdn), attn(gdn), size=16) == BAD
    assert attend(gdn, cache(gdn), attn(gdn), name="gdn_latent_decode") == BAD
    assert attend(gdn, latent(gdn), attn(gdn)) == BAD
    assert attend(gdn, latent(gdn, dk=256, dv=512), attn(gdn), name="gdn_latent_decode") == BAD
    assert attend(gdn, latent(gdn, num_kv_heads=2), attn(gdn), name="gdn_latent_decode") == BAD
    # an empty batch is no call at all
    assert attend(gdn, cache(gdn), attn(gdn, batch=0)) == 0
    size = ctypes.c_size_t()
    assert lib.gdn_attn_workspace(ctypes.byref(cache(gdn)), 1, 1, 8, None) == BAD
    assert lib.gdn_attn_workspace(ctypes.byref(cache(gdn)), 1, 1, 6, ctypes.byref(size)) == BAD
    assert lib.gdn_attn_workspace(ctypes.byref(cache(gdn)), 1, 4096, 8, ctypes.byref(size)) == NO
    sizes = []
    for tokens in (1, 2, 16):
        assert lib.gdn_attn_workspace(ctypes.byref(cache(gdn)), 1, tokens, 8, ctypes.byref(size)) == 0
        sizes.append(size.value)
    assert 0 < sizes[0] <= sizes[1] <= sizes[2] < 1 << 27  # grows with the columns, never with the batch


def test_append_arguments_are_checked(gdn):
    lib = gdn._abi.load()
    s2, odd = (ctypes.c_int64 * 2)(512, 128), (ctypes.c_int64 * 2)(510, 128)
    kv, bf16 = ctypes.byref(cache(gdn)), gdn.QKV_BF16
    assert lib.gdn_kv_append(None, 1, FAKE, s2, FAKE, s2, FAKE, bf16, None, None) == BAD
    assert lib.gdn_kv_append(kv, -1, FAKE, s2, FAKE, s2, FAKE, bf16, None, None) == BAD
    assert lib.gdn_kv_append(kv, 1, FAKE, s2, FAKE, s2, FAKE, gdn.FUSE_CONV, None, None) == BAD
    assert lib.gdn_kv_append(kv, 0, None, None, None, None, None, bf16, None, None) == 0
    for args in ((None, s2, FAKE, s2, FAKE), (FAKE, None, FAKE, s2, FAKE), (FAKE, s2, None, s2, FAKE),
                 (FAKE, s2, FAKE, None, FAKE), (FAKE, s2, FAKE, s2, None)):
        assert lib.gdn_kv_append(kv, 1, *args, bf16, None, None) == BAD
    for args in ((FAKE + 8, s2, FAKE, s2, FAKE), (FAKE, odd, FAKE, s2, FAKE), (FAKE, s2, FAKE, odd, FAKE)):
        assert lib.gdn_kv_append(kv, 2, *args, bf16, None, None) == NO
    assert lib.gdn_kv_append(kv, 2, FAKE, odd, FAKE, s2, FAKE, 0, None, None) == NO  # fp32: multiples of 4
    # a latent cache without a tail needs no second source
    assert lib.gdn_kv_append(ctypes.byref(latent(gdn)), 1, FAKE, s2, None, None, FAKE, bf16, None, None) == BAD


def test_plan_and_release_arguments_are_checked(gdn):
    lib = gdn._abi.load()

    def plan(batch=2, pages=4, size=16, total=8, room=8, capacity=2, **kw):
        ptr = dict(cached=FAKE, new=None, held=FAKE, table=FAKE, free=FAKE, count=FAKE, kv=FAKE, cu=FAKE, slots=FAKE,
                   held_out=FAKE, count_out=FAKE)
        ptr.update(kw)
        return lib.gdn_kv_plan(batch, pages, size, total, room, capacity, *ptr.values(), None, None)

    for kw in (dict(batch=-1), dict(pages=0), dict(size=0), dict(total=0), dict(room=-1), dict(capacity=-1)):
        assert plan(**kw) == BAD, kw
    assert plan(batch=4097) == NO
    assert plan(batch=0) == 0
    for name in ("cached", "held", "table", "free", "count", "kv", "cu", "slots", "held_out", "count_out"):
        assert plan(**{name: None}) == BAD, name

    def release(batch=2, pages=4, total=8, n=1, **kw):
        ptr = dict(requests=FAKE, n=n, table=FAKE, held=FAKE, free=FAKE, count=FAKE)
        ptr.update(kw)
        return lib.gdn_kv_release(batch, pages, total, *ptr.values(), None, None)

    for kw in (dict(batch=-1), dict(pages=0), dict(total=0), dict(n=-1), dict(requests=None), dict(table=None),
               dict(held=None), dict(free=None), dict(count=None)):
        assert release(**kw) == BAD, kw
    assert release(n=0, requests=None) == 0


def test_tensors_on_the_host_are_refused(gdn):
    pages = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        gdn.make_paged_kv(pages, pages)
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="cached_len"):
        gdn.kv_plan(ints, None, ints, ints[None], ints, ints[:1], kv_len=ints, cu_new=ints, slot_map=ints,
                    held_out=ints, free_count_out=ints, page_size=16, num_pages=4)
    with pytest.raises(ValueError, match="requests"):
        gdn.kv_release(ints, ints, ints[None], ints, ints[:1])


def test_packed_structs_are_the_c_structs(gdn):
    """The binding packs the structs by hand: the same bytes as the ctypes layout of gdn.h."""
    from linear_attention_decode_gdn_gb300 import paged
    kv = cache(gdn, k=3 << 40, k_strides=(1 << 33, 16, 8), v_strides=(24, 1 << 34, 32))
    assert bytes(kv) == paged._pack_kv(kv.k, kv.v, *kv.k_strides, *kv.v_strides, kv.num_pages, kv.page_size, kv.num_kv_heads,
                                       kv.dk, kv.dv)
    a = attn(gdn, window=7, scale=0.25, lse=5 << 40)
    assert bytes(a) == paged._pack_attn(a.batch, a.num_tokens, a.num_heads, a.max_pages, a.window, a.scale, a.q, *a.q_strides,
                                        a.block_table, a.kv_len, a.o, a.lse)
