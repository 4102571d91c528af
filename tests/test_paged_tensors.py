"""What the paged-cache binding refuses of tensors, without a GPU: stand-ins that say where they live, and a
library that only counts its calls."""
import pytest
import torch

BF16, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


class On:
    """A contiguous tensor's face on device `at` (-1: the host)."""

    def __init__(self, shape, dtype, at=0):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, at
        self.device = torch.device("cpu") if at < 0 else torch.device("cuda", at)
        self.is_cuda, self.nbytes = at >= 0, self.numel() * torch.empty(0, dtype=dtype).element_size()

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def stride(self, i=None):
        s = torch.empty(self.shape, device="meta").stride()
        return s if i is None else s[i]


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*_):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def paged(monkeypatch):
    from linear_attention_decode_gdn_gb300 import paged
    lib = Library()
    monkeypatch.setattr(paged._abi, "load", lambda: lib)
    monkeypatch.setattr(paged, "_current_device", lambda: 0)
    monkeypatch.setattr(paged, "_raw_stream", lambda device: 7)
    paged.lib = lib
    return paged


def calls(paged, latent):
    """(function, positional and keyword tensors by name) of every entry point."""
    B, n, pages, ps, hk, dk, dv = 3, 5, 4, 16, 1 if latent else 2, 64, 48
    pool = {"k": On((pages, ps, hk, dk), BF16), "v": None if latent else On((pages, ps, hk, dv), BF16)}
    make = lambda d: paged.make_paged_kv(d["k"], d["v"], dv=dv)  # noqa: E731
    plan = dict(cached_len=On((B,), I32), new_len=On((B,), I32), held=On((B,), I32), block_table=On((B, 4), I32), free_list=On((9,), I32),
                free_count=On((1,), I32), kv_len=On((B,), I32), cu_new=On((B + 1,), I32), slot_map=On((n,), I64), held_out=On((B,), I32),
                free_count_out=On((1,), I32), status=On((1,), I32))
    yield lambda d: paged.kv_plan(*(d[x] for x in list(d)[:6]), **{x: d[x] for x in list(d)[6:]}, page_size=ps, num_pages=pages), plan
    yield (lambda d: paged.kv_release(*(d[x] for x in list(d)[:5]), status=d["status"]),
           dict(requests=On((2,), I32), held=On((B,), I32), block_table=On((B, 4), I32), free_list=On((9,), I32), free_count=On((1,), I32),
                status=On((1,), I32)))
    first, second = (dv, dk - dv) if latent else (dk, dv)
    yield (lambda d: paged.kv_append(make(pool), d["k"], d["v"], d["slot_map"], status=d["status"]),
           dict(k=On((n, hk, first), F32), v=On((n, hk, second), F32), slot_map=On((n,), I64), status=On((1,), I32)))
    attend = paged.latent_decode if latent else paged.attn_decode
    yield (lambda d: attend(make(pool), d["q"], d["block_table"], d["kv_len"], d["o"], d["workspace"], lse=d["lse"], status=d["status"]),
           dict(q=On((B, 2, 4, dk), BF16), block_table=On((B, 4), I32), kv_len=On((B,), I32), o=On((B, 2, 4, dv), BF16),
                workspace=On((64,), torch.uint8), lse=On((B, 2, 4), F32), status=On((1,), I32)))


@pytest.mark.parametrize("latent", [False, True])
def test_every_tensor_of_a_call_lives_on_the_current_device(paged, latent, monkeypatch):
    for call, tensors in calls(paged, latent):
        paged.lib.calls = 0
        call(tensors)
        assert paged.lib.calls == 1
        for name, t in tensors.items():
            for at in (-1, 1):
                with pytest.raises(ValueError):
                    call({**tensors, name: On(t.shape, t.dtype, at)})
                assert paged.lib.calls == 1, name
        # all beside one another, but not where the launch goes
        with monkeypatch.context() as m:
            m.setattr(paged, "_current_device", lambda: 1)
            with pytest.raises(ValueError, match="current"):
                call(tensors)
        assert paged.lib.calls == 1
    elsewhere = On((4, 16, 2, 64), BF16, 1)
    with pytest.raises(ValueError, match="beside"):
        paged.make_paged_kv(On((4, 16, 2, 64), BF16), elsewhere)
    kv = paged.make_paged_kv(elsewhere, elsewhere)
    with pytest.raises(ValueError, match="current"):
        paged.attn_decode(kv, On((1, 1, 2, 64), BF16, 1), On((1, 1), I32, 1), On((1,), I32, 1), On((1, 1, 2, 64), BF16, 1), On((64,), I32, 1))


def test_the_status_word_is_checked(paged):
    for call, tensors in calls(paged, False):
        paged.lib.calls = 0
        call({**tensors, "status": None})
        call({**tensors, "status": On((3,), I32)})  # its first word
        assert paged.lib.calls == 2
        for bad in (On((1,), torch.uint8), On((1,), I64), On((0,), I32), On((1,), I32, -1)):
            with pytest.raises(ValueError, match="status"):
                call({**tensors, "status": bad})
        assert paged.lib.calls == 2


def test_an_empty_batch_writes_nothing():
    """The library itself, with arrays of the host behind the pointers: no call is launched, so none is touched."""
    import ctypes
    from linear_attention_decode_gdn_gb300 import _abi, build
    build.build()
    arrays = [(ctypes.c_int64 * 8)(*[77] * 8) for _ in range(11)]
    assert _abi.load().gdn_kv_plan(0, 4, 16, 8, 8, 8, *arrays, None, None) == 0
    assert all(list(a) == [77] * 8 for a in arrays)
