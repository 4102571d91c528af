"""Host-side checks of the calls of selective state space layers: what the library and the binding
refuse before anything is launched. Only invalid arguments (or empty calls) reach the library."""
import ctypes

import pytest
import torch

from test_paged_tensors import On

FAKE = 1 << 20  # never dereferenced: every call below returns from validation
BAD, NO = 1, 2  # GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED
BF16, FP32, E4M3, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


@pytest.fixture(scope="module")
def gdn():
    from linear_attention_decode_gdn_gb300 import build
    build.build()
    import linear_attention_decode_gdn_gb300 as g
    return g


def filled(struct, values):
    s = struct()
    for name, value in values.items():
        setattr(s, name, (ctypes.c_int64 * len(value))(*value) if name.endswith("strides") else value)
    return s


def norm(gdn, **kw):
    d = dict(rows=3, width=256, x_type=0, residual_type=0, o_type=0, group=0, eps=1e-6, x=FAKE, x_stride=256, residual=FAKE,
             residual_stride=256, weight=FAKE, o=FAKE, scales=None)
    return filled(gdn._abi.Norm, {**d, **kw})


def conv(gdn, **kw):
    d = dict(batch=2, num_tokens=4, channels=64, num_slots=3, flags=gdn.QKV_BF16 | gdn.CONV_SILU, x=FAKE, x_strides=(256, 64), w=FAKE,
             bias=FAKE, pool=FAKE, slot=FAKE, seq_lens=None, o=2 * FAKE)
    return filled(gdn._abi.Conv, {**d, **kw})


def ssm(gdn, **kw):
    d = dict(batch=2, num_tokens=4, channels=64, state_size=16, num_groups=2, num_slots=3, flags=gdn.QKV_BF16 | gdn.DT_SOFTPLUS, u=FAKE,
             u_strides=(256, 64), dt=FAKE, dt_strides=(256, 64), b=FAKE, b_strides=(128, 32, 16), c=FAKE, c_strides=(128, 32, 16), z=FAKE,
             z_strides=(512, 128), a=FAKE, skip=FAKE, dt_bias=FAKE, state=FAKE, slot=FAKE, seq_lens=None, y=FAKE)
    return filled(gdn._abi.Ssm, {**d, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(width=0), BAD), (dict(x_type=2), BAD), (dict(x_type=-1), BAD), (dict(residual_type=2), BAD), (dict(o_type=3), BAD),
    (dict(group=128), NO), (dict(o_type=2, scales=FAKE, group=64), NO), (dict(width=252), NO), (dict(width=16392), NO), (dict(x=None), BAD),
    (dict(o=None), BAD), (dict(o_type=2), BAD), (dict(x=FAKE + 8), NO), (dict(residual=FAKE + 2), NO), (dict(weight=FAKE + 4), NO),
    (dict(o=FAKE + 8), NO), (dict(x_stride=260), NO), (dict(x_stride=-256), NO), (dict(residual_stride=260), NO), (dict(x_type=1, x_stride=258), NO),
    (dict(residual_stride=0), BAD), (dict(residual_stride=128), BAD)])
def test_norm_is_checked(gdn, kw, code):
    assert gdn._abi.load().gdn_add_rms_norm(ctypes.byref(norm(gdn, **kw)), None) == code


def test_empty_calls_launch_nothing(gdn):
    lib = gdn._abi.load()
    assert lib.gdn_add_rms_norm(ctypes.byref(norm(gdn, rows=0, x=None, o=None)), None) == 0
    for kw in (dict(batch=0), dict(num_tokens=0)):
        assert lib.gdn_causal_conv(ctypes.byref(conv(gdn, x=None, **kw)), None, None) == 0
        assert lib.gdn_ssm_scan(ctypes.byref(ssm(gdn, u=None, **kw)), None, 0, None, None) == 0
    assert lib.gdn_ssm_step(ctypes.byref(ssm(gdn, batch=0, num_tokens=1, u=None)), None, None) == 0
    assert lib.gdn_add_rms_norm(None, None) == BAD and lib.gdn_causal_conv(None, None, None) == BAD
    assert lib.gdn_ssm_scan(None, None, 0, None, None) == BAD and lib.gdn_ssm_step(None, None, None) == BAD


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(num_tokens=-1), BAD), (dict(channels=0), BAD), (dict(num_slots=0), BAD), (dict(flags=1 << 11), BAD),
    (dict(flags=1 << 1), BAD), (dict(channels=60), NO), (dict(batch=1 << 20, num_tokens=1 << 12), NO), (dict(batch=1 << 14, num_tokens=1 << 16, channels=512), NO),
    (dict(channels=(1 << 24) + 8), NO), (dict(batch=(1 << 31) - 1, num_tokens=(1 << 31) - 1, channels=(1 << 31) - 8), NO),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(pool=None), BAD), (dict(slot=None), BAD), (dict(o=None), BAD), (dict(x=FAKE + 8), NO),
    (dict(x_strides=(256, 60)), NO), (dict(x_strides=(-256, 64)), NO), (dict(w=FAKE + 4), NO), (dict(bias=FAKE + 4), NO), (dict(pool=FAKE + 2), NO),
    (dict(o=FAKE + 8), NO), (dict(o=FAKE), BAD)])
def test_conv_is_checked(gdn, kw, code):
    assert gdn._abi.load().gdn_causal_conv(ctypes.byref(conv(gdn, **kw)), None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(num_tokens=-1), BAD), (dict(channels=0), BAD), (dict(num_groups=0), BAD), (dict(num_slots=0), BAD),
    (dict(flags=1 << 12), BAD), (dict(state_size=0), NO), (dict(state_size=24), NO), (dict(state_size=128), NO), (dict(channels=72), NO),
    (dict(num_groups=16), NO), (dict(num_groups=1 << 29), NO), (dict(batch=1 << 20, num_tokens=1 << 12), NO),
    (dict(batch=1 << 22, num_tokens=1, channels=1 << 16), NO), (dict(channels=(1 << 24) + 16), NO),
    (dict(batch=(1 << 31) - 1, num_tokens=(1 << 31) - 1, channels=(1 << 31) - 16, state_size=64), NO), (dict(u=None), BAD), (dict(dt=None), BAD), (dict(b=None), BAD), (dict(c=None), BAD),
    (dict(a=None), BAD), (dict(state=None), BAD), (dict(slot=None), BAD), (dict(y=None), BAD), (dict(u=FAKE + 8), NO), (dict(dt=FAKE + 8), NO),
    (dict(b=FAKE + 2), NO), (dict(c=FAKE + 2), NO), (dict(z=FAKE + 2), NO), (dict(u_strides=(256, 60)), NO), (dict(dt_strides=(-8, 64)), NO),
    (dict(b_strides=(128, 36, 16)), NO), (dict(c_strides=(128, 32, 4)), NO), (dict(z_strides=(516, 128)), NO), (dict(a=FAKE + 4), NO),
    (dict(skip=FAKE + 4), NO), (dict(dt_bias=FAKE + 4), NO), (dict(state=FAKE + 4), NO), (dict(y=FAKE + 4), NO)])
def test_scan_and_step_are_checked(gdn, kw, code):
    lib = gdn._abi.load()
    assert lib.gdn_ssm_scan(ctypes.byref(ssm(gdn, **kw)), FAKE, 1 << 40, None, None) == code
    kw = {**kw, "num_tokens": kw.get("num_tokens", 1)}
    if kw["num_tokens"] == 1 and not any(name.endswith("strides") for name in kw):  # one token's stride may be any
        assert lib.gdn_ssm_step(ctypes.byref(ssm(gdn, **kw)), None, None) == code


def test_step_takes_one_token(gdn):
    lib = gdn._abi.load()
    for kw in (dict(num_tokens=2), dict(num_tokens=0), dict(num_tokens=1, seq_lens=FAKE)):
        assert lib.gdn_ssm_step(ctypes.byref(ssm(gdn, **kw)), None, None) == BAD


def test_workspace_sizes(gdn):
    lib = gdn._abi.load()
    size = ctypes.c_size_t()
    assert lib.gdn_ssm_workspace(1, 1, 64, 16, None) == BAD
    for args in ((-1, 1, 64, 16), (1, -1, 64, 16), (1, 1, 0, 16)):
        assert lib.gdn_ssm_workspace(*args, ctypes.byref(size)) == BAD
    for args in ((1, 1, 64, 24), (1, 1, (1 << 24) + 8, 16), (1 << 20, 1 << 20, 64, 16), ((1 << 31) - 1, 1, 1 << 24, 64)):
        assert lib.gdn_ssm_workspace(*args, ctypes.byref(size)) == NO
    assert gdn.ssm_workspace_bytes(0, 1000, 64, 16) == 0 == gdn.ssm_workspace_bytes(8, 0, 64, 16)
    need = gdn.ssm_workspace_bytes(1, 8192, 2048, 16)
    if need:  # a scan in parts
        s = ctypes.byref(ssm(gdn, batch=1, num_tokens=8192, channels=2048, num_groups=1))
        assert lib.gdn_ssm_scan(s, FAKE, need - 1, None, None) == BAD
        assert lib.gdn_ssm_scan(s, None, need, None, None) == BAD
        assert lib.gdn_ssm_scan(s, FAKE + 8, need, None, None) == NO


def test_packed_structs_are_the_c_structs(gdn):
    from linear_attention_decode_gdn_gb300 import selective
    big = 5 << 40
    n = norm(gdn, x=big, x_stride=1 << 33, residual=big + 16, residual_stride=1 << 34, eps=0.25, o_type=2, group=128, scales=big + 32)
    assert bytes(n) == selective._pack_norm(n.rows, n.width, n.x_type, n.residual_type, n.o_type, n.group, n.eps, n.x, n.x_stride, n.residual,
                                            n.residual_stride, n.weight, n.o, n.scales)
    c = conv(gdn, x=big, x_strides=(1 << 33, 8), seq_lens=big + 4, o=big + 64)
    assert bytes(c) == selective._pack_conv(c.batch, c.num_tokens, c.channels, c.num_slots, c.flags, c.x, *c.x_strides, c.w, c.bias, c.pool, c.slot,
                                            c.seq_lens, c.o)
    s = ssm(gdn, u=big, u_strides=(1 << 33, 8), b_strides=(1 << 34, 1 << 33, 16), seq_lens=big + 4, y=big + 64)
    assert bytes(s) == selective._pack_ssm(s.batch, s.num_tokens, s.channels, s.state_size, s.num_groups, s.num_slots, s.flags, s.u, *s.u_strides, s.dt,
                                           *s.dt_strides, s.b, *s.b_strides, s.c, *s.c_strides, s.z, *s.z_strides, s.a, s.skip, s.dt_bias, s.state,
                                           s.slot, s.seq_lens, s.y)


# ---- the binding, with stand-ins that say where they live ----------------------------------------
class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*_):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def selective(monkeypatch):
    from linear_attention_decode_gdn_gb300 import selective
    lib = Library()
    monkeypatch.setattr(selective._abi, "load", lambda: lib)
    monkeypatch.setattr(selective, "_current_device", lambda: 0)
    monkeypatch.setattr("linear_attention_decode_gdn_gb300.paged._raw_stream", lambda device: 7)
    selective.lib = lib
    return selective


def calls(m):
    yield (lambda d: m.add_rms_norm(d["x"], d["o"], residual=d["residual"], weight=d["weight"], scales=d["scales"], group=128),
           dict(x=On((3, 136), BF16), o=On((3, 136), E4M3), residual=On((3, 136), FP32), weight=On((136,), FP32), scales=On((3, 2), FP32)))
    for at in ((2, 4), (2,)):
        yield (lambda d: m.causal_conv(d["x"], d["weight"], d["pool"], d["slot"], d["o"], bias=d["bias"], seq_lens=d["seq_lens"], status=d["status"]),
               dict(x=On(at + (64,), BF16), weight=On((64, 4), FP32), pool=On((5, 64, 3), BF16), slot=On((2,), I32), o=On(at + (64,), BF16),
                    bias=On((64,), FP32), seq_lens=On((2,), I32), status=On((1,), I32)))
        layer = dict(u=On(at + (64,), FP32), dt=On(at + (64,), FP32), a=On((64, 16), FP32), b=On(at + (2, 16), FP32), c=On(at + (2, 16), FP32),
                     state=On((5, 64, 16), FP32), slot=On((2,), I32), y=On(at + (64,), FP32), z=On(at + (64,), FP32), skip=On((64,), FP32),
                     dt_bias=On((64,), FP32), status=On((1,), I32))
        if len(at) == 1:
            yield lambda d: m.ssm_step(*list(d.values())[:8], **{k: d[k] for k in ("z", "skip", "dt_bias", "status")}), layer
        else:
            yield (lambda d: m.ssm_scan(*list(d.values())[:8], d["workspace"], **{k: d[k] for k in ("z", "skip", "dt_bias", "seq_lens", "status")}),
                   {**layer, "seq_lens": On((2,), I32), "workspace": On((64,), torch.uint8)})


def test_every_tensor_of_a_call_lives_on_the_current_device(selective, monkeypatch):
    for call, tensors in calls(selective):
        selective.lib.calls = 0
        call(tensors)
        assert selective.lib.calls == 1
        for name, t in tensors.items():
            for at in (-1, 1):
                with pytest.raises(ValueError):
                    call({**tensors, name: On(t.shape, t.dtype, at)})
        with monkeypatch.context() as m:
            m.setattr(selective, "_current_device", lambda: 1)
            with pytest.raises(ValueError, match="current"):
                call(tensors)
        assert selective.lib.calls == 1


def test_types_and_shapes_are_checked(selective):
    for call, tensors in calls(selective):
        selective.lib.calls = 0
        for name, t in tensors.items():
            if name == "workspace":  # bytes of any kind
                continue
            wrong = [On(t.shape, torch.float16)]
            if name != "status":  # its first word counts
                wrong.append(On((*t.shape[:-1], t.shape[-1] + 8), t.dtype))
            if t.dtype is not I32:  # a list of integers may have any dimensions
                wrong.append(On((1, 1, *t.shape), t.dtype))
            for bad in wrong:
                with pytest.raises(ValueError):
                    call({**tensors, name: bad})
                    pytest.fail(f"{name}: {bad.dtype} {bad.shape}")
        assert selective.lib.calls == 0


def test_norm_outputs_and_scales_go_together(selective):
    x, o = On((3, 136), BF16), On((3, 136), BF16)
    for kw in (dict(scales=On((3, 1), FP32)), dict(group=128)):
        with pytest.raises(ValueError, match="8 bits"):
            selective.add_rms_norm(x, o, **kw)
    with pytest.raises(ValueError, match="8 bits"):
        selective.add_rms_norm(x, On((3, 136), E4M3))
    selective.add_rms_norm(x, On((3, 136), E4M3), scales=On((3,), FP32))
    assert selective.lib.calls == 1
