"""Host-side checks of the selective state space layers' calls at edges that the other tests leave out. Only
invalid arguments reach the library."""
import ctypes
import random

import pytest

from test_paged_tensors import On
from test_selective_host import BAD, FAKE, NO, calls, conv, gdn, norm, selective, ssm  # noqa: F401


def test_a_workspace_of_the_largest_call_serves_all(gdn):  # noqa: F811
    """Fewer requests or positions never need more than the largest call, although they are cut into more parts."""
    need = gdn.ssm_workspace_bytes
    assert need(64, 1024, 4096, 16) >= need(16, 1024, 4096, 16) >= need(4, 896, 4096, 16) > 0
    assert need(64, 2045, 4096, 16) >= need(8, 2045, 4096, 16) >= need(4, 2045, 4096, 16) > 0
    r = random.Random(7)
    for _ in range(20000):
        channels, states = 8 * r.randint(1, 2048), r.choice([8, 16, 32, 64])
        batch, tokens = int(2 ** r.uniform(0, 10)), int(2 ** r.uniform(0, 15))
        less = need(r.randint(0, batch), r.randint(0, tokens), channels, states)
        assert less <= need(batch, tokens, channels, states) <= 32 << 20


@pytest.mark.parametrize("B,T,D", [(1, 8192, 2048), (4, 2045, 4096), (4, 896, 4096), (1, 600, 64)])
def test_scans_in_parts_want_their_workspace(gdn, B, T, D):  # noqa: F811
    lib = gdn._abi.load()
    need = gdn.ssm_workspace_bytes(B, T, D, 16)
    assert need > 0
    for lens in (None, FAKE):
        s = ctypes.byref(ssm(gdn, batch=B, num_tokens=T, channels=D, num_groups=1, u_strides=(T * D, D), seq_lens=lens))
        assert lib.gdn_ssm_scan(s, FAKE, need - 1, None, None) == BAD
        assert lib.gdn_ssm_scan(s, None, need, None, None) == BAD
        assert lib.gdn_ssm_scan(s, FAKE + 8, need, None, None) == NO


# ---- memory that a call writes and reads ----------------------------------------------------------------
# Distinct addresses for every operand, 2^30 apart; the calls below are all refused for what they share.
FAR = 1 << 30


def test_norm_refuses_shared_memory(gdn):  # noqa: F811
    lib = gdn._abi.load()
    x, residual, weight, o, scales = (FAR * i for i in range(1, 6))
    bf16 = dict(rows=4, width=256, x=x, x_stride=256, residual=residual, residual_stride=256, weight=weight, o=o)  # 512 bytes a row
    e4m3 = dict(bf16, o_type=2, scales=scales)
    shared = [dict(bf16, o=x + 512), dict(bf16, o=x - 1536), dict(bf16, o=x + 16), dict(bf16, x_stride=512, o=x), dict(bf16, x_stride=0, o=x),
              dict(bf16, x_type=1, o=x), dict(bf16, o=residual), dict(bf16, o=residual - 2032), dict(bf16, residual_stride=2048, o=residual + 3 * 4096),
              dict(bf16, o=weight + 512), dict(bf16, o=weight - 1536), dict(e4m3, o=x), dict(e4m3, scales=o + 1020), dict(e4m3, scales=o - 12),
              dict(e4m3, scales=x + 2044), dict(e4m3, scales=residual), dict(e4m3, scales=weight + 1020), dict(bf16, weight=residual + 512),
              dict(bf16, x=residual + 512), dict(bf16, x=residual - 512), dict(bf16, x=residual, x_stride=0), dict(bf16, x=residual, residual_type=1),
              dict(bf16, x=residual + 3 * 512 + 16), dict(bf16, x=residual - 3 * 512 - 16), dict(bf16, x_stride=512, x=residual + 1024, residual_stride=264),
              dict(bf16, x_stride=272, x=residual - 512 - 16, residual_stride=512)]
    for kw in shared:
        assert lib.gdn_add_rms_norm(ctypes.byref(norm(gdn, **kw)), None) == BAD, kw
        assert b"overlaps" in lib.gdn_last_error()


def test_convolution_refuses_shared_memory(gdn):  # noqa: F811
    lib = gdn._abi.load()
    x, w, bias, pool, slot, lens, o = (FAR * i for i in range(1, 8))
    # x: 2 requests of 4 rows of 128 bytes, 256 apart; pool: 3 rows of 384; o: 1024 bytes
    kw = dict(x=x, x_strides=(1024, 128), w=w, bias=bias, pool=pool, slot=slot, seq_lens=lens, o=o)
    shared = [dict(kw, o=x), dict(kw, o=x + 2048 + 3 * 256), dict(kw, o=x - 1008), dict(kw, o=x + 1024 - 128 - 1024), dict(kw, o=w + 1008), dict(kw, o=bias - 1008), dict(kw, o=pool + 1136),
              dict(kw, o=pool - 1008), dict(kw, slot=o + 1020), dict(kw, seq_lens=o), dict(kw, pool=x), dict(kw, pool=x + 3 * 256 + 112), dict(kw, pool=w),
              dict(kw, pool=bias + 240), dict(kw, slot=pool + 1148), dict(kw, seq_lens=pool)]
    for s in shared:
        assert lib.gdn_causal_conv(ctypes.byref(conv(gdn, **s)), None, None) == BAD, s
        assert b"overlaps" in lib.gdn_last_error()


def test_recurrence_refuses_shared_memory(gdn):  # noqa: F811
    lib = gdn._abi.load()
    names = ("u", "dt", "b", "c", "z", "a", "skip", "dt_bias", "state", "slot", "seq_lens", "y")
    at = {name: FAR * (i + 1) for i, name in enumerate(names)}
    # y: 2 requests of 4 rows of 128 bytes; state: 3 slots of 4096
    far = dict(b_strides=(128, 32, 16), c_strides=(128, 32, 16), z_strides=(512, 128))
    shared = [dict(y=at["u"] + 128), dict(y=at["dt"] - 1008), dict(y=at["z"]), dict(y=at["z"] + 1024 + 3 * 256 + 112), dict(y=at["b"] + 496), dict(y=at["c"] - 1008),
              dict(y=at["a"] + 4080), dict(y=at["skip"] + 240), dict(y=at["dt_bias"]), dict(slot=at["y"] + 1020), dict(seq_lens=at["y"] + 1016),
              dict(y=at["state"] + 3 * 4096 - 16), dict(state=at["u"] + 1008), dict(state=at["z"] + 1024), dict(state=at["b"]), dict(state=at["c"] - 3 * 4096 + 16),
              dict(state=at["a"] + 16), dict(skip=at["state"] + 4096), dict(dt_bias=at["state"] + 8192), dict(slot=at["state"] + 12284), dict(seq_lens=at["state"]),
              dict(y=at["u"], u_strides=(512, 64)), dict(y=at["u"], u_strides=(0, 64)), dict(y=at["u"], u_strides=(64, 128))]
    for kw in shared:
        s = ssm(gdn, **{**at, **far, **kw})
        assert lib.gdn_ssm_scan(ctypes.byref(s), None, 0, None, None) == BAD, kw
        assert b"overlaps" in lib.gdn_last_error()
    one = dict(num_tokens=1, seq_lens=None, u_strides=(64, 8), dt_strides=(64, 8))
    for kw in (dict(y=at["u"] + 16), dict(y=at["z"]), dict(state=at["dt"]), dict(y=at["b"])):
        assert lib.gdn_ssm_step(ctypes.byref(ssm(gdn, **{**at, **far, **one, **kw})), None, None) == BAD, kw
        assert b"overlaps" in lib.gdn_last_error()
    size = gdn.ssm_workspace_bytes(1, 2048, 64, 16)
    long = dict(batch=1, num_tokens=2048, num_slots=1, u_strides=(0, 64), dt_strides=(0, 64))
    for name in names:
        assert lib.gdn_ssm_scan(ctypes.byref(ssm(gdn, **{**at, **far, **long})), at[name] - size + 16, size, None, None) == BAD, name
        assert b"workspace overlaps" in lib.gdn_last_error()


# ---- the binding's errors ----------------------------------------------------------------------------------
def test_operands_of_any_number_of_dimensions_are_refused_by_name(selective):  # noqa: F811
    for call, tensors in calls(selective):
        for name, t in tensors.items():
            if name in ("slot", "seq_lens", "status", "workspace"):  # lists, of any dimensions
                continue
            for shape in ((), (8,), (2, 8), (2, 4, 8), (2, 4, 2, 8), (1, 2, 4, 2, 8)):
                if shape == tuple(t.shape):
                    continue
                with pytest.raises(ValueError, match=r"^\w+: .*\[|^\w+: .*\("):  # the operand, and what it should be
                    call({**tensors, name: On(shape, t.dtype)})
    assert selective.lib.calls == 0
