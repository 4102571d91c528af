"""The calls of selective state space layers at edges that the other tests leave out: quantised values next to a
border, single tokens that are not what they should be, states that grow, outputs in place of inputs."""
import importlib.util
import os

import pytest
import torch

from test_gpu_selective import BF16, E, E4M3, FP32, HALF, Layer, check_conv, gdn, gen, ints, randn  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- norm ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("rows,width,group", [(8191, 4096, 0), (8191, 4096, 128), (60000, 256, 128), (300, 4096, 0)])
def test_norm_stores_the_quotients_nearest_value(gdn, rows, width, group):  # noqa: F811
    """What is stored is e4m3(o / s), bit for bit, of the o and s that the call itself gives: a product with 1 / s is
    up to one and a half roundings off, which puts quotients next to a border on its other side."""
    g = gen(rows + group)
    x, weight = randn(g, rows, width, dtype=BF16), 1 + 0.1 * randn(g, width)
    o, q = torch.empty(rows, width, device="cuda"), torch.empty(rows, width, dtype=E4M3, device="cuda")
    scales = torch.empty(rows, -(-width // (group or width)), device="cuda")
    gdn.add_rms_norm(x, o, weight=weight)
    gdn.add_rms_norm(x, q, weight=weight, scales=scales, group=group)
    tops = o.abs().unflatten(1, (scales.shape[1], -1)).amax(-1)
    assert torch.equal(scales, tops / torch.full_like(tops, 448))  # by a number torch multiplies with its inverse
    want = (o.unflatten(1, (scales.shape[1], -1)) / scales[..., None]).flatten(1).to(E4M3)
    wrong = q.view(torch.uint8) != want.view(torch.uint8)
    assert not wrong.any(), (int(wrong.sum()), wrong.numel())


@pytest.mark.parametrize("group", [0, 128])
def test_norm_of_outputs_past_fp32(gdn, group):  # noqa: F811
    """An output that weight makes infinite makes its scale infinite: itself NaN, the others of that scale 0."""
    x, weight = torch.ones(2, 256, device="cuda"), torch.ones(256, device="cuda")
    x[0, 3], weight[3] = 100.0, 3e38
    x[1, 3] = 1e-30
    q, scales = torch.empty(2, 256, dtype=E4M3, device="cuda"), torch.empty(2, 2 if group else 1, device="cuda")
    gdn.add_rms_norm(x, q, weight=weight, scales=scales, group=group)
    got, first = q.float(), group or 256
    assert scales[0, 0] == float("inf") and torch.isfinite(scales[1]).all()
    assert got[0, 3].isnan() and (got[0, :3] == 0).all() and (got[0, 4:first] == 0).all() and (got[0, first:] == 448).all()
    # 1e-30 times 3e38 is 3e8, beside which 1 is below half of the least value, 2^-10
    assert got[1, 3] == 448 and (got[1, :3] == 0).all() and (got[1, 4:first] == 0).all() and (got[1, first:] == 448).all()


def test_norm_of_the_most_rows(gdn):  # noqa: F811
    """2^31 - 1 rows, the most that a call can name: four of them a CTA, counted past 32 bits."""
    rows = 2 ** 31 - 1
    x = randn(gen(9), 1, 8, dtype=BF16)
    q, scales = torch.zeros(rows, 8, dtype=E4M3, device="cuda"), torch.zeros(rows, dtype=FP32, device="cuda")
    gdn.add_rms_norm(x.expand(rows, 8), q, scales=scales)
    one, scale = torch.empty(1, 8, dtype=E4M3, device="cuda"), torch.empty(1, device="cuda")
    gdn.add_rms_norm(x, one, scales=scale)
    whole, want = q.view(torch.int64).flatten(), one.view(torch.int64).flatten()
    assert all((part == want).all() for part in whole.split(2 ** 28)) and all((part == scale).all() for part in scales.split(2 ** 28))


# ---- convolution of single tokens ---------------------------------------------------------------------
# From 100000 vectors of eight channels on a thread takes four requests (323 x 2568 are 103683 vectors): the last
# group of a batch may be shorter, and where rows are no multiple of 256 channels a warp's lanes are of several groups.
@pytest.mark.parametrize("B,D", [(321, 4096), (322, 2568), (323, 4104), (513, 1560), (323, 2568), (3, 64), (5, 264)])
@pytest.mark.parametrize("kind", [BF16, FP32])
def test_conv_of_single_tokens(gdn, kind, B, D):  # noqa: F811
    rows = list(range(B + 2))[::-1]
    assert check_conv(gdn, B, 1, D, kind, seed=B) == 0
    assert check_conv(gdn, B, 1, D, kind, slot=[-1 - i if i % 3 == 1 else rows[i] for i in range(B)], silu=False, wide=2) == 0
    assert check_conv(gdn, B, 1, D, kind, lens=[i % 5 != 2 for i in range(B)], slot=rows[:B], bias=False) == 0
    # what is wrong leaves its request alone and none of its group: the last request, the first, one in the middle
    bad = [rows[i] for i in range(B)]
    bad[-1], bad[0] = B + 2, 2 ** 31 - 1
    assert check_conv(gdn, B, 1, D, kind, slot=bad) == gdn.STATUS_BAD_SLOT
    lens = [1] * B
    lens[-1], lens[B // 2] = 2, -1
    assert check_conv(gdn, B, 1, D, kind, lens=lens, slot=rows[:B]) == gdn.STATUS_BAD_LEN
    lens[0], bad[-1] = 0, -7
    assert check_conv(gdn, B, 1, D, kind, lens=lens, slot=bad) == gdn.STATUS_BAD_SLOT | (gdn.STATUS_BAD_LEN if bad[B // 2] >= 0 else 0)
    assert check_conv(gdn, B, 1, D, kind, lens=[2] * B, slot=[-1] * B) == 0


# ---- recurrence -------------------------------------------------------------------------------------
def test_one_workspace_for_all_admissions(gdn):  # noqa: F811
    """A buffer of the largest batch serves smaller ones, which are cut into more parts, and none writes past it."""
    D, N, most = 512, 16, (48, 700)
    size = gdn.ssm_workspace_bytes(*most, D, N)
    room = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    for i, (B, T, lens) in enumerate([(48, 700, None), (4, 700, None), (1, 700, None), (16, 512, [512, 3] * 8), (3, 100, None), (1, 64, [64]), (2, 20, None),
                                      (48, 700, [700 - 14 * j for j in range(48)])]):
        layer, alone = (Layer(gdn, B, T, D, N, kind=(BF16, FP32)[i % 2], lens=lens, seed=i) for _ in range(2))
        assert alone.workspace.numel() <= max(size, 16)
        alone.call()
        layer.workspace = room[:size]
        layer.call()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, alone.y) and torch.equal(layer.state, alone.state) and (room[size:] == 77).all()


def test_scans_of_whole_prompts_need_no_workspace(gdn):  # noqa: F811
    for B, T, D in ((2, 20, 64), (64, 300, 4096)):
        layer, alone = (Layer(gdn, B, T, D, 16, seed=4) for _ in range(2))
        alone.call()
        layer.workspace = None
        layer.call()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, alone.y) and torch.equal(layer.state, alone.state)


class Exact(Layer):
    """A Layer whose tolerances count what the kernels round, and nothing for joining parts where there are none."""

    def want(self):
        D, N, T = self.D, self.N, self.T
        # A prompt of at most 32 positions is never cut. Of others the steps of a part are summed, each sum rounded.
        joined = T * E if T > 32 else 0.0
        live = [b for b in range(self.B) if 0 <= self.slot[b] < self.num_slots and 0 <= self.lens[b] <= T]
        rows, lens = torch.tensor([self.slot[b] for b in live], device="cuda"), ints([self.lens[b] for b in live])
        u, dt, b, c = (torch.nan_to_num(x[live].double()) for x in (self.u, self.dt, self.b, self.c))
        x = dt + (0 if self.bias is None else self.bias.double())
        # Its argument is off by a rounding of dt and one of the sum, over which softplus has a relative slope of at
        # most 1 + |x|; its exponential, series or logarithm and their sum are off by 8 roundings.
        s = torch.nn.functional.softplus(x, threshold=1e3) if self.softplus else x
        ds = (9 + x.abs() + dt.abs()) * E if self.softplus else torch.full_like(x, E)
        a, state, off = self.a.double(), self.state.double(), torch.zeros(self.state.shape, dtype=torch.float64, device="cuda")
        h, err = state[rows].clone(), off[rows].clone()
        y, off_y = torch.full((self.B, T, D), float("nan"), dtype=torch.float64, device="cuda"), torch.zeros(self.B, T, D, dtype=torch.float64, device="cuda")
        for t in range(T):
            on = (t < lens)[:, None]
            st, dst, ut = s[:, t, :, None], ds[:, t, :, None], u[:, t, :, None]
            bt, ct = (v[:, t].repeat_interleave(D // self.G, 1) for v in (b, c))
            decay, put = torch.exp(st * a), st * ut * bt
            # two products and log2(e) make the exponent; 2^-22.5 of the result is the exponential's own
            wrong = (st * a).abs() * (2.25 * E + dst + joined) + 3 * E
            new = decay * h + put
            err_new = decay * (err + h.abs() * wrong) + put.abs() * (dst + 2 * E) + new.abs() * E
            h, err = torch.where(on[..., None], new, h), torch.where(on[..., None], err_new, err)
            row, far = (h * ct).sum(-1), (err * ct.abs()).sum(-1) + (h * ct).abs().sum(-1) * (N // 4 + 4) * E
            if self.skip is not None:
                own = self.skip.double() * u[:, t]
                row, far = row + own, far + E * (row + own).abs()
            if self.z is not None:
                z = torch.nan_to_num(self.z[live][:, t].double())
                gate = z * torch.sigmoid(z)
                row, far = row * gate, far * gate.abs() + 8 * E * (row * gate).abs()
            y[live, t] = torch.where(on, row, torch.nan)
            off_y[live, t] = (far + row.abs() * HALF[self.kind]) * 1.01 + 1e-35
        state[rows], off[rows] = h, err * 1.01 + 1e-35
        return y, off_y, state, off

    def step(self):
        one = lambda x: None if x is None else x[:, 0]  # noqa: E731
        y = self.y[:, 0].contiguous()
        self.gdn.ssm_step(one(self.u), one(self.dt), self.a, one(self.b), one(self.c), self.state, ints(self.slot), y, z=one(self.z), skip=self.skip,
                          dt_bias=self.bias, softplus=self.softplus, status=self.status)
        self.y = y[:, None]


@pytest.mark.parametrize("kw", [dict(), dict(z=False), dict(skip=False), dict(bias=False), dict(softplus=False), dict(softplus=False, bias=False, z=False, skip=False)])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("kind", [BF16, FP32])
def test_step_and_short_scans_to_their_roundings(gdn, kind, N, kw):  # noqa: F811
    for B, T, D, G in ((1, 1, 2048, 1), (37, 1, 264, 3), (2, 1, 72, 9)):
        layer = Exact(gdn, B, T, D, N, G, kind, seed=N + B, **kw)
        assert layer.check(layer.step) == 0
    for B, T, D, G, lens in ((3, 1, 72, 1, None), (2, 17, 264, 1, None), (5, 32, 64, 4, [32, 8, 7, 1, 0]), (25, 21, 2048, 1, None)):
        assert Exact(gdn, B, T, D, N, G, kind, lens, seed=N + T, **kw).check() == 0


@pytest.mark.parametrize("B,T,D,N,lens", [(1, 64, 2048, 16, [64]), (1, 300, 264, 32, [300]), (16, 260, 1024, 16, [260] * 16), (40, 96, 2048, 8, [96] * 39 + [5]), (3, 500, 64, 64, None)])
@pytest.mark.parametrize("kind", [BF16, FP32])
def test_scans_to_their_roundings(gdn, kind, B, T, D, N, lens):  # noqa: F811
    assert Exact(gdn, B, T, D, N, 1, kind, lens, seed=T).check() == 0


@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_scan_of_states_that_grow_keeps_zeros(gdn, N):  # noqa: F811
    """With a > 0 the product of a part's decays passes fp32 (e^4 a position), and a state of zero stays zero."""
    B, T, D = 1, 600, 64
    u = torch.zeros(B, T, D, device="cuda")
    u[:, T - 3:] = randn(gen(N), B, 3, D)
    dt, a = torch.full_like(u, 2.0), torch.full((D, N), 2.0, device="cuda")
    b, c = randn(gen(N + 1), B, T, 1, N), randn(gen(N + 2), B, T, 1, N)
    state, y = torch.zeros(2, D, N, device="cuda"), torch.full_like(u, 7.0)
    workspace = torch.empty(max(16, gdn.ssm_workspace_bytes(B, T, D, N)), dtype=torch.uint8, device="cuda")
    gdn.ssm_scan(u, dt, a, b, c, state, ints([1]), y, workspace, softplus=False)
    h = torch.zeros(D, N, dtype=torch.float64, device="cuda")
    assert (y[:, :T - 3] == 0).all()
    for t in range(T - 3, T):
        h = h * torch.exp(torch.tensor(4.0, dtype=torch.float64)) + 2 * u[0, t].double()[:, None] * b[0, t].double()
        want = (h * c[0, t].double()).sum(-1)
        size = (h.abs() * c[0, t].double().abs()).sum(-1)  # every factor and sum is off by some roundings of what it adds to
        assert ((y[0, t].double() - want).abs() <= size * 2.0 ** -18).all()
    assert ((state[1].double() - h).abs() <= 2.0 ** -18 * h.abs().max()).all()


# ---- outputs in place of inputs -------------------------------------------------------------------------
@pytest.mark.parametrize("rows,width", [(1, 2048), (5, 256), (300, 4096), (4200, 4104)])
@pytest.mark.parametrize("kind", [BF16, FP32])
def test_norm_in_place(gdn, rows, width, kind):  # noqa: F811
    """The bits of separate tensors: o in x, x the residual itself, x and residual side by side in rows of both."""
    g = gen(rows)
    x, old, weight = randn(g, rows, width, dtype=kind), randn(g, rows, width, dtype=kind), randn(g, width)
    want, sums = torch.empty_like(x), old.clone()
    gdn.add_rms_norm(x, want, residual=sums, weight=weight)
    o, residual = x.clone(), old.clone()
    gdn.add_rms_norm(o, o, residual=residual, weight=weight)
    assert torch.equal(o, want) and torch.equal(residual, sums)
    both = torch.cat([x, old], 1)
    o = torch.empty_like(x)
    gdn.add_rms_norm(both[:, :width], o, residual=both[:, width:], weight=weight)
    assert torch.equal(o, want) and torch.equal(both[:, :width], x) and torch.equal(both[:, width:], sums)
    sums = x.clone()
    gdn.add_rms_norm(x, want, residual=sums, weight=weight)
    gdn.add_rms_norm(x, o, residual=x, weight=weight)
    assert torch.equal(o, want) and torch.equal(x, sums)


@pytest.mark.parametrize("B,T,D,lens", [(3, 1, 264, None), (2, 21, 64, None), (2, 900, 264, None), (3, 700, 64, [700, 0, 333])])
def test_recurrence_in_place(gdn, B, T, D, lens):  # noqa: F811
    for name in ("u", "dt", "z"):
        first, second = (Layer(gdn, B, T, D, 16, kind=BF16, lens=lens, seed=T) for _ in range(2))
        for layer in (first, second):
            layer.z = layer.z.contiguous()
        first.y = getattr(first, name).clone()
        second.y = getattr(second, name)
        first.call(), second.call()
        torch.cuda.synchronize()
        assert torch.equal(first.y.view(torch.int16), second.y.view(torch.int16)) and torch.equal(first.state, second.state)  # NaN past a prompt's end


def test_step_in_place(gdn):  # noqa: F811
    B, D, N = 300, 264, 16
    for name in ("u", "dt", "z"):
        g = gen(5)
        x = {k: randn(g, B, D, dtype=BF16) for k in ("u", "dt", "z")}
        a, b, c, state = -torch.rand(D, N, generator=g, device="cuda"), randn(g, B, 1, N, dtype=BF16), randn(g, B, 1, N, dtype=BF16), randn(g, B, D, N)
        slot = torch.arange(B, dtype=torch.int32, device="cuda")
        y, again = torch.empty_like(x["u"]), state.clone()
        gdn.ssm_step(x["u"], x["dt"], a, b, c, state, slot, y, z=x["z"])
        gdn.ssm_step(x["u"], x["dt"], a, b, c, again, slot, x[name], z=x["z"])
        assert torch.equal(x[name], y) and torch.equal(again, state)


def test_outputs_between_the_rows_of_inputs(gdn):  # noqa: F811
    """Memory that rows of an input leave between them is no part of it."""
    g = gen(6)
    T, D = 40, 64
    room = randn(g, 2, 3 * T * D, dtype=BF16)
    x, o = room[:, :T * D].unflatten(1, (T, D)), room[0, T * D:].view(2, T, D)
    w, pool = randn(g, D, 4), randn(g, 2, D, 3, dtype=BF16)
    want, rows = torch.empty(2, T, D, dtype=BF16, device="cuda"), pool.clone()
    gdn.causal_conv(x.contiguous(), w, rows, ints([1, 0]), want)
    gdn.causal_conv(x, w, pool, ints([1, 0]), o)
    assert torch.equal(o, want) and torch.equal(pool, rows)
    with pytest.raises(gdn.GDNError, match="overlaps"):
        gdn.causal_conv(x, w, pool, ints([1, 0]), room.view(-1)[T * D + 8:3 * T * D + 8].view(2, T, D))  # its last row meets the second request's first


# ---- the example's stack -----------------------------------------------------------------------------------
@pytest.mark.parametrize("layers", [0, 1, 2, 5])
def test_hybrid_stacks_of_any_depth(gdn, layers):  # noqa: F811
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    hybrid = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(hybrid)
    model = hybrid.HybridDecoder(3, heads=2, heads_kv=1, layers=layers, max_len=128)
    model.admit([5, 1, 64])
    model.step()
    model.capture()
    model.step()
    torch.cuda.synchronize()
    assert model.status.item() == 0 and model.length.tolist() == [7, 3, 66] and torch.isfinite(model.y).all()
    assert torch.equal(model.y, model.x) == (layers == 0)
