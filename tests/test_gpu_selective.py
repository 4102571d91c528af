"""The calls of selective state space layers against plain sums in 64 bits, with tolerances that
follow the roundings of each output element."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E = 2.0 ** -24  # half a step of fp32, relative
HALF = {BF16: 2.0 ** -8, FP32: E}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def gdn():
    from linear_attention_decode_gdn_gb300 import build
    build.build()
    import linear_attention_decode_gdn_gb300 as g
    return g


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=FP32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def close(got, want, tolerance):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    far = (got - want).abs() - tolerance
    far[(got == want) | torch.isnan(want)] = 0
    worst = int(far.argmax()) if far.numel() else 0
    assert far.numel() == 0 or float(far.max()) <= 0, (got.flatten()[worst].item(), want.flatten()[worst].item(),
                                                       tolerance.expand(got.shape).flatten()[worst].item(), worst)


# ---- norm ---------------------------------------------------------------------------------------
def norm_want(x, residual, weight, eps):
    r = x.double() if residual is None else x.double() + residual.double()
    y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    return r, y if weight is None else y * weight.double()


def check_norm(gdn, x, residual, weight, out, group=0, eps=1e-6):
    rows, width = x.shape
    r, y = norm_want(x, residual, weight, eps)
    o = torch.full((rows, width), 3.0, device="cuda").to(out)
    wide = group or width
    scales = torch.full((rows, -(-width // wide)), NAN, device="cuda") if out is E4M3 else None
    gdn.add_rms_norm(x, o, residual=residual, weight=weight, eps=eps, scales=scales, group=group)
    torch.cuda.synchronize()
    if residual is not None:  # one rounding of the fp32 sum, and its own
        close(residual, r, r.abs() * (HALF[residual.dtype] + (E if residual.dtype is BF16 else 0)) * 1.01 + 1e-40)
    # The sum of squares: 16 in a thread, five rounds of lanes, five of warps, each half of it under the
    # root; then mean, eps, root, quotient, two products and the first sum. Below 32 roundings in all.
    off = 32 * E
    if out is not E4M3:
        close(o, y, y.abs() * (HALF[out] + off) * 1.01 + 1e-37)
        return
    pad = torch.nn.functional.pad(y, (0, -width % wide)).unflatten(-1, (-1, wide))
    top = pad.abs().amax(-1).clamp(min=1e-30) / 448
    close(scales, top, top * (off + 3 * E))
    want = (pad / scales.double()[..., None]).flatten(1)[:, :width].clamp(-448, 448)
    # half a step of e4m3: 2^-4 of the value, or half of the least value there is, 2^-9
    close(o.float(), want, (want.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) + want.abs() * (off + 4 * E) * 1.01)


@pytest.mark.parametrize("rows,width", [(1, 8), (3, 24), (5, 128), (2, 136), (257, 1024), (3, 2056), (66, 4096), (700, 4104), (9, 6144), (2, 8192), (3, 12008), (2, 16384),
                                        (609, 8), (700, 256), (700, 264), (613, 1024), (610, 1032), (640, 16384), (4100, 4096), (1025, 16384)])
@pytest.mark.parametrize("kind,res", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16), (BF16, None), (FP32, None)])
def test_norm(gdn, rows, width, kind, res):
    g = gen(rows * 31 + width)
    for out, group in ((BF16, 0), (FP32, 0), (E4M3, 0), (E4M3, 128)):
        x = randn(g, rows, width, dtype=kind)
        residual = None if res is None else (4 * randn(g, rows, width)).to(res)
        check_norm(gdn, x, residual, 1 + 0.2 * randn(g, width), out, group)


def test_norm_rows_in_strides_and_no_weight(gdn):
    g = gen(5)
    wide, room = randn(g, 37, 3 * 520, dtype=BF16), randn(g, 37, 2 * 520, dtype=FP32)
    before_x, before = wide.clone(), room.clone()
    check_norm(gdn, wide[:, 520:1040], room[:, 520:], None, E4M3, 128)
    assert torch.equal(wide, before_x) and torch.equal(room[:, :520], before[:, :520])
    check_norm(gdn, wide[:1, 520:1040], None, None, FP32)
    # one row for all: a stride of zero
    check_norm(gdn, wide[:1, :520].expand(7, -1), room[:7, :520], None, BF16)


def test_norm_of_zeros_and_of_no_numbers(gdn):
    for out, group in ((BF16, 0), (E4M3, 0), (E4M3, 128)):
        check_norm(gdn, torch.zeros(3, 264, device="cuda"), None, None, out, group)
        check_norm(gdn, torch.full((3, 264), 1e-25, device="cuda"), None, None, out, group, eps=1.0)
    x = randn(gen(8), 4, 264, dtype=BF16)
    x[1, 200], x[2, 3], x[3, 5], x[3, 6] = NAN, INF, -INF, 3e38
    r, y = norm_want(x, None, None, 1e-6)
    for out in (BF16, FP32):
        o = torch.empty(4, 264, dtype=out, device="cuda")
        gdn.add_rms_norm(x, o)
        close(o, y, y.abs() * (HALF[out] + 32 * E) * 1.01)
    for group in (0, 128):
        o, scales = torch.empty(4, 264, dtype=E4M3, device="cuda"), torch.empty(4, 3 if group else 1, device="cuda")
        gdn.add_rms_norm(x, o, scales=scales, group=group)
        value = o.float() * scales.repeat_interleave(group or 264, 1)[:, :264]
        assert not value[0].isnan().any() and value[1].isnan().all()
        n = group or 264  # the infinity's group
        assert value[2:, :n].isnan().all() and (value[2:, n:] == 0).all()


def test_norm_sum_past_fp32(gdn):
    x = torch.full((2, 64), 1e20, device="cuda")
    o = torch.empty_like(x)
    gdn.add_rms_norm(x, o)
    assert (o == 0).all()


# ---- convolution ----------------------------------------------------------------------------------
def conv_want(x, w, bias, pool, slot, lens, silu, num_slots):
    """o (NaN where it is to be left alone), what its sum weighs, and the pool, in 64 bits."""
    B, T, D = x.shape
    o, size, rows = torch.full((B, T, D), NAN, dtype=torch.float64, device="cuda"), torch.zeros(B, T, D, dtype=torch.float64, device="cuda"), pool.clone()
    for b, (row, n) in enumerate(zip(slot, lens)):
        if row < 0 or row >= num_slots or n < 0 or n > T:
            continue
        line = torch.cat([pool[row].T, x[b, :n]])
        wide, taps = line.double(), w.double()
        parts = [wide[j:j + n] * taps[:, j] for j in range(4)]
        total = sum(parts) + (0 if bias is None else bias.double())
        size[b, :n] = sum(p.abs() for p in parts) + (0 if bias is None else bias.double().abs())
        o[b, :n] = total * torch.sigmoid(total) if silu else total
        rows[row] = line[n:].T
    return o, size, rows


def check_conv(gdn, B, T, D, kind, lens=None, slot=None, seed=1, silu=True, bias=True, wide=1, strange=()):
    g = gen(seed)
    num_slots = B + 2
    x = randn(g, B, T, wide * D, dtype=kind)[..., (wide - 1) * D:]
    slot = torch.randperm(num_slots, generator=torch.Generator().manual_seed(seed))[:B].tolist() if slot is None else slot
    n = [T] * B if lens is None else lens
    for b, k in enumerate(n):
        x[b, max(k, 0):] = NAN  # never read
    w, bs = 0.5 * randn(g, D, 4), 0.3 * randn(g, D) if bias else None
    pool = randn(g, num_slots, D, 3, dtype=kind)
    want, size, rows = conv_want(x, w, bs, pool, slot, n, silu, num_slots)
    o, status = torch.full((B, T, D), 77.0, dtype=kind, device="cuda"), ints([0])
    gdn.causal_conv(x, w, pool, ints(slot), o, bias=bs, silu=silu, seq_lens=None if lens is None else ints(lens), status=status)
    torch.cuda.synchronize()
    alone = want.isnan()
    assert (o[alone] == 77).all()
    assert torch.equal(pool, rows)
    # five roundings of the sum, times SiLU's slope (below 1.1), and SiLU itself: exponential, sum, quotient
    tolerance = want.abs() * (HALF[kind] + 8 * E) * 1.01 + 5.5 * E * size * 1.01 + 1e-37
    want[alone], tolerance[alone] = 77.0, 0
    close(o, want, tolerance)
    return status.item()


@pytest.mark.parametrize("kind", [BF16, FP32])
@pytest.mark.parametrize("B,T,D,lens", [
    (1, 1, 8, None), (5, 1, 6144, None), (300, 1, 264, None), (3, 2, 64, None), (2, 3, 40, None), (4, 31, 264, None), (2, 33, 2048, None), (3, 517, 72, None),
    (60, 300, 2048, [0, 1, 2, 3, 126, 127, 128, 129, 130, 131, 255, 256, 257, 259, 299] * 4), (320, 1, 4096, [1, 0, 1, 1, 0] * 64), (320, 1, 4096, None),
    (7, 9, 64, [0, 1, 2, 3, 4, 8, 9]), (6, 130, 136, [0, 1, 32, 33, 65, 130]), (3, 1, 64, [0, 1, 1]), (1, 4099, 512, None)])
def test_conv(gdn, kind, B, T, D, lens):
    assert check_conv(gdn, B, T, D, kind, lens) == 0
    assert check_conv(gdn, B, T, D, kind, lens, silu=False, bias=False, wide=2, seed=2) == 0


def test_conv_skips_padding_and_what_is_wrong(gdn):
    assert check_conv(gdn, 4, 40, 64, BF16, [40, 7, 0, 33], slot=[-1, 2, -5, 0]) == 0
    assert check_conv(gdn, 3, 40, 64, FP32, slot=[1, 5, 0]) == gdn.STATUS_BAD_SLOT
    assert check_conv(gdn, 3, 40, 64, BF16, [3, -1, 40], slot=[1, 2, 0]) == gdn.STATUS_BAD_LEN
    assert check_conv(gdn, 3, 40, 64, BF16, [3, 41, 40], slot=[1, 2, 0]) == gdn.STATUS_BAD_LEN
    assert check_conv(gdn, 3, 40, 64, BF16, [3, 41, 40], slot=[1, -1, 0]) == 0


@pytest.mark.parametrize("kind", [BF16, FP32])
def test_conv_of_large_values(gdn, kind):
    """SiLU far from zero on either side, and infinities, which reach four positions."""
    g = gen(4)
    x, w = (300 * randn(g, 2, 40, 64)).to(kind), randn(g, 64, 4)
    for silu in (True, False):
        pool = randn(g, 3, 64, 3, dtype=kind)
        want, size, rows = conv_want(x, w, None, pool, [2, 0], [40, 40], silu, 3)
        o = torch.empty_like(x)
        gdn.causal_conv(x, w, pool, ints([2, 0]), o, silu=silu)
        close(o, want, want.abs() * (HALF[kind] + 8 * E) * 1.01 + 5.5 * E * size * 1.01 + 1e-35)
        assert torch.equal(pool, rows)
    x[0, 20, 5], x[1, 3, 7] = INF, NAN
    o = torch.empty_like(x)
    gdn.causal_conv(x, w, torch.zeros(3, 64, 3, dtype=kind, device="cuda"), ints([2, 0]), o, silu=False)
    bad = ~torch.isfinite(o)
    where = torch.zeros_like(bad)
    where[0, 20:24, 5], where[1, 3:7, 7] = True, True
    assert torch.equal(bad, where)


@pytest.mark.parametrize("kind", [BF16, FP32])
def test_conv_in_pieces(gdn, kind):
    """A prompt in pieces, and then token by token, gives the bits of the whole."""
    g = gen(3)
    B, T, D = 3, 75, 136
    x, w, bias = randn(g, B, T, D, dtype=kind), 0.5 * randn(g, D, 4), 0.1 * randn(g, D)
    slot = ints([2, 0, 3])
    pool = randn(g, 4, D, 3, dtype=kind)
    pieces = pool.clone()
    whole = torch.empty_like(x)
    gdn.causal_conv(x, w, pool, slot, whole, bias=bias)
    at = 0
    for n in (1, 2, 40, 1, 1, 3, 26, 1):
        part = torch.empty(B, n, D, dtype=kind, device="cuda")
        if n == 1:
            part = part[:, 0].contiguous()
            gdn.causal_conv(x[:, at], w, pieces, slot, part, bias=bias)
            part = part[:, None]
        else:
            gdn.causal_conv(x[:, at:at + n], w, pieces, slot, part, bias=bias)
        assert torch.equal(part, whole[:, at:at + n])
        at += n
    assert at == T and torch.equal(pool, pieces)


# ---- recurrence -------------------------------------------------------------------------------------
class Layer:
    """Inputs of a scan, and the recurrence in 64 bits with what each element may be off by."""

    def __init__(self, gdn, B, T, D, N, G=1, kind=BF16, lens=None, slot=None, seed=1, z=True, skip=True, bias=True, softplus=True, step=(0.001, 0.1)):
        g = gen(seed)
        self.gdn, self.B, self.T, self.D, self.N, self.G, self.kind, self.softplus = gdn, B, T, D, N, G, kind, softplus
        self.num_slots = B + 2
        self.u, self.dt = randn(g, B, T, D, dtype=kind), (0.5 * randn(g, B, T, D)).to(kind)
        mixed = randn(g, B, T, 16 + 2 * G * N, dtype=kind)
        self.b, self.c = mixed[..., 16:16 + G * N].unflatten(-1, (G, N)), mixed[..., 16 + G * N:].unflatten(-1, (G, N))
        self.z = randn(g, B, T, 2 * D, dtype=kind)[..., D:] if z else None
        self.a = -torch.arange(1, N + 1, device="cuda").float() * torch.exp(0.2 * randn(g, D, N))
        self.skip = 1 + 0.2 * randn(g, D) if skip else None
        s = torch.exp(torch.rand(D, generator=g, device="cuda") * torch.log(torch.tensor(step[1] / step[0])) + torch.log(torch.tensor(step[0])))
        self.bias = s + torch.log(-torch.expm1(-s)) if bias else None
        if not softplus:  # the step itself
            self.dt = (self.dt.float().abs() * 0.1).to(kind)
            self.bias = s if bias else None
        self.state = randn(g, self.num_slots, D, N)
        self.slot = torch.randperm(self.num_slots, generator=torch.Generator().manual_seed(seed))[:B].tolist() if slot is None else slot
        self.lens = [T] * B if lens is None else lens
        self.given = lens is not None
        for b, n in enumerate(self.lens):
            for x in (self.u, self.dt, self.b, self.c) + ((self.z,) if z else ()):
                x[b, max(n, 0):] = NAN  # never read
        self.y = torch.full((B, T, D), 77.0, dtype=kind, device="cuda")
        self.status = ints([0])
        size = gdn.ssm_workspace_bytes(B, T, D, N)
        self.workspace = torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        self.gdn.ssm_scan(self.u, self.dt, self.a, self.b, self.c, self.state, ints(self.slot), self.y, self.workspace, z=self.z, skip=self.skip,
                          dt_bias=self.bias, softplus=self.softplus, seq_lens=ints(self.lens) if self.given else None, status=self.status,
                          stream=stream)

    def want(self):
        """y and its tolerance, the pool and its tolerance; y NaN where it is to be left alone."""
        D, N, G, T = self.D, self.N, self.G, self.T
        live = [b for b in range(self.B) if 0 <= self.slot[b] < self.num_slots and 0 <= self.lens[b] <= T]
        y = torch.full((self.B, T, D), NAN, dtype=torch.float64, device="cuda")
        off_y = torch.zeros_like(y)
        state, off = self.state.double(), torch.zeros(self.state.shape, dtype=torch.float64, device="cuda")
        if not live:
            return y, off_y, state, off
        rows, lens = torch.tensor([self.slot[b] for b in live], device="cuda"), ints([self.lens[b] for b in live])
        u, dt, b, c = (torch.nan_to_num(x[live].double()) for x in (self.u, self.dt, self.b, self.c))
        x = dt + (0 if self.bias is None else self.bias.double())
        # the step: the sum with the bias is rounded once, where softplus falls by at most its relative slope |x| + 1;
        # softplus itself (exponential, quotient, series) is off by 8 roundings
        s = torch.nn.functional.softplus(x, threshold=1e3) if self.softplus else x
        ds = (8 + x.abs() + 1) * E if self.softplus else torch.full_like(x, E)
        a, h, size, err = self.a.double(), state[rows].clone(), state[rows].abs(), torch.zeros_like(state[rows])
        # Parts of a prompt may be scanned apart and joined by exp(a sum s): the sum of up to 2048 steps, rounded
        # each time, is off by as much of itself, which is |s a| of each step.
        joined = 2048 * E
        for t in range(T):
            st, ut, dst = s[:, t, :, None], u[:, t, :, None], ds[:, t, :, None]
            bt, ct = (v[:, t].repeat_interleave(D // G, 1) for v in (b, c))
            decay, put = torch.exp(st * a), st * ut * bt
            # exp: two roundings of its argument, the step's own, and 2^-22 of the result; the sum's rounding
            wrong = (st * a).abs() * (3 * E + dst + joined) + 4 * E + E
            new = decay * h + put
            size_new = decay * size + put.abs()
            err_new = decay * err + decay * size * wrong + put.abs() * (dst + 4 * E) + size_new * E
            on = (t < lens)[:, None, None]
            h, size, err = torch.where(on, new, h), torch.where(on, size_new, size), torch.where(on, err_new, err)
            row = (h * ct).sum(-1)
            weight = (size * ct.abs()).sum(-1)
            wrong_row = (err * ct.abs()).sum(-1) + weight * (N // 4 + 4) * E
            if self.skip is not None:
                row, wrong_row = row + self.skip.double() * u[:, t], wrong_row + 2 * E * (row.abs() + (self.skip.double() * u[:, t]).abs())
            if self.z is not None:
                z = torch.nan_to_num(self.z[live][:, t].double())
                gate = z * torch.sigmoid(z)
                row, wrong_row = row * gate, wrong_row * gate.abs() + 8 * E * (row * gate).abs()
            on = (t < lens)[:, None]
            y[live, t] = torch.where(on, row, NAN)
            off_y[live, t] = wrong_row * 1.01 + row.abs() * HALF[self.kind] * 1.01 + 1e-35
        state[rows], off[rows] = h, err * 1.01 + 1e-35
        return y, off_y, state, off

    def check(self, call=None):
        y, off_y, state, off = self.want()
        untouched = y.isnan()
        (call or self.call)()
        torch.cuda.synchronize()
        assert (self.y[untouched] == 77).all()
        y[untouched], off_y[untouched] = 77.0, 0
        close(self.y, y, off_y)
        close(self.state, state, off)
        return self.status.item()


@pytest.mark.parametrize("kind", [BF16, FP32])
@pytest.mark.parametrize("B,T,D,N,G,lens", [
    (1, 1, 8, 8, 1, None), (2, 2, 64, 16, 1, None), (3, 17, 40, 16, 1, None), (2, 33, 264, 8, 1, None), (2, 40, 72, 32, 3, None), (1, 64, 64, 64, 4, None),
    (2, 100, 128, 16, 16, None), (9, 70, 64, 16, 2, [0, 1, 2, 15, 16, 17, 31, 32, 70]), (1, 1021, 2048, 16, 1, None), (2, 700, 136, 64, 1, [700, 513]),
    (1, 2500, 96, 8, 1, None), (3, 1300, 64, 32, 2, [1300, 1, 0]), (12, 200, 64, 16, 1, [0, 1, 8, 31, 32, 33, 40, 63, 64, 65, 199, 200]),
    (25, 21, 2048, 16, 1, None), (24, 40, 512, 64, 4, [40, 3, 39, 8, 9, 0] * 4), (50, 70, 4096, 8, 1, None)])
def test_scan(gdn, kind, B, T, D, N, G, lens):
    assert Layer(gdn, B, T, D, N, G, kind, lens).check() == 0


def test_scan_without_the_optional_parts(gdn):
    for i, kw in enumerate((dict(z=False), dict(skip=False), dict(bias=False), dict(softplus=False), dict(z=False, skip=False, bias=False, softplus=False))):
        assert Layer(gdn, 2, 90, 72, 16, kind=(BF16, FP32)[i % 2], seed=i, **kw).check() == 0


def test_scan_with_long_and_short_memories(gdn):
    """Steps of 1e-5 keep the state of the whole prompt, steps of 20 nothing."""
    assert Layer(gdn, 1, 3000, 64, 16, kind=FP32, seed=4, step=(1e-5, 1e-4)).check() == 0
    assert Layer(gdn, 2, 300, 64, 16, kind=FP32, seed=5, step=(0.5, 20.0)).check() == 0
    layer = Layer(gdn, 1, 50, 64, 16, kind=FP32, seed=6)
    layer.dt[0, 7], layer.dt[0, 8], layer.dt[0, 9] = 60.0, -60.0, -200.0
    assert layer.check() == 0


@pytest.mark.parametrize("kind", [BF16, FP32])
def test_scan_with_far_gates(gdn, kind):
    layer = Layer(gdn, 1, 60, 64, 16, kind=kind, seed=7)
    layer.z[0, :8] = torch.tensor([-20.0, -87, -89, -100, -1000, 50, 100, 3e4], device="cuda").to(kind)[:, None]
    assert layer.check() == 0


def test_scan_skips_padding_and_what_is_wrong(gdn):
    assert Layer(gdn, 4, 40, 64, 16, lens=[40, 7, 0, 33], slot=[-1, 2, -5, 0]).check() == 0
    assert Layer(gdn, 3, 40, 64, 16, slot=[1, 5, 0]).check() == gdn.STATUS_BAD_SLOT
    assert Layer(gdn, 3, 40, 64, 16, lens=[3, -1, 40], slot=[1, 2, 0]).check() == gdn.STATUS_BAD_LEN
    assert Layer(gdn, 3, 1200, 64, 16, lens=[3, 1201, 40], slot=[1, 2, 0]).check() == gdn.STATUS_BAD_LEN
    assert Layer(gdn, 3, 1200, 64, 16, lens=[3, 1201, 1200], slot=[1, -1, 7]).check() == gdn.STATUS_BAD_SLOT


@pytest.mark.parametrize("kind", [BF16, FP32])
def test_scan_of_one_token_in_any_stride(gdn, kind):
    """The distance to a next token, where there is none, need not be a multiple of anything."""
    layer = Layer(gdn, 3, 1, 64, 16, 2, kind, seed=11)

    def apart(x):
        wide = x[0].numel() + 66
        strides = (4 * wide, wide, 1) if x.dim() == 3 else (4 * wide, wide, x.shape[3], 1)
        return torch.zeros(12 * wide, dtype=kind, device="cuda").as_strided(x.shape, strides, 32).copy_(x)

    for name in ("u", "dt", "z", "b", "c"):
        setattr(layer, name, apart(getattr(layer, name)))
    assert layer.u.stride(1) % 8 == 2 and layer.b.stride(1) % 8 == 2
    assert layer.check() == 0


def test_scan_gives_the_same_bits_again(gdn):
    runs = []
    for _ in range(3):
        layer = Layer(gdn, 2, 1500, 264, 16, seed=9)
        layer.call()
        runs.append((layer.y, layer.state))
    torch.cuda.synchronize()
    assert all(torch.equal(runs[0][i], r[i]) for r in runs for i in (0, 1))


@pytest.mark.parametrize("kind", [BF16, FP32])
@pytest.mark.parametrize("B,D,N,G,slot", [(1, 8, 8, 1, None), (1, 2048, 16, 1, None), (5, 264, 16, 3, None), (3, 72, 32, 1, None), (33, 64, 64, 4, None),
                                          (261, 4096, 16, 1, [i if i % 7 else -1 for i in range(260)] + [9999]),
                                          (6, 136, 16, 1, [0, -1, 3, 7, -2, 1]), (7, 64, 8, 2, [5, 4, 3, 99, 1, 0, -1])])
def test_step(gdn, kind, B, D, N, G, slot):
    for z in (True, False):
        layer = Layer(gdn, B, 1, D, N, G, kind, slot=slot, seed=B + D, z=z, bias=z)
        bad = any(x >= layer.num_slots for x in layer.slot)

        def call():
            one = lambda x: None if x is None else x[:, 0]  # noqa: E731
            y = layer.y[:, 0].contiguous()
            gdn.ssm_step(one(layer.u), one(layer.dt), layer.a, one(layer.b), one(layer.c), layer.state, ints(layer.slot), y, z=one(layer.z),
                         skip=layer.skip, dt_bias=layer.bias, status=layer.status)
            layer.y = y[:, None]
        assert layer.check(call) == (gdn.STATUS_BAD_SLOT if bad else 0)


def test_far_slots_and_rows(gdn):
    """Offsets past 32 bits: the last slots of large pools, and requests far from one another."""
    g = gen(12)
    B, T, D, N, far = 2, 70, 8192, 32, 8300  # 2.2e9 states
    small = Layer(gdn, B, T, D, N, seed=3, slot=[1, 0])
    big = Layer(gdn, B, T, D, N, seed=3, slot=[far - 1, 0])
    big.num_slots = far
    big.state = torch.zeros(far, D, N, device="cuda")
    big.state[far - 1], big.state[0] = small.state[1], small.state[0]
    room = torch.empty(2 ** 31 + 8 + T * D, dtype=BF16, device="cuda")
    u = room.as_strided((B, T, D), (2 ** 31 + 8, D, 1))
    u.copy_(big.u)
    big.u = u
    small.call(), big.call()
    assert torch.equal(small.y, big.y) and torch.equal(small.state[:2], big.state[[0, far - 1]])
    for x in (small, big):
        gdn.ssm_step(x.u[:, 5], x.dt[:, 5], x.a, x.b[:, 5], x.c[:, 5], x.state, ints(x.slot), x.y[:, 5].contiguous(), skip=x.skip)
    assert torch.equal(small.state[:2], big.state[[0, far - 1]])
    del big.state
    w, slots = 0.5 * randn(g, D, 4), 90000  # 2.2e9 elements
    pool = torch.zeros(slots, D, 3, dtype=BF16, device="cuda")
    near = randn(g, 2, D, 3, dtype=BF16)
    pool[slots - 1], pool[0] = near[1], near[0]
    for x_small, x_big in ((small.u, u), (small.u[:, 3], u[:, 3])):
        o = [torch.empty(x_small.shape, dtype=BF16, device="cuda") for _ in range(2)]
        gdn.causal_conv(x_small, w, near, ints([1, 0]), o[0])
        gdn.causal_conv(x_big, w, pool, ints([slots - 1, 0]), o[1])
        assert torch.equal(o[0], o[1]) and torch.equal(near, pool[[0, slots - 1]])


# ---- together -----------------------------------------------------------------------------------
class Mixer:
    """One selective layer: norm into 8 bits, projections, convolution, recurrence, all of a request in slots."""

    def __init__(self, gdn, width=256, N=16, rank=16, slots=6, seed=0):
        g = gen(seed)
        self.gdn, self.width, self.N, self.rank = gdn, width, N, rank
        D = self.D = 2 * width
        weight = lambda r, c: (randn(g, r, c) * r ** -0.5).to(BF16)  # noqa: E731
        self.w_in, self.w_x, self.w_dt, self.w_out = weight(width, 2 * D), weight(D, rank + 2 * N), weight(rank, D), weight(D, width)
        self.conv_w, self.conv_b, self.norm_w = 0.5 * randn(g, D, 4), 0.1 * randn(g, D), 1 + 0.1 * randn(g, width)
        self.a, self.skip, self.bias = -torch.arange(1, N + 1, device="cuda").float().repeat(D, 1), torch.ones(D, device="cuda"), randn(g, D) - 3
        self.pool, self.state = torch.zeros(slots, D, 3, dtype=BF16, device="cuda"), torch.zeros(slots, D, N, device="cuda")
        self.status = ints([0])

    def forward(self, x, residual, slot, lens=None):
        """x, residual [B, T, width], or [B, width] for one token each."""
        gdn, D, N = self.gdn, self.D, self.N
        at, flat = x.shape[:-1], (-1, self.width)
        q, scales = torch.empty(x.shape, dtype=E4M3, device="cuda"), torch.empty(at.numel(), 2, device="cuda")
        gdn.add_rms_norm(x.reshape(flat), q.view(flat), residual=residual.view(flat), weight=self.norm_w, scales=scales, group=128)
        normed = (q.view(flat).float() * scales.repeat_interleave(128, 1)).to(BF16)
        mixed = (normed @ self.w_in).view(*at, 2 * D)
        u = torch.zeros(*at, D, dtype=BF16, device="cuda")
        gdn.causal_conv(mixed[..., :D], self.conv_w, self.pool, slot, u, bias=self.conv_b, seq_lens=lens, status=self.status)
        low = u @ self.w_x
        dt = low[..., :self.rank] @ self.w_dt
        b, c = low[..., None, self.rank:self.rank + N], low[..., None, self.rank + N:]
        y = torch.zeros_like(u)
        kw = dict(z=mixed[..., D:], skip=self.skip, dt_bias=self.bias, status=self.status)
        if x.dim() == 2:
            gdn.ssm_step(u, dt, self.a, b, c, self.state, slot, y, **kw)
        else:
            size = gdn.ssm_workspace_bytes(*u.shape, N)
            gdn.ssm_scan(u, dt, self.a, b, c, self.state, slot, y, torch.empty(max(size, 16), dtype=torch.uint8, device="cuda"), seq_lens=lens, **kw)
        return y @ self.w_out


def test_prompt_then_tokens(gdn):
    """A prompt at once leaves what its tokens one by one leave, and both go on alike; one-token
    steps in a replayed graph give the eager steps' bits."""
    prompt, more, B = 45, 5, 3
    g = gen(21)
    x = randn(g, B, prompt + more, 256, dtype=BF16)
    slot, lens = ints([4, 0, 2]), [45, 31, 1]
    whole, single, graph = (Mixer(gdn) for _ in range(3))
    first = x[:, :prompt].contiguous()
    whole.forward(first, torch.zeros_like(first), slot, ints(lens))
    for t in range(prompt):
        live = torch.tensor([t < n for n in lens], device="cuda")
        single.forward(x[:, t].contiguous(), torch.zeros(B, 256, dtype=BF16, device="cuda"), torch.where(live, slot, -1))
    # matrix products of other shapes may round the inputs of conv and scan otherwise
    assert (whole.pool - single.pool).abs().max() <= 2.0 ** -4 * single.pool.abs().max()
    assert (whole.state - single.state).norm() <= 2e-2 * single.state.norm()
    assert whole.state[[1, 3, 5]].abs().max() == 0 and whole.pool[[1, 3, 5]].abs().max() == 0
    graph.pool.copy_(whole.pool), graph.state.copy_(whole.state)
    token, residual = x[:, prompt].clone(), torch.zeros(B, 256, dtype=BF16, device="cuda")
    graph.forward(token, residual, slot)  # once before the capture
    graph.pool.copy_(whole.pool), graph.state.copy_(whole.state)
    captured = torch.cuda.CUDAGraph()
    with torch.cuda.graph(captured):
        out = graph.forward(token, residual, slot)
    graph.pool.copy_(whole.pool), graph.state.copy_(whole.state)
    for t in range(prompt, prompt + more):
        eager = whole.forward(x[:, t].contiguous(), torch.zeros(B, 256, dtype=BF16, device="cuda"), slot)
        token.copy_(x[:, t]), residual.zero_()
        captured.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(graph.state, whole.state) and torch.equal(graph.pool, whole.pool)
    assert whole.status.item() == single.status.item() == graph.status.item() == 0


def test_streams_at_once(gdn):
    """Scans that share the GPU, each with its workspace: the bits of the scans alone."""
    make = lambda: [Layer(gdn, 1, 2000, 264, 16, seed=1), Layer(gdn, 3, 700, 128, 64, kind=FP32, seed=2), Layer(gdn, 2, 1500, 72, 8, seed=3)]  # noqa: E731
    alone, layers = make(), make()
    for layer in alone:
        layer.call()
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    first = [(x.state.clone(), x) for x in layers]
    for _ in range(10):
        for (before, layer), stream in zip(first, streams):
            with torch.cuda.stream(stream):
                layer.state.copy_(before)
                layer.call()
    torch.cuda.synchronize()
    for x, y in zip(alone, layers):
        assert torch.equal(x.y, y.y) and torch.equal(x.state, y.state)


def test_two_graphs_share_a_workspace(gdn):
    layers = [Layer(gdn, 1, 1800, 264, 16, seed=1), Layer(gdn, 1, 1800, 264, 16, seed=2)]
    eager = [Layer(gdn, 1, 1800, 264, 16, seed=1), Layer(gdn, 1, 1800, 264, 16, seed=2)]
    slots = [ints(x.slot) for x in layers]
    graphs = []
    for layer, slot in zip(layers, slots):
        before = layer.state.clone()
        run = lambda: gdn.ssm_scan(layer.u, layer.dt, layer.a, layer.b, layer.c, layer.state, slot, layer.y, layers[0].workspace, z=layer.z,  # noqa: E731,B023
                                   skip=layer.skip, dt_bias=layer.bias)
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        layer.state.copy_(before)
        graphs.append(graph)
    for i in (0, 1, 0):
        graphs[i].replay()
    for i in (0, 1, 0):
        eager[i].call()
    torch.cuda.synchronize()
    for x, y in zip(layers, eager):
        assert torch.equal(x.y, y.y) and torch.equal(x.state, y.state)
