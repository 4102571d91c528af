"""Paged-cache calls on the GPU against plain definitions: the plan against a Python loop, the
append bit for bit, attention against 64-bit softmax sums."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_decode_gdn_gb300 as g
    return g


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- plan -------------------------------------------------------------------------------------
def plan_reference(cached, new, held, table, free, count, page, pages, capacity):
    """Request by request, as gdn.h says it. Returns what the call writes, and the status."""
    S = dict(NO_PAGES=0x10, BAD_LEN=4, BAD_PAGE=0x20)
    bad, avail, given = 0, count, count
    if not 0 <= count <= len(free):  # the list's room
        bad, avail = S["BAD_LEN"], 0
    table, held, free = [list(r) for r in table], list(held), list(free)
    length, cu, slots, used, full = [], [0], [-1] * capacity, 0, False
    for b, c in enumerate(cached):
        n = 0 if c < 0 else (1 if new is None else new[b])
        ok = c >= 0
        if n < 0:
            n, ok, bad = 0, False, bad | S["BAD_LEN"]
        cu.append(cu[-1] + n)
        need = -(-(c + n) // page)
        if ok and (not 0 <= held[b] <= len(table[b]) or need > len(table[b]) or c + n > 2 ** 31 - 1 or cu[-1] > capacity):
            ok, bad = False, bad | S["BAD_LEN"]
        want = max(0, need - held[b]) if ok else 0
        if want and (full or used + want > avail):
            ok, full, bad = False, True, bad | S["NO_PAGES"]
        if not ok:
            length.append(max(c, 0))
            continue
        for j in range(want):
            x = free[avail - 1 - used]
            if not 0 <= x < pages:
                x, bad = -1, bad | S["BAD_PAGE"]
            table[b][held[b] + j] = x
            used += 1
        held[b] += want
        length.append(c + n)
        for i in range(n):
            x = table[b][(c + i) // page]
            if 0 <= x < pages:
                slots[cu[b] + i] = x * page + (c + i) % page
            else:
                bad |= S["BAD_PAGE"]
    return dict(kv_len=length, cu=[min(x, 2 ** 31 - 1) for x in cu], slots=slots, table=table, held=held, count=given if given != avail else avail - used), bad


def run_plan(gdn, cached, new, held, table, free, count, page, pages, capacity, in_place=False):
    t = ints(table)
    c, h, k = ints(cached), ints(held), ints([count])
    out = dict(kv_len=torch.full_like(c, -7), held=torch.full_like(h, -7), count=torch.full_like(k, -7))
    if in_place:
        out = dict(kv_len=c, held=h, count=k)
    cu = torch.full((len(cached) + 1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((capacity,), -7, dtype=torch.int64, device="cuda")
    st = status()
    gdn.kv_plan(c, None if new is None else ints(new), h, t, ints(free), k, kv_len=out["kv_len"], cu_new=cu, slot_map=slots,
                held_out=out["held"], free_count_out=out["count"], page_size=page, num_pages=pages, status=st)
    torch.cuda.synchronize()
    return dict(kv_len=out["kv_len"].tolist(), cu=cu.tolist(), slots=slots.tolist(), table=t.tolist(),
                held=out["held"].tolist(), count=out["count"].item()), st.item()


@pytest.mark.parametrize("batch,page,most,new_most,short,seed", [
    (1, 16, 40, 1, 0, 1), (1, 1, 5, 9, 0, 2), (7, 16, 100, 1, 0, 3), (64, 64, 1000, 70, 0, 4), (513, 16, 300, 40, 0, 5),
    (600, 7, 90, 30, 100, 6), (2100, 32, 64, 3, 500, 7), (4096, 16, 50, 2, 1, 8), (5, 16, 0, 0, 0, 9), (9, 16, 90, 300, 3, 10),
])
def test_plan(gdn, batch, page, most, new_most, short, seed):
    r = random.Random(seed)
    cached = [-1 if r.random() < 0.05 else r.randint(0, most) for _ in range(batch)]
    new = None if new_most == 1 else [r.randint(0, new_most) for _ in range(batch)]
    # some requests hold more than they use (rejected drafts), one in twenty a page less than they should
    held = [0 if c < 0 else -(-c // page) + (r.random() < 0.2) for c in cached]
    width = -(-(most + max(new_most, 1)) // page) + 2
    pages = sum(held) + sum(-(-(n or 0) // page) + 1 for n in (new or [1] * batch)) + 1
    ids = list(range(pages))
    r.shuffle(ids)
    table = [[-1] * width for _ in range(batch)]
    for b in range(batch):
        for j in range(held[b]):
            table[b][j] = ids.pop()
    wants = sum(max(0, -(-(c + (1 if new is None else new[b])) // page) - held[b]) for b, c in enumerate(cached) if c >= 0)
    count = max(0, min(len(ids), wants) - short)
    total = sum(0 if c < 0 else (1 if new is None else new[b]) for b, c in enumerate(cached))
    for capacity in (total + 3, max(0, total - 2)):
        want, bad = plan_reference(cached, new, held, table, ids, count, page, pages, capacity)
        for in_place in (False, True):
            got, st = run_plan(gdn, cached, new, held, table, ids, count, page, pages, capacity, in_place)
            assert got == want
            assert st == bad
        if short and capacity > total:
            assert bad & gdn.STATUS_NO_PAGES


@pytest.mark.parametrize("kw", [
    dict(new=[1, -2, 1]), dict(cached=[10, 3000, 4]), dict(held=[1, -1, 1]), dict(held=[1, 99, 1]),
    dict(cached=[2 ** 31 - 1, 3, 4]), dict(new=[2 ** 30, 2 ** 30, 2 ** 30]), dict(count=-3), dict(count=99), dict(count=5),
    dict(table=[[0, -1], [77, -1], [2, -1]]), dict(free=[8, -5, 7, 99], cached=[16, 16, 16]),
])
def test_plan_reports_what_cannot_be(gdn, kw):
    d = dict(cached=[10, 11, 4], new=[1, 1, 1], held=[1, 1, 1], table=[[0, -1], [1, -1], [2, -1]], free=[3, 4, 5, 6], count=4)
    d.update(kw)
    args = (d["cached"], d["new"], d["held"], d["table"], d["free"], d["count"], 16, 9, 8)
    want, bad = plan_reference(*args)
    got, st = run_plan(gdn, *args)
    assert got == want and st == bad and bad


def test_release_then_plan_again(gdn):
    r = random.Random(3)
    batch, width, pages = 700, 5, 4000
    held = [r.randint(0, width) for _ in range(batch)]
    ids = list(range(pages))
    r.shuffle(ids)
    table = [[ids.pop() if j < held[b] else -1 for j in range(width)] for b in range(batch)]
    free = ids + [-1] * (pages - len(ids))
    done = r.sample(range(batch), 600) + [-1, -4]
    r.shuffle(done)
    st, h, f, c, t = status(), ints(held), ints(free), ints([len(ids)]), ints(table)
    gdn.kv_release(ints(done), h, t, f, c, status=st)
    for b in done:
        if b >= 0:
            ids += table[b][:held[b]]
            held[b] = 0
    assert st.item() == 0 and h.tolist() == held and c.item() == len(ids) and f.tolist()[:len(ids)] == ids
    # what cannot be: an unknown request, a count past the row, a list that is full
    gdn.kv_release(ints([batch, 1]), ints([0, 9] + [0] * (batch - 2)), t, f, c, status=st)
    assert st.item() == (gdn.STATUS_BAD_SLOT | gdn.STATUS_BAD_LEN) and c.item() == len(ids)
    st, h, c = status(), ints([2, 2, 1]), ints([3])
    gdn.kv_release(ints([0, 1, 2]), h, ints([[1, 2], [3, 4], [5, 6]]), ints([7, 8, 9, -1, -1, -1]), c, status=st)
    assert st.item() == gdn.STATUS_BAD_LEN and c.item() == 5 and h.tolist() == [0, 2, 1]


# ---- append -----------------------------------------------------------------------------------
@pytest.mark.parametrize("n,heads,dk,dv,page,dtype,latent", [
    (1, 1, 8, 8, 1, torch.bfloat16, False), (5, 2, 64, 64, 16, torch.float32, False), (130, 8, 128, 128, 64, torch.bfloat16, False),
    (1001, 3, 96, 40, 7, torch.bfloat16, False), (77, 4, 256, 256, 32, torch.float32, False),
    (3, 1, 576, 512, 64, torch.float32, True), (999, 1, 576, 512, 16, torch.bfloat16, True), (65, 1, 64, 64, 8, torch.bfloat16, True),
    (20011, 8, 128, 128, 16, torch.bfloat16, False),
])
def test_append(gdn, n, heads, dk, dv, page, dtype, latent):
    g = torch.Generator(device="cuda").manual_seed(n)
    pages = -(-n // page) + 3
    # pages padded between positions and heads, in an order of its own
    k_pool = torch.randn(heads, pages, page, dk + 8, generator=g, device="cuda").bfloat16()[..., :dk].permute(1, 2, 0, 3)
    v_pool = None if latent else torch.randn(pages, page, heads, dv, generator=g, device="cuda").bfloat16()
    kv = gdn.make_paged_kv(k_pool, dv=dv) if latent else gdn.make_paged_kv(k_pool, v_pool)
    first, second = (dv, dk - dv) if latent else (dk, dv)
    mixed = torch.randn(n, heads, first + second, generator=g, device="cuda").to(dtype)
    k, v = mixed[..., :first], mixed[..., first:] if second else None
    if dtype is torch.float32:  # halfway cases and values that round up to the next power of two
        k[0, 0, :4] = torch.tensor([1.00390625, 1.01171875, -1.9999999, 3.0e-39], device="cuda")
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n]
    if n > 2:
        slots[1], slots[n // 2] = -1, pages * page + 5
    want_k, want_v = k_pool.clone().reshape(-1, heads, dk), None if latent else v_pool.clone().reshape(-1, heads, dv)
    live = (slots >= 0) & (slots < pages * page)
    rows = mixed.bfloat16()[live]
    if latent:
        want_k[slots[live]] = rows
    else:
        want_k[slots[live]], want_v[slots[live]] = rows[..., :first], rows[..., first:]
    st = status()
    gdn.kv_append(kv, k, v, slots, status=st)
    torch.cuda.synchronize()
    assert st.item() == (gdn.STATUS_BAD_SLOT if n > 2 else 0)
    assert torch.equal(k_pool.reshape(-1, heads, dk).view(torch.int16), want_k.view(torch.int16))
    if not latent:
        assert torch.equal(v_pool.reshape(-1, heads, dv).view(torch.int16), want_v.view(torch.int16))


# ---- attention --------------------------------------------------------------------------------
class Problem:
    """Pages in a shuffled order with NaN and infinities wherever no query looks, block tables with
    entries that name no page wherever none is needed."""

    def __init__(self, gdn, lens, T=1, heads=4, heads_kv=2, dk=128, dv=None, page=16, window=0, latent=False, seed=0, scale=None,
                 spread=1.0, permuted=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dv = dk if dv is None else dv
        self.gdn, self.lens, self.T, self.window, self.page = gdn, list(lens), T, window, page
        self.heads, self.heads_kv, self.dk, self.dv, self.latent = heads, heads_kv, dk, dv, latent
        self.scale = dk ** -0.5 if scale is None else scale
        counts = [-(-max(n, 0) // page) for n in lens]
        total = sum(counts) + 2
        perm = torch.randperm(total, generator=g, device="cuda").tolist()
        width = max(1, max(counts)) + 1
        table, self.own_pages = [], []
        for c in counts:
            mine = [perm.pop() for _ in range(c)]
            self.own_pages.append(mine)
            table.append(mine + [[-1, total, 2 ** 31 - 1, -2 ** 31][len(table) % 4]] * (width - c))
        for b, n in enumerate(lens):  # pages that a window has left behind are gone
            gone = max(0, n - T - window + 1) // page if window else 0
            for j in range(min(gone, counts[b])):
                table[b][j] = -1
        self.table, self.kv_len = ints(table), ints(self.lens)

        def pool(d):
            shape = (total, heads_kv, page, d) if permuted else (total, page, heads_kv, d)
            x = torch.randn(shape, generator=g, device="cuda").mul_(spread).bfloat16()
            x = x.permute(0, 2, 1, 3) if permuted else x
            seen = torch.zeros(total, page, dtype=torch.bool, device="cuda")
            for b, n in enumerate(lens):
                if n > 0:
                    p = torch.arange(n, device="cuda")
                    p = p[p > n - T - window] if window else p
                    seen[torch.tensor(self.own_pages[b], device="cuda")[p // page], p % page] = True
            bad = torch.tensor([NAN, math.inf, -math.inf, 3e38], device="cuda", dtype=torch.bfloat16)
            fill = bad[torch.randint(0, 4, (total, page, 1, 1), generator=g, device="cuda")]
            x.copy_(torch.where(seen[..., None, None], x, fill))
            return x

        self.k = pool(dk)
        self.v = None if latent else pool(dv)
        wide = torch.randn(len(lens), T, heads + 1, dk + 8, generator=g, device="cuda").mul_(spread).bfloat16()
        self.q = wide[:, :, 1:, :dk]  # a slice of a wider projection
        self.o = torch.full((len(lens), T, heads, dv), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((len(lens), T, heads), 7.0, device="cuda")
        self.status = status()
        self.kv = gdn.make_paged_kv(self.k, dv=dv) if latent else gdn.make_paged_kv(self.k, self.v)
        size = gdn.attn_workspace_bytes(self.kv, len(lens), T, heads)
        self.workspace = torch.full((size // 4,), NAN, device="cuda")

    def call(self, **kw):
        f = self.gdn.latent_decode if self.latent else self.gdn.attn_decode
        f(self.kv, self.q, self.table, self.kv_len, self.o, self.workspace, lse=self.lse, scale=self.scale, window=self.window,
          status=self.status, **kw)

    def expected(self, b):
        """(o, lse, tolerance of o, tolerance of lse) of request b in 64 bits, [T, heads, ..].

        Tolerances: the output is rounded to bf16 (2^-8 of the value at most) and each weight may be
        (2^-8 of it, so 2^-8 of sum w |v|). The score is a sum of dk products in fp32: it is off by at
        most (dk + 4) 2^-24 sum |q k| scale (the products of bf16 are exact), a weight by that factor
        and 2^-21 for the exponential, and a sum of n weights by n 2^-24 of itself."""
        n, T, G = self.lens[b], self.T, self.heads // self.heads_kv
        o = torch.zeros(T, self.heads, self.dv, dtype=torch.float64, device="cuda")
        to, tl = torch.zeros_like(o), torch.zeros(T, self.heads, dtype=torch.float64, device="cuda")
        lse = torch.full((T, self.heads), -math.inf, dtype=torch.float64, device="cuda")
        if n <= 0:
            return o, lse, to, tl
        at = torch.tensor(self.own_pages[b], device="cuda")
        k = self.k[at].flatten(0, 1)[:n].double()
        v = k[..., :self.dv] if self.latent else self.v[at].flatten(0, 1)[:n].double()
        usable = torch.tensor([0 <= x < self.k.shape[0] for x in self.table[b].tolist()], device="cuda")
        usable = usable.repeat_interleave(self.page)[:n]
        for t in range(T):
            pos = n - T + t
            j = torch.arange(n, device="cuda")
            j = j[(j <= pos) & usable & ((j > pos - self.window) if self.window else (j >= 0))]
            if not len(j):
                continue
            for h in range(self.heads):
                q = self.q[b, t, h].double()
                s = k[j, h // G] @ q * self.scale
                size = float((k[j, h // G].abs() @ q.abs()).max()) * abs(self.scale)
                w = torch.softmax(s, 0)
                o[t, h], lse[t, h] = w @ v[j, h // G], torch.logsumexp(s, 0)
                off = (self.dk + 4) * 2.0 ** -24 * size + 2.0 ** -21
                to[t, h] = o[t, h].abs() * 2.0 ** -8 + (w @ v[j, h // G].abs()) * (2.0 ** -8 + 2 * off + (len(j) + 64) * 2.0 ** -24) * 1.01
                tl[t, h] = off + (len(j) + 64) * 2.0 ** -24 + lse[t, h].abs() * 2.0 ** -22
        return o, lse, to, tl

    def check(self, bad=0):
        torch.cuda.synchronize()
        assert self.status.item() == bad
        worst = 0.0
        for b, n in enumerate(self.lens):
            if n < 0 or n > self.table.shape[1] * self.page:
                assert bool((self.o[b] == 7).all()) and bool((self.lse[b] == 7).all()), b
                continue
            o, lse, to, tl = self.expected(b)
            got, got_lse = self.o[b].double(), self.lse[b].double()
            empty = torch.isinf(lse)
            assert torch.equal(torch.isinf(got_lse) & (got_lse < 0), empty), (b, n)
            assert bool((got[empty] == 0).all()), (b, n)
            assert not bool(torch.isnan(got).any()), (b, n)
            far = ((got - o).abs() - to)[~empty]
            assert far.numel() == 0 or float(far.max()) <= 0, (b, n, float(far.max()), float((got - o).abs().max()))
            off = ((got_lse - lse).abs() - tl)[~empty]
            assert off.numel() == 0 or float(off.max()) <= 0, (b, n, float(off.max()))
            worst = max(worst, float((got - o).abs().max()))
        return worst


RAGGED = [0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 1000]

SHAPES = [
    # general shapes (CUDA cores)
    dict(dk=16, page=1, heads=2, heads_kv=1), dict(dk=32, page=24), dict(dk=128, dv=64, page=16), dict(dk=64, dv=128, page=8),
    dict(dk=192, dv=128, page=48, heads=6, heads_kv=2), dict(dk=80, page=10, heads=9, heads_kv=3),
    dict(dk=256, dv=512, page=33), dict(dk=576, dv=512, page=3, heads=4, heads_kv=1),
    # head sizes and pages of the tensor-core kernel
    dict(dk=64, page=16, heads=8, heads_kv=2), dict(dk=64, page=128, heads=3, heads_kv=3), dict(dk=128, page=16),
    dict(dk=128, page=32, heads=8, heads_kv=1), dict(dk=128, page=64, heads=40, heads_kv=2), dict(dk=128, page=256, heads=32, heads_kv=1),
    dict(dk=256, page=64, heads=16, heads_kv=2), dict(dk=256, page=128, heads=24, heads_kv=1), dict(dk=256, page=16, heads=70, heads_kv=1),
    dict(dk=128, page=64, heads=130, heads_kv=1),
]
LATENT = [
    dict(dk=64, dv=48, page=5, heads=3), dict(dk=512, dv=512, page=16, heads=16), dict(dk=576, dv=512, page=16, heads=1),
    dict(dk=576, dv=512, page=32, heads=16), dict(dk=576, dv=512, page=64, heads=32), dict(dk=576, dv=512, page=128, heads=20),
    dict(dk=576, dv=512, page=64, heads=128), dict(dk=576, dv=512, page=640, heads=65),
]


def name_of(d):
    return "-".join(f"{k}{v}" for k, v in d.items())


@pytest.mark.parametrize("shape", SHAPES, ids=name_of)
def test_attention_over_ragged_lengths(gdn, shape):
    p = Problem(gdn, RAGGED, seed=1, **shape)
    p.call()
    p.check()


@pytest.mark.parametrize("shape", LATENT, ids=name_of)
def test_latent_over_ragged_lengths(gdn, shape):
    p = Problem(gdn, RAGGED, latent=True, heads_kv=1, seed=2, **shape)
    p.call()
    p.check()


@pytest.mark.parametrize("T", [2, 3, 5])
@pytest.mark.parametrize("window", [0, 1, 2, 100, 128, 5000])
@pytest.mark.parametrize("shape", [dict(dk=32, page=6, heads=4, heads_kv=2), dict(dk=64, page=16, heads=8, heads_kv=2),
                                   dict(dk=128, page=64, heads=32, heads_kv=2), dict(dk=256, page=32, heads=4, heads_kv=4),
                                   dict(dk=576, dv=512, page=64, heads=16, heads_kv=1, latent=True)], ids=name_of)
def test_several_positions_and_windows(gdn, shape, T, window):
    p = Problem(gdn, RAGGED, T=T, window=window, seed=3, **shape)
    p.call()
    p.check()


@pytest.mark.parametrize("shape", [dict(dk=96, page=16), dict(dk=64, page=16, heads=7, heads_kv=1), dict(dk=128, page=32, heads=8, heads_kv=2),
                                   dict(dk=256, page=128, heads=16, heads_kv=1),
                                   dict(dk=576, dv=512, page=64, heads=32, heads_kv=1, latent=True)], ids=name_of)
@pytest.mark.parametrize("lens", [[1], [40000], [3, 20001, 1, 9000], [129] * 333, [0] * 5 + [1] * 700], ids=lambda x: f"{len(x)}x{max(x)}")
def test_splits(gdn, shape, lens):
    """Units cut over many CTAs, CTAs with many units, batches past the block's threads."""
    if len(lens) * max(lens) > 40000:
        lens = lens[:1] + lens[-150:] if len(lens) > 150 else lens
    p = Problem(gdn, lens, seed=4, **shape)
    p.call()
    p.check()
    first, first_lse = p.o.clone(), p.lse.clone()
    p.o.fill_(7), p.lse.fill_(7)
    p.workspace.fill_(NAN)
    p.call()
    torch.cuda.synchronize()
    assert torch.equal(p.o, first) and torch.equal(p.lse, first_lse)  # the same bits every time


@pytest.mark.parametrize("shape", [dict(dk=48, page=16), dict(dk=128, page=16, heads=8, heads_kv=2), dict(dk=256, page=64, heads=4, heads_kv=2),
                                   dict(dk=576, dv=512, page=32, heads=16, heads_kv=1, latent=True)], ids=name_of)
def test_large_scores_strides_and_scales(gdn, shape):
    # scores of several hundred: all weight on a few positions, maxima that rise from tile to tile
    for kw in (dict(spread=6.0), dict(scale=-0.3), dict(scale=0.0), dict(permuted=True), dict(permuted=True, T=2, window=70)):
        p = Problem(gdn, [1, 130, 700, 1500], seed=5, **shape, **kw)
        p.call()
        p.check()
    # keys that grow along the request, so that the maximum rises in every tile
    p = Problem(gdn, [2000], seed=6, **shape)
    ramp = torch.linspace(0.1, 12.0, 2000, device="cuda")
    at = torch.tensor(p.own_pages[0], device="cuda")
    pos = torch.arange(2000, device="cuda")
    rows = (at[pos // p.page], pos % p.page)
    p.k[rows] = (p.q[0, 0, :1].float() * ramp[:, None, None] / p.dk ** 0.5).expand(-1, p.heads_kv, -1).bfloat16()
    p.call()
    p.check()


@pytest.mark.parametrize("shape", [dict(dk=40, page=16), dict(dk=128, page=16, heads=8, heads_kv=2), dict(dk=64, page=64, heads=8, heads_kv=2),
                                   dict(dk=576, dv=512, page=64, heads=16, heads_kv=1, latent=True)], ids=name_of)
def test_requests_and_pages_that_are_left_out(gdn, shape):
    p = Problem(gdn, [-1, 300, 5, 4000, -9, 0, 700], seed=7, **shape)
    p.lens[3] = 1 << 20  # more than the table holds
    p.kv_len[3] = 1 << 20
    p.call()
    p.check(gdn.STATUS_BAD_LEN)
    # unusable pages take no part; a request with none left is empty
    p = Problem(gdn, [300, 5, 700, 64], seed=8, **shape)
    p.table[0, 1] = -1
    p.table[2, 0] = p.k.shape[0]
    p.table[2, 5 if p.page == 16 else 2] = -2 ** 31
    p.table[1] = -1
    p.table[3] = 2 ** 31 - 1
    p.call()
    p.check(gdn.STATUS_BAD_PAGE)


def test_without_lse_or_status_on_another_stream_and_in_a_graph(gdn):
    p = Problem(gdn, [700, 3, 129], heads=8, heads_kv=2, T=2, page=32, seed=9)
    args = (p.kv, p.q, p.table, p.kv_len, p.o, p.workspace)
    p.call()
    torch.cuda.synchronize()
    want = p.o.clone()
    p.o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gdn.attn_decode(*args, stream=side)
    side.synchronize()
    assert torch.equal(p.o, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call()
    p.o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.o, want)
    # the lengths are read on the device: the same graph serves other lengths
    p.lens = [650, 0, 1]
    p.kv_len.copy_(ints(p.lens))
    graph.replay()
    p.check()
    with pytest.raises(ValueError):
        gdn.attn_decode(p.kv, p.q.float(), *args[2:])
    with pytest.raises(ValueError):
        gdn.attn_decode(p.kv, p.q, p.table, p.kv_len.long(), p.o, p.workspace)
    with pytest.raises(gdn.GDNError):
        gdn.attn_decode(p.kv, p.q, p.table, p.kv_len, p.o, p.workspace[:4])
    with pytest.raises(gdn.GDNError):
        gdn.latent_decode(*args)


def test_offsets_past_32_bits(gdn):
    """A cache of more than 2^32 bytes a pool: pages at its far end are found."""
    page, heads_kv, dk = 64, 8, 128
    pages = (1 << 32) // (page * heads_kv * dk) + 40  # 2^32 elements and some
    if torch.cuda.mem_get_info()[0] < 3 * pages * page * heads_kv * dk * 2:
        pytest.skip("needs 30 GB")
    p = Problem(gdn, [200, 500], heads=16, heads_kv=heads_kv, dk=dk, page=page, seed=10)
    big_k = torch.empty(pages, page, heads_kv, dk, dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty_like(big_k)
    shift = pages - p.k.shape[0]
    big_k[shift:], big_v[shift:] = p.k, p.v
    p.k, p.v = big_k, big_v
    p.own_pages = [[x + shift for x in mine] for mine in p.own_pages]
    table = [mine + [-1] * (p.table.shape[1] - len(mine)) for mine in p.own_pages]
    p.table.copy_(ints(table))
    p.kv = gdn.make_paged_kv(p.k, p.v)
    p.call()
    p.check()
    slots = ints([pages * page - 1, shift * page], torch.int64)
    new = torch.randn(2, 2 * heads_kv, dk, device="cuda").bfloat16()
    gdn.kv_append(p.kv, new[:, :heads_kv], new[:, heads_kv:], slots, status=p.status)
    torch.cuda.synchronize()
    assert p.status.item() == 0
    assert torch.equal(big_k[-1, -1], new[0, :heads_kv]) and torch.equal(big_v[shift, 0], new[1, heads_kv:])


# ---- together ---------------------------------------------------------------------------------
def load_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_hybrid_steps_in_a_graph(gdn):
    """The example's stack: replayed graphs give the eager steps' bits, pages are handed out as
    lengths pass them, and both attention layers agree with 64-bit sums over what was appended."""
    hybrid = load_example()
    lens = [1, 63, 64, 200, 5]
    eager, graph = (hybrid.HybridDecoder(len(lens), heads=8, heads_kv=2, layers=8, max_len=400, seed=3) for _ in range(2))
    for m in (eager, graph):
        m.admit(lens)
    history = {i: [] for i, x in enumerate(eager.layers) if "kv" in x}
    for step in range(4):
        for m in (eager, graph):
            m.step()
        if step == 0:
            graph.capture()
        torch.cuda.synchronize()
        assert torch.equal(eager.y, graph.y)
        assert eager.length.tolist() == [n + step + 1 for n in lens]
        assert eager.held.tolist() == [-(-(n + step + 1) // 64) for n in lens]
        assert eager.free_count.item() == eager.num_pages - sum(eager.held.tolist())
        for i in history:
            rows = eager.layers[i]["k"].flatten(0, 1)[eager.slots]
            history[i].append(rows.clone())
            assert torch.equal(rows, graph.layers[i]["k"].flatten(0, 1)[graph.slots])
    assert eager.status.item() == 0 and graph.status.item() == 0
    for i, rows in history.items():
        layer = eager.layers[i]
        latent = layer["kind"] == "latent"
        for b, n in enumerate(lens):
            total = n + 4
            pages = eager.table[b, :eager.held[b]].long()
            k = layer["k"][pages].flatten(0, 1)[:total]
            assert torch.equal(k[n:], torch.stack([r[b] for r in rows]))  # the appended rows, in order
            v = k[..., :512] if latent else layer["v"][pages].flatten(0, 1)[:total]
            for h in range(8):
                kh = 0 if latent else h // 4
                q = layer["q"][b, 0, h].double()
                scale = q.numel() ** -0.5
                s = k[:, kh].double() @ q * scale
                w = torch.softmax(s, 0)
                want, size = w @ v[:, kh].double(), w @ v[:, kh].double().abs()
                # output and weights rounded to bf16; scores summed in fp32 (see Problem.expected)
                off = (q.numel() + 4) * 2.0 ** -24 * float((k[:, kh].double().abs() @ q.abs()).max()) * scale + 2.0 ** -21
                tolerance = want.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2 * off + (total + 64) * 2.0 ** -24) * 1.01
                assert bool(((layer["o"][b, 0, h].double() - want).abs() <= tolerance).all()), (i, b, h)


def test_two_streams_at_once(gdn):
    """Calls that share the GPU, each with its workspace: the bits of the calls alone."""
    problems = [Problem(gdn, [900, 30, 2000, 0, 129], heads=8, heads_kv=2, dk=128, page=32, seed=11),
                Problem(gdn, [1500, 1, 700], heads=32, heads_kv=1, dk=576, dv=512, page=64, latent=True, seed=12),
                Problem(gdn, [64, 3000], heads=4, heads_kv=2, dk=48, page=10, T=2, seed=13)]
    alone = []
    for p in problems:
        p.call()
        torch.cuda.synchronize()
        alone.append((p.o.clone(), p.lse.clone()))
        p.o.zero_(), p.lse.zero_()
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    for _ in range(30):
        for p, s in zip(problems, streams):
            p.call(stream=s)
    torch.cuda.synchronize()
    for p, (o, lse) in zip(problems, alone):
        assert torch.equal(p.o, o) and torch.equal(p.lse, lse) and p.status.item() == 0
