"""Paged-cache calls at their edges: rings that hold one tile, waits that run out, padding over several
steps, batches around the shared-memory limit, values that are no numbers among the newest positions."""
import time

import pytest
import torch

from test_gpu_paged import Problem, name_of, plan_reference, run_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import linear_attention_decode_gdn_gb300 as g
    return g


@pytest.mark.parametrize("shape", [dict(heads=24, heads_kv=1), dict(heads=32, heads_kv=2, T=4), dict(heads=16, heads_kv=1, T=2),
                                   dict(heads=16, heads_kv=1, T=3, window=1000), dict(heads=40, heads_kv=2, window=300)], ids=name_of)
def test_cold_requests_whose_last_tile_is_partial(gdn, shape):
    """Heads of 256 with more than 16 query rows a kv head: the ring of pages holds about one tile, so the
    rows that are zeroed in a partial tile are next to values that may still be on their way."""
    p = Problem(gdn, [9001, 130, 7777, 257, 1, 5003, 129, 2049], dk=256, page=64, seed=14, **shape)
    sweep = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(8):
        sweep.zero_()  # the pages come from memory
        p.call()
        if first is None:
            p.check()
            first = p.o.clone(), p.lse.clone()
        torch.cuda.synchronize()
        assert torch.equal(p.o, first[0]) and torch.equal(p.lse, first[1])


# ---- waits that run out ---------------------------------------------------------------------------
def starve(gdn, p, wait):
    """Problem p's call with a wait that runs out; how long it took."""
    from linear_attention_decode_gdn_gb300 import _abi, paged
    call = lambda kv, a, *rest: _abi.load().gdn_attn_starve_wait(kv, a, wait, *rest)  # noqa: E731
    torch.cuda.synchronize()
    begin = time.perf_counter()
    paged._attend(call, "gdn_attn_starve_wait", p.kv, p.q, p.table, p.kv_len, p.o, p.workspace, p.lse, p.scale, p.window, p.status, None)
    torch.cuda.synchronize()
    return time.perf_counter() - begin


STARVED = [dict(dk=128, page=64, heads=8, heads_kv=1), dict(dk=128, page=16, heads=48, heads_kv=1), dict(dk=64, page=32, heads=8, heads_kv=1),
           dict(dk=256, page=128, heads=40, heads_kv=1), dict(dk=576, dv=512, page=64, heads=16, heads_kv=1, latent=True),
           dict(dk=576, dv=512, page=32, heads=64, heads_kv=1, latent=True)]


@pytest.mark.parametrize("wait", [1, 2])
@pytest.mark.parametrize("shape", STARVED, ids=name_of)
def test_a_wait_that_runs_out_is_reported(gdn, shape, wait):
    p = Problem(gdn, [20000, 20000], seed=15, **shape)
    starve(gdn, p, wait)
    assert p.status.item() == gdn.STATUS_TIMEOUT
    p.status.zero_()
    p.call()  # the next call finds everything as it should be
    p.check()


def test_the_test_switch_is_checked(gdn):
    p = Problem(gdn, [30], dk=128, page=16)
    with pytest.raises(gdn.GDNError):
        starve(gdn, p, 3)
    p = Problem(gdn, [30], dk=32, page=16)
    with pytest.raises(gdn.GDNError):  # the kernel on the CUDA cores waits for nothing
        starve(gdn, p, 1)


def test_a_latent_call_that_gives_up_waits_for_its_own_loads_alone(gdn):
    """One limit until the wait for the first weights runs out, and no other for loads that were never begun."""
    took = []
    for shape in (STARVED[1], STARVED[5]):
        p = Problem(gdn, [20000, 20000], seed=16, **shape)
        p.call()
        took.append(min(starve(gdn, p, 2) for _ in range(2)))
        assert p.status.item() == gdn.STATUS_TIMEOUT
    assert took[1] < 1.4 * took[0], took


@pytest.mark.parametrize("wait", [1, 2])
@pytest.mark.parametrize("shape", STARVED, ids=name_of)
def test_what_is_given_up_is_not_written(gdn, shape, wait):
    """The first worker's share begins the first request, cut over several workers: its rows stay as they
    were, whatever the workspace held before, and those of the other requests are right."""
    p = Problem(gdn, [20000, 3000, 9000, 0, 15000], seed=17, **shape)
    q = Problem(gdn, [20000, 3000, 9000, 0, 15000], seed=18, **shape)
    q.workspace = p.workspace
    q.call()  # another call's sums are in the workspace
    starve(gdn, p, wait)
    assert p.status.item() == gdn.STATUS_TIMEOUT
    assert bool((p.o[0] == 7).all()) and bool((p.lse[0] == 7).all())
    want = p.o.clone(), p.lse.clone()
    p.status.zero_()
    p.call()
    p.check()
    assert torch.equal(p.o[1:], want[0][1:]) and torch.equal(p.lse[1:], want[1][1:])


@pytest.mark.parametrize("shape", [dict(dk=128, page=64, heads=8, heads_kv=2), dict(dk=64, page=16, heads=8, heads_kv=4, T=4),
                                   dict(dk=576, dv=512, page=64, heads=32, heads_kv=1, latent=True)], ids=name_of)
def test_rows_are_right_or_untouched_after_a_wait_ran_out(gdn, shape):
    """Short requests, many of them to a worker: each element is the one of an undisturbed call or is not written."""
    p = Problem(gdn, [3, 200, 129, 700] * 60, seed=19, **shape)
    starve(gdn, p, 1)
    assert p.status.item() == gdn.STATUS_TIMEOUT
    o, lse = p.o.clone(), p.lse.clone()
    p.call()
    torch.cuda.synchronize()
    assert bool(((o == p.o) | (o == 7)).all()) and bool(((lse == p.lse) | (lse == 7)).all())
    assert bool((o[:1] == 7).all()) and bool((o[-1] == p.o[-1]).all())


# ---- the plan -------------------------------------------------------------------------------------
PLANS = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import linear_attention_decode_gdn_gb300 as gdn
from test_gpu_paged import plan_reference, run_plan
for batch in (2030, 2036, 2037, 2038, 2042, 2045, 2047, 2048, 2444, 2445, 2450, 2454, 2455, 2457, 2458, 4096):
    cached = [b % 40 for b in range(batch)]
    held = [-(-c // 16) for c in cached]
    table, ids = [[-1] * 3 for _ in cached], list(range(4 * batch))
    for b, h in enumerate(held):
        table[b][:h] = [ids.pop() for _ in range(h)]
    args = (cached, None, held, table, ids, len(ids), 16, 4 * batch, batch)
    want, bad = plan_reference(*args)
    got, st = run_plan(gdn, *args, in_place={in_place})
    assert got == want and st == bad == 0, batch
print("planned")
"""


@pytest.mark.parametrize("in_place", [False, True])
def test_batches_around_the_shared_memory_limit(in_place):
    """Rising batches in a process of its own, so that no larger one has raised the kernel's limit before."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", PLANS.format(root=os.path.dirname(tests), tests=tests, in_place=in_place)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "planned" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("batch", [6, 1500])
@pytest.mark.parametrize("graph", [False, True])
def test_padding_lasts_over_steps_in_place(gdn, batch, graph):
    """Steps with kv_len, held_out and free_count_out in their inputs' arrays: rows retired with LEN_PADDING
    take no page and no slot in any of them, the live rows' slots close up, and attention leaves the retired
    rows of its output as they are. What -1 pads is an empty request after one step."""
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    page, width, heads, dk = 16, 4, 4, 64
    start = [gdn.LEN_PADDING if b % 3 == 1 else -77 if b % 3 == 2 and b % 2 else 14 + b % 5 for b in range(batch)]
    length, held = ints(start), ints([1 if n < 0 else -(-n // page) for n in start])
    pages = 3 * batch + 5
    table = [[-1] * width for _ in range(batch)]
    ids = list(range(pages))
    for b, h in enumerate(held.tolist()):
        table[b][:h] = [ids.pop() for _ in range(h)]
    free, count, cu = ints(ids), ints([len(ids)]), ints([0] * (batch + 1))
    table, slots, status = ints(table), torch.zeros(batch, dtype=torch.int64, device="cuda"), ints([0])
    k, v = (torch.randn(pages, page, 2, dk, device="cuda").bfloat16() for _ in range(2))
    kv = gdn.make_paged_kv(k, v)
    q = torch.randn(batch, 1, heads, dk, device="cuda").bfloat16()
    o = torch.full((batch, 1, heads, dk), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gdn.attn_workspace_bytes(kv, batch, 1, heads), dtype=torch.uint8, device="cuda")

    def step():
        gdn.kv_plan(length, None, held, table, free, count, kv_len=length, cu_new=cu, slot_map=slots, held_out=held,
                    free_count_out=count, page_size=page, num_pages=pages, status=status)
        gdn.attn_decode(kv, q, table, length, o, ws, status=status)

    run = step
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        run = captured.replay
    live = [b for b, n in enumerate(start) if n >= 0]
    for i in range(1, 5):
        run()
        torch.cuda.synchronize()
        assert status.item() == 0
        assert length.tolist() == [n + i if n >= 0 else n for n in start]
        want = [-(-(n + i) // page) if n >= 0 else 1 for n in start]
        assert held.tolist() == want and count.item() == pages - sum(want)
        sums = [0]
        for n in start:
            sums.append(sums[-1] + (n >= 0))
        assert cu.tolist() == sums
        rows = table.tolist()
        at = [rows[b][(start[b] + i - 1) // page] * page + (start[b] + i - 1) % page for b in live]
        assert slots.tolist() == at + [-1] * (batch - len(live)) and len(set(at)) == len(at)
        retired = torch.tensor([n < 0 for n in start], device="cuda")
        assert bool((o[retired] == 7).all()) and not bool((o[~retired] == 7).flatten(1).all(1).any())
    length[1] = -1
    run()
    assert length[1].item() == 0


# ---- values that are no numbers -------------------------------------------------------------------
@pytest.mark.parametrize("lens", [[1, 5, 128, 131, 700, 40], [9000, 260]], ids=lambda x: f"{len(x)}x{max(x)}")
@pytest.mark.parametrize("T,window", [(4, 0), (3, 130), (5, 2)])
@pytest.mark.parametrize("shape", [dict(dk=32, page=6, heads=4, heads_kv=2), dict(dk=64, page=16, heads=8, heads_kv=2),
                                   dict(dk=64, page=32, heads=20, heads_kv=1), dict(dk=128, page=64, heads=4, heads_kv=2),
                                   dict(dk=128, page=128, heads=32, heads_kv=2), dict(dk=256, page=32, heads=4, heads_kv=4),
                                   dict(dk=256, page=64, heads=24, heads_kv=2),
                                   dict(dk=576, dv=512, page=64, heads=4, heads_kv=1, latent=True),
                                   dict(dk=576, dv=512, page=32, heads=20, heads_kv=1, latent=True)], ids=name_of)
def test_values_that_only_some_positions_see(gdn, shape, T, window, lens):
    """The newest position's value holds NaN and infinities (of a latent row: the key too), and so does the oldest
    one that the first query sees through its window. Queries that do not see them give what they give without."""
    p = Problem(gdn, lens, T=T, window=window, seed=20, **shape)
    bad = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda").bfloat16()
    rows = p.k if p.latent else p.v
    first = {}  # by request: the oldest position, and the newest
    for b, n in enumerate(lens):
        spoiled = {n - 1}
        if window and n - T - window + 1 >= 0:
            spoiled.add(n - T - window + 1)
        for j in spoiled:
            rows[p.own_pages[b][j // p.page], j % p.page, :, 3::7] = bad[torch.arange(len(range(3, rows.shape[3], 7)), device="cuda") % 3]
        first[b] = sorted(spoiled)
    p.call()
    torch.cuda.synchronize()
    assert p.status.item() == 0
    for b, n in enumerate(lens):
        o, lse, to, tl = p.expected(b)
        got, got_lse = p.o[b].double(), p.lse[b].double()
        for t in range(T):
            pos = n - T + t
            sees = [j for j in first[b] if j <= pos and (not window or j > pos - window)]
            if not sees:
                assert bool(((got[t] - o[t]).abs() <= to[t]).all()), (b, n, t)
                assert bool(((got_lse[t] == lse[t]) | ((got_lse[t] - lse[t]).abs() <= tl[t])).all()), (b, n, t)
            elif p.latent:
                assert bool(torch.isnan(got[t]).all()), (b, n, t)
            else:
                whole = torch.ones(p.dv, dtype=torch.bool, device="cuda")
                whole[3::7] = False
                assert bool(((got[t] - o[t]).abs() <= to[t])[:, whole].all()), (b, n, t)
                assert not bool(torch.isfinite(got[t][:, ~whole]).any()), (b, n, t)
                assert torch.equal(torch.isnan(got[t]), torch.isnan(o[t])) and torch.equal(got[t] == float("inf"), o[t] == float("inf"))


def test_a_plan_without_a_free_list(gdn):
    """A list of no room (an empty tensor has no address): requests that need no page go on, the others are told."""
    args = ([3, 16, 7], None, [1, 1, 1], [[0, -1], [1, -1], [2, -1]], [], 0, 16, 3, 3)
    want, bad = plan_reference(*args)
    got, st = run_plan(gdn, *args)
    assert got == want and st == bad == gdn.STATUS_NO_PAGES


@pytest.mark.parametrize("T,window,heads", [(4, 0, 8), (7, 5, 8), (70, 0, 4), (70, 200, 4), (150, 60, 2)])
@pytest.mark.parametrize("shape", [dict(dk=64, page=32), dict(dk=128, page=16), dict(dk=256, page=64), dict(dk=128, page=128, permuted=True),
                                   dict(dk=48, page=9)], ids=name_of)
def test_values_of_every_newest_position(gdn, shape, T, window, heads):
    """Each of the newest positions (and of the oldest that a window leaves) spoils two value elements of its own:
    every query gives NaN and infinities where it sees them, and its sums everywhere else."""
    lens = [1, 140, 260, 1000]
    p = Problem(gdn, lens, T=T, window=window, heads=heads, heads_kv=2, seed=21, **shape)
    kinds = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda").bfloat16()
    for b, n in enumerate(lens):
        for j in range(max(0, n - T - window + 1 if window else n - T), n):
            row = p.v[p.own_pages[b][j // p.page], j % p.page]
            row[:, (5 * j) % p.dv], row[:, (5 * j + 11) % p.dv] = kinds[j % 3], kinds[(j // 3) % 3]
    p.call()
    torch.cuda.synchronize()
    assert p.status.item() == 0
    for b in range(len(lens)):
        o, lse, to, tl = p.expected(b)
        got, got_lse = p.o[b].double(), p.lse[b].double()
        number = torch.isfinite(o)
        assert torch.equal(torch.isnan(got), torch.isnan(o)) and torch.equal(got[~number].nan_to_num(0, 1, -1), o[~number].nan_to_num(0, 1, -1))
        assert bool(((got - o).abs() <= to)[number].all())
        assert bool(((got_lse == lse) | ((got_lse - lse).abs() <= tl)).all())


def test_a_spoiled_value_costs_little(gdn):
    """A request of 40,000 positions with NaN in its newest value takes no more than a few times what it takes without."""
    took = []
    for spoiled in (False, True):
        p = Problem(gdn, [40000, 30000], T=4, heads=16, heads_kv=1, dk=576, dv=512, page=64, latent=True, seed=22)
        if spoiled:
            p.k[p.own_pages[0][39999 // 64], 39999 % 64, 0, 100] = float("nan")
        p.call()
        torch.cuda.synchronize()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(20):
            p.call()
        end.record()
        torch.cuda.synchronize()
        took.append(begin.elapsed_time(end))
    assert took[1] < 4 * took[0], took
