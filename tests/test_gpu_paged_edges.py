"""Paged-cache calls at their edges: rings that hold one tile, waits that run out, padding over several
steps, batches around the shared-memory limit, values that are no numbers among the newest positions."""
import pytest
import torch

from test_gpu_paged import Problem, name_of

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
