"""Host-side checks of the selective state space layers' calls at edges that the other tests leave out. Only
invalid arguments reach the library."""
import ctypes
import random

import pytest

from test_selective_host import BAD, FAKE, NO, gdn, ssm  # noqa: F401


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
