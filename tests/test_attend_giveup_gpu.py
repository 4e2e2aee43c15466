"""Attention of prompts over the 8-bit cache whose device waits give up: no product is under way when its block ends.

The warps that issue products may have issued all of them when the softmax threads give up (a cache of one step of 64 tokens, or
the last steps of any), or may be in a wait themselves.  A block that ended then would free tensor memory that is still written.
"""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import serve
from test_serve_debug_gpu import checked  # noqa: F401 (a fixture)
from test_serve_gpu import BF, attend_case

pytestmark = pytest.mark.gpu

CASES = [([150], [60], 4, 2),                          # one step; tiles of 128 rows in pairs
         ([20], [20], 4, 2),                           # one tile
         ([150, 20], [700, 300], 4, 2), ([70], [3001], 4, 1)]     # several steps; the cache in parts


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


def attend(case, **kw):
    q, kc, vc, ks, vs, table, kv, cu = case[0]
    return cg.cache_attend(q, kc, vc, ks, vs, table, kv, cu, max_q=max(case[1]), max_kv=max(case[2]), path=cg.ATTEND_TILES, **kw)


def made(seed, sizes):
    q_lens, kv_lens, Hq, Hkv = sizes
    return attend_case(seed, q_lens, kv_lens, Hq, Hkv, 128, 64, BF), q_lens, kv_lens


@pytest.mark.parametrize("sizes", CASES)
def test_nothing_is_under_way_at_a_blocks_end(monkeypatch, checked, sizes):  # noqa: F811
    case, status = made(8, sizes), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = attend(case)
    monkeypatch.setattr(serve, "lib", lambda: checked)
    for polls in (-3, -200):
        status.zero_()
        attend(case, status=status, wait_polls=polls)
        assert int(status) == cg.ERR_TIMEOUT                              # and not the code of the check
    for polls in (1, 2, 10):
        status.zero_()
        got = attend(case, status=status, wait_polls=polls)
        assert int(status) in (cg.OK, cg.ERR_TIMEOUT)
        assert int(status) == cg.ERR_TIMEOUT or torch.equal(got, want)
    status.zero_()
    assert torch.equal(attend(case, status=status), want) and int(status) == cg.OK


@pytest.mark.parametrize("polls", [-3, 1])
@pytest.mark.parametrize("sizes", CASES)
def test_calls_that_follow_are_right(sizes, polls):
    case, status, spoiled = made(8, sizes), *(torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    want, got = attend(case), []
    for _ in range(10):
        attend(case, status=spoiled, wait_polls=polls)
        got.append(attend(case, status=status))
    torch.cuda.synchronize()
    assert int(status) == cg.OK and int(spoiled) in ((cg.ERR_TIMEOUT,) if polls < 0 else (cg.OK, cg.ERR_TIMEOUT))
    assert all(torch.equal(o, want) for o in got)
