"""8-bit products whose device waits give up: what a block had under way is over before the block is.

A block that ends with copies still landing in its shared memory, or with products still reading it and writing its tensor
memory, spoils the block that gets both next.  The warps that copy and multiply may have issued all they had to when another
warp's wait gives up (K of few blocks, or the last blocks of any K), or may themselves be in a wait (K of more blocks than there
are stages and sums), so both lengths are here, for each tile width, with K in parts and whole.  Two hooks: a negative
``wait_polls`` makes the first wait of every CTA one for something that never comes, and a limit of one poll lets some
CTAs give up and others not.  The index-checking build looks, at each block's end, whether all it had issued is over.
"""
import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import layer
from test_layer_gpu import BF, operands
from test_serve_debug_gpu import checked  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

FEW, TILES = cg.MATMUL_FEW, cg.MATMUL_TILES
CASES = [(FEW, 4, 640, 512),                           # parts of 2 blocks, 5 stages and 4 sums
         (FEW, 4, 640, 12288), (FEW, 20, 300, 8200), (FEW, 40, 300, 12288),    # parts of 12, 9 (ragged) and 12 blocks; 16, 32 and 64 rows a tile
         (FEW, 64, 20000, 1500), (FEW, 64, 20000, 256),                        # K in one part, 12 blocks and 2
         (TILES, 300, 640, 512), (TILES, 300, 640, 4112),                      # 128 columns: 4 blocks, 33
         (TILES, 2500, 4096, 256), (TILES, 2500, 4096, 1000)]                  # 256 columns, three tiles a CTA: 2 blocks, 8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()



@pytest.mark.parametrize("case", CASES)
def test_nothing_is_under_way_at_a_blocks_end(monkeypatch, checked, case):  # noqa: F811
    path, n, N, K = case
    args = operands(60, n, N, K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = cg.fp8_matmul(*args, path=path)
    monkeypatch.setattr(layer, "lib", lambda: checked)
    for polls in (-3, -200):
        status.zero_()
        cg.fp8_matmul(*args, path=path, wait_polls=polls, status=status)
        assert int(status) == cg.ERR_TIMEOUT                              # and not the code of the check
    for polls in (1, 2, 10):
        status.zero_()
        got = cg.fp8_matmul(*args, path=path, wait_polls=polls, status=status)
        assert int(status) in (cg.OK, cg.ERR_TIMEOUT)
        assert int(status) == cg.ERR_TIMEOUT or torch.equal(got, want)
    status.zero_()
    assert torch.equal(cg.fp8_matmul(*args, path=path, status=status), want) and int(status) == cg.OK


@pytest.mark.parametrize("polls", [-3, 1])
@pytest.mark.parametrize("case", CASES)
def test_calls_that_follow_are_right(case, polls):
    """The next calls, of this shape and of others, take over the shared and tensor memory while nothing waits on the host."""
    path, n, N, K = case
    args, other = operands(60, n, N, K), operands(64, 130, 700, 900)
    spoiled, status = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    want, wants = cg.fp8_matmul(*args, path=path), {p: cg.fp8_matmul(*other, path=p, dtype=BF) for p in (FEW, TILES)}
    got = []
    for _ in range(10):
        cg.fp8_matmul(*args, path=path, wait_polls=polls, status=spoiled)
        got.append((cg.fp8_matmul(*args, path=path, status=status), want))
        for p in (FEW, TILES):
            cg.fp8_matmul(*args, path=path, wait_polls=polls, status=spoiled)
            got.append((cg.fp8_matmul(*other, path=p, dtype=BF, status=status), wants[p]))
    torch.cuda.synchronize()
    assert int(status) == cg.OK and int(spoiled) in ((cg.ERR_TIMEOUT,) if polls < 0 else (cg.OK, cg.ERR_TIMEOUT))
    assert all(torch.equal(a, b) for a, b in got)
