"""GPU tests of the serving operators at the edges of their inputs, against the plain 64-bit forms.

Tolerances are those of test_serve_gpu.py.
"""
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
import serve_ref as ref
from test_serve_gpu import BF, F32, attend_case, check_attend, close, gen, offsets, rms, scan_inputs, scan_ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = [(F32, 128, cg.ATTEND_ROWS), (F32, 64, cg.ATTEND_ROWS), (BF, 128, cg.ATTEND_ROWS), (BF, 32, cg.ATTEND_ROWS),
           (BF, 128, cg.ATTEND_TILES)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_channelwise_gb300 import build
    build.build()
    cg.lib()


# ------------------------------------------------------------------------------------ attention


@pytest.mark.parametrize("dtype,D,path", KERNELS)
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-6, 1e-8, 1e-20])
def test_attend_pages_of_zeros_beside_small_values(dtype, D, path, size):
    """Attention is linear in v: a third of the pages hold zeros, the others values of any size."""
    kv_lens = [200, 333, 64]
    case = attend_case(50, [1, 40, 3], kv_lens, 4, 2, D, 16, dtype)
    vs, table = case[4], case[5]
    vs *= size
    for b, kv in enumerate(kv_lens):
        vs[table[b, :-(-kv // 16):3].long()] = 0
    check_attend(case, dtype, path=path)


@pytest.mark.parametrize("dtype,D,path", KERNELS)
def test_attend_nothing_but_zeros(dtype, D, path):
    case = attend_case(52, [1, 40], [5000, 333], 4, 2, D, 16, dtype)
    case[4].zero_()
    assert not check_attend(case, dtype, path=path).any()


@pytest.mark.parametrize("dtype,D,path", KERNELS)
@pytest.mark.parametrize("which", [3, 4])                                # k's scale, v's
def test_attend_nan_scale_reaches_only_the_rows_that_see_its_page(dtype, D, path, which):
    """Prompts over six and ten pages, a later one with a NaN scale: rows before it are as if it were not there."""
    case = attend_case(51, [90, 7], [90, 150], 4, 2, D, 16, dtype)
    table = case[5]
    case[which][table[0, 5]] = float("nan")
    case[which][table[1, 9], 1] = float("nan")                           # of one head, seen by the last six rows
    o = check_attend(case, dtype, path=path)                             # NaN exactly where the formula has it
    assert torch.isfinite(o[:80]).all() and torch.isnan(o[80:90]).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_attend_more_pages_than_a_block_holds_at_a_time(dtype):
    """29 requests that share 325 pages of 16 tokens: 928 units with a block each, which looks up 320 pages, then the rest."""
    B, page, kv, Hkv, D = 29, 16, 5200, 32, 32
    q, kc, vc, ks, vs, table, _, _ = attend_case(53, [9 * B], [kv], Hkv, Hkv, D, page, dtype)
    lens = torch.full((B,), kv, dtype=torch.int32, device="cuda")
    case = (q, kc, vc, ks, vs, table.expand(B, -1).contiguous(), lens, offsets([9] * B))
    assert cg.cache_attend_workspace_size(B, 9 * B, Hkv, Hkv, D, page, table.shape[1], max_q=9, max_kv=kv, dtype=dtype) == 0
    check_attend(case, dtype)


@pytest.mark.parametrize("path", [cg.ATTEND_AUTO, cg.ATTEND_ROWS, cg.ATTEND_TILES])
def test_attend_one_prompt_among_many_single_tokens_bf16(path):
    q_lens = [1] * 20 + [600] + [0, 1] * 10
    kv_lens = [(37 * i) % 300 for i in range(20)] + [700] + [5, 129] * 10
    check_attend(attend_case(54, q_lens, kv_lens, 8, 2, 128, 32, BF), BF, path=path)


# ------------------------------------------------------------------------------------ scan


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [16, 64])
@pytest.mark.parametrize("lens", [[5000], [3000, 0, 1701, 40]])
def test_scan_many_chunks(dtype, N, lens):
    """Sequences of dozens of chunks.  The states here forget within some 300 tokens (rates of 0.4 a unit of time
    and more, steps of 0.03 and more in all but a few), so the bound for 300 tokens holds for any number."""
    g = gen(12 + N)
    n, B, cu = sum(lens), len(lens), offsets(lens)
    s = scan_inputs(g, n, B, 24, N, 1, dtype, True)
    assert cg.scan_workspace_size(B, 0, 24, N, n_tokens=n, dtype=dtype) > 20 * 4 * 24 * N
    want, new = scan_ref(s, ref.spans_of(0, 0, cu))
    o = cg.scan_prefill(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["state"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                        cu_seqlens=cu)
    close(o, want, 1e-4 * rms(want), dtype)
    close(s["state"], new, 1e-4 * rms(new))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [16, 128])
@pytest.mark.parametrize("lens", [[1], [3, 9], [200]])                   # a step, ragged tiles, a prompt in chunks
def test_scan_rates_beyond_fp32(dtype, N, lens):
    """A third of the states decay by exp(100) a unit of time, a channel takes steps that round to zero."""
    g = gen(11)
    n, B, cu = sum(lens), len(lens), offsets(lens)
    s = scan_inputs(g, n, B, 24, N, 1, dtype, True)
    s["A_log"][:, ::3] = 100.0
    s["dt"][:, 5] = -200.0
    want, new = scan_ref(s, ref.spans_of(0, 0, cu))
    args = [s[k] for k in ("x", "dt", "A_log", "Bm", "Cm", "state")]
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    o = cg.scan_decode(*args, **kw) if n == 1 else cg.scan_prefill(*args, cu_seqlens=cu, **kw)
    close(o, want, 1e-4 * rms(want), dtype)
    close(s["state"], new, 1e-4 * rms(new))


# ------------------------------------------------------------------------------------ cache plan


FRESH_PLAN = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import gated_delta_rule_channelwise_gb300 as cg
B = int(sys.argv[2])
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
p = cg.cache_plan(torch.zeros(B, 1, dtype=torch.int32, device="cuda"), ints([0] * B), ints([1] * B), ints(list(range(B))),
                  ints([B]), B, 16)
assert p.slots.tolist() == [16 * (B - 1 - b) for b in range(B)] and p.free_count.tolist() == [0]
"""


@pytest.mark.parametrize("B", [6127, 6128, 6143, 6144])                  # around 48 KB of shared memory
def test_plan_of_any_size_in_a_fresh_process(B):
    """Whether a launch is accepted does not depend on the calls before it."""
    r = subprocess.run([sys.executable, "-c", FRESH_PLAN, ROOT, str(B)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
