"""C-ABI checks of the serving operators that need no GPU: argument blocks and refusals.

No call here launches a kernel: the pointers are made up, and each call is refused or has no work."""
import os
import subprocess

import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import build as cbuild
from gated_delta_rule_channelwise_gb300 import serve

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
BLOCKS = {"cgdr_conv_args": serve.CONV, "cgdr_scan_args": serve.SCAN, "cgdr_plan_args": serve.PLAN,
          "cgdr_append_args": serve.APPEND, "cgdr_attend_args": serve.ATTEND}


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cg.lib()


def test_blocks_match_the_c_structs(tmp_path):
    body = "".join('printf("%s . %%zu\\n", sizeof(%s));\n' % (s, s) + "".join(
        'printf("%s %s %%zu\\n", offsetof(%s, %s));\n' % (s, f, s, f) for f, _ in b.fields) for s, b in BLOCKS.items())
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "cgdr_serve.h"\nint main(void){%sreturn 0;}\n' % body)
    subprocess.run(["gcc", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        s, f, at = line.split()
        assert int(at) == (BLOCKS[s].size if f == "." else BLOCKS[s].offset(f)), (s, f)


P = 1 << 20     # a made-up, aligned address

CONV = dict(B=2, T=5, C=64, W=4, dtype=cg.BF16, silu=1, n_tokens=0, reserved=0, x=P, x_sb=5 * 64, x_st=64, o=2 * P,
            o_sb=5 * 64, o_st=64, weight=3 * P, bias=0, state=4 * P, cu=0, status=0)
SCAN = dict(B=2, T=5, C=64, N=16, G=2, dtype=cg.BF16, o_dtype=cg.BF16, softplus=1, n_tokens=0, reserved=0, x=P,
            x_sb=320, x_st=64, dt=P, dt_sb=320, dt_st=64, z=0, z_sb=0, z_st=0, Bm=P, Bm_sb=160, Bm_st=32, Cm=P,
            Cm_sb=160, Cm_st=32, o=2 * P, o_sb=320, o_st=64, A_log=3 * P, D=0, dt_bias=0, state=4 * P, cu=0, status=0)
PLAN = dict(B=2, width=8, page=16, n_tokens=4, F=3, num_pages=99, block_table=P, table_sb=8, seq_lens=2 * P,
            new_lens=3 * P, free_pages=4 * P, free_count=5 * P, free_count_out=6 * P, kv_lens=7 * P, cu=8 * P,
            requests=9 * P, positions=10 * P, slots=11 * P, status=0)
APPEND = dict(n=3, Hkv=2, D=64, page=16, dtype=cg.BF16, num_pages=9, k=P, k_st=128, k_sh=64, v=2 * P, v_st=128, v_sh=64,
              slots=3 * P, k_cache=4 * P, v_cache=5 * P, k_scale=6 * P, v_scale=7 * P, status=0)
ATTEND = dict(B=2, n=2, Hq=4, Hkv=2, D=64, page=16, width=8, dtype=cg.BF16, num_pages=9, max_q=1, max_kv=100, path=0,
              wait_polls=0, scale=0.0,
              q=P, q_st=256, q_sh=64, o=2 * P, o_st=256, o_sh=64, k_cache=3 * P, v_cache=4 * P, k_scale=5 * P,
              v_scale=6 * P, block_table=7 * P, table_sb=8, kv_lens=8 * P, cu=9 * P, status=0)


def call(lib, name, good, **kw):
    values = dict(good, **kw)
    block = {"conv": serve.CONV, "scan": serve.SCAN, "plan": serve.PLAN, "append": serve.APPEND, "attend": serve.ATTEND}[name]
    args = block.pack(*(values[f] for f, _ in block.fields))
    if name == "scan":
        return lib.cgdr_scan(args, None, 0, None)
    if name == "attend":
        return lib.cgdr_cache_attend(args, None, 0, None)
    return {"conv": lib.cgdr_conv, "plan": lib.cgdr_cache_plan, "append": lib.cgdr_cache_append}[name](args, None)


INV, UNS, ALN = cg.ERR_INVALID_ARG, cg.ERR_UNSUPPORTED, cg.ERR_ALIGNMENT


@pytest.mark.parametrize("name,good,kw,code", [
    ("conv", CONV, dict(B=-1), INV), ("conv", CONV, dict(C=0), INV), ("conv", CONV, dict(T=-1), INV),
    ("conv", CONV, dict(cu=P, n_tokens=-1), INV), ("conv", CONV, dict(x=0), INV), ("conv", CONV, dict(weight=0), INV),
    ("conv", CONV, dict(state=0), INV), ("conv", CONV, dict(W=1), UNS), ("conv", CONV, dict(W=5), UNS),
    ("conv", CONV, dict(C=60), UNS), ("conv", CONV, dict(dtype=2), UNS), ("conv", CONV, dict(B=1 << 20, T=1 << 20), UNS),
    ("conv", CONV, dict(x=P + 2), ALN), ("conv", CONV, dict(x_st=68), ALN), ("conv", CONV, dict(o_sb=-64), ALN),
    ("conv", CONV, dict(cu=P + 2, n_tokens=4), ALN), ("conv", CONV, dict(state=P + 8), ALN),
    ("scan", SCAN, dict(G=0), INV), ("scan", SCAN, dict(G=3), INV), ("scan", SCAN, dict(A_log=0), INV),
    ("scan", SCAN, dict(Cm=0), INV), ("scan", SCAN, dict(N=8), UNS), ("scan", SCAN, dict(N=48), UNS),
    ("scan", SCAN, dict(C=40), UNS), ("scan", SCAN, dict(o_dtype=5), UNS), ("scan", SCAN, dict(B=40000), UNS),
    ("scan", SCAN, dict(dt_st=4), ALN), ("scan", SCAN, dict(z=P, z_sb=4), ALN), ("scan", SCAN, dict(state=P + 4), ALN),
    ("plan", PLAN, dict(B=-1), INV), ("plan", PLAN, dict(n_tokens=-1), INV), ("plan", PLAN, dict(free_count=0), INV),
    ("plan", PLAN, dict(seq_lens=0), INV), ("plan", PLAN, dict(slots=0), INV), ("plan", PLAN, dict(table_sb=7), INV),
    ("plan", PLAN, dict(free_count_out=5 * P), INV), ("plan", PLAN, dict(kv_lens=2 * P), INV),
    ("plan", PLAN, dict(free_pages=0), INV), ("plan", PLAN, dict(page=48), UNS), ("plan", PLAN, dict(B=8193), UNS),
    ("plan", PLAN, dict(slots=P + 4), ALN), ("plan", PLAN, dict(cu=P + 2), ALN),
    ("append", APPEND, dict(n=-1), INV), ("append", APPEND, dict(Hkv=0), INV), ("append", APPEND, dict(v_scale=0), INV),
    ("append", APPEND, dict(D=96), UNS), ("append", APPEND, dict(page=8), UNS), ("append", APPEND, dict(dtype=9), UNS),
    ("append", APPEND, dict(k=P + 8), ALN), ("append", APPEND, dict(v_sh=60), ALN), ("append", APPEND, dict(k_cache=P + 8), ALN),
    ("attend", ATTEND, dict(Hq=3), INV), ("attend", ATTEND, dict(path=3), INV), ("attend", ATTEND, dict(path=-1), INV), ("attend", ATTEND, dict(max_q=-1), INV), ("attend", ATTEND, dict(q=0), INV),
    ("attend", ATTEND, dict(cu=0), INV), ("attend", ATTEND, dict(block_table=0), INV), ("attend", ATTEND, dict(table_sb=4), INV),
    ("attend", ATTEND, dict(D=256), UNS), ("attend", ATTEND, dict(page=24), UNS), ("attend", ATTEND, dict(max_kv=1 << 30), UNS),
    ("attend", ATTEND, dict(q_st=4), ALN), ("attend", ATTEND, dict(v_cache=P + 4), ALN), ("attend", ATTEND, dict(o_sh=-1), ALN),
    ("attend", ATTEND, dict(max_kv=1 << 20, width=1 << 16, table_sb=1 << 16), cg.ERR_WORKSPACE),
])
def test_refusals(lib, name, good, kw, code):
    assert call(lib, name, good, **kw) == code


@pytest.mark.parametrize("name,good,kw", [
    ("conv", CONV, dict(B=0, x=0, o=0, weight=0, state=0)), ("conv", CONV, dict(T=0, x=0, o=0)),
    ("conv", CONV, dict(cu=P, n_tokens=0, x=0)), ("scan", SCAN, dict(B=0, x=0, A_log=0)), ("scan", SCAN, dict(T=0, x=0)),
    ("append", APPEND, dict(n=0, k=0, v=0, slots=0)), ("attend", ATTEND, dict(n=0, q=0, o=0)),
    ("attend", ATTEND, dict(B=0)), ("attend", ATTEND, dict(max_q=0))])
def test_nothing_to_do(lib, name, good, kw):
    assert call(lib, name, good, **kw) == cg.OK


def test_null_blocks(lib):
    assert lib.cgdr_conv(None, None) == INV and lib.cgdr_scan(None, None, 0, None) == INV
    assert lib.cgdr_cache_plan(None, None) == INV and lib.cgdr_cache_append(None, None) == INV
    assert lib.cgdr_cache_attend(None, None, 0, None) == INV
    assert lib.cgdr_scan_workspace_size(None) == 0 and lib.cgdr_cache_attend_workspace_size(None) == 0


def test_workspace_sizes(lib):
    assert cg.scan_workspace_size(64, 1, 4096, 16) == 0                       # single tokens
    assert cg.scan_workspace_size(64, 100, 4096, 16) == 0                     # enough sequences: no chunks
    assert cg.scan_workspace_size(1, 16384, 64, 16) > 0
    assert cg.cache_attend_workspace_size(1, 1, 32, 8, 128, 64, 2048, max_q=1) > 0
    assert cg.cache_attend_workspace_size(64, 64, 32, 8, 128, 64, 2, max_q=1) == 0
    big = dict(max_q=2000, max_kv=4000)                                       # enough rows: tiles, which need none
    assert cg.cache_attend_workspace_size(4, 8000, 32, 8, 128, 64, 64, **big) == 0
    assert cg.cache_attend_workspace_size(4, 8000, 32, 8, 128, 64, 64, path=cg.ATTEND_ROWS, **big) == 0   # a block a unit
    few = dict(max_q=40, max_kv=100000)                                       # few units of many steps: the cache is split
    assert cg.cache_attend_workspace_size(1, 40, 32, 8, 128, 64, 1600, path=cg.ATTEND_TILES, **few) > 0
    assert cg.cache_attend_workspace_size(1, 40, 32, 8, 128, 64, 1600, path=cg.ATTEND_ROWS, **few) > 0
    assert cg.cache_attend_workspace_size(1, 40, 32, 8, 128, 64, 3, path=cg.ATTEND_TILES, **few) == 0


def test_python_checks_types_and_shapes():
    """What the binding refuses before the library is reached: it has no CPU path, and shapes have to agree."""
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    with pytest.raises(ValueError, match="CUDA"):
        cg.conv_prefill(z(1, 2, 8), z(8, 4), z(1, 3, 8))
    with pytest.raises(ValueError, match="packed"):
        cg.conv_prefill(z(2, 8), z(8, 4), z(1, 3, 8))
    with pytest.raises(ValueError, match=r"\[B, C\]"):
        cg.conv_decode(z(1, 1, 8), z(8, 4), z(1, 3, 8))
    with pytest.raises(ValueError, match="CUDA"):
        cg.scan_decode(z(1, 8), z(1, 8), z(8, 16), z(1, 1, 16), z(1, 1, 16), z(1, 8, 16))
    with pytest.raises(ValueError, match="scan|packed|Bm"):
        cg.scan_prefill(z(2, 8), z(2, 8), z(8, 16), z(2, 1, 16), z(2, 1, 16), z(1, 8, 16))
    with pytest.raises(ValueError, match="CUDA"):
        cg.cache_append(z(1, 1, 32), z(1, 1, 32), z(1, dtype=torch.int64), *[z(2, 1, 16, 32, dtype=torch.int8)] * 2, z(2, 1), z(2, 1))
