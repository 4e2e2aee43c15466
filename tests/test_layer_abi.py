"""C-ABI checks of the operators around a layer's state that need no GPU: argument blocks and refusals.

No call here launches a kernel: the pointers are made up, and each call is refused or has no work."""
import os
import subprocess

import pytest
import torch

import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import build as cbuild
from gated_delta_rule_channelwise_gb300 import layer

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
BLOCKS = {"cgdr_norm_args": layer.NORM, "cgdr_quantize_args": layer.QUANTIZE, "cgdr_matmul_args": layer.MATMUL, "cgdr_rotary_args": layer.ROTARY}


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cg.lib()


def test_blocks_match_the_c_structs(tmp_path):
    body = "".join('printf("%s . %%zu\\n", sizeof(%s));\n' % (s, s) + "".join(
        'printf("%s %s %%zu\\n", offsetof(%s, %s));\n' % (s, f, s, f) for f, _ in b.fields) for s, b in BLOCKS.items())
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "cgdr_layer.h"\nint main(void){%sreturn 0;}\n' % body)
    subprocess.run(["gcc", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        s, f, at = line.split()
        assert int(at) == (BLOCKS[s].size if f == "." else BLOCKS[s].offset(f)), (s, f)


P = 1 << 20     # a made-up, aligned address

NORM = dict(n=3, H=1, C=64, dtype=cg.BF16, eps=1e-6, x=P, x_st=64, x_sh=0, residual=2 * P, residual_st=64, residual_sh=0, weight=3 * P,
            o=4 * P, o_st=64, o_sh=0, y8=0, y8_st=0, y_scale=0, status=0)
NORM8 = dict(NORM, o=0, o_st=0, y8=5 * P, y8_st=64, y_scale=6 * P)
QUANTIZE = dict(n=3, C=64, dtype=cg.F32, block_rows=1, x=P, x_st=64, y8=2 * P, y8_st=64, y_scale=3 * P, status=0)
MATMUL = dict(n=3, N=64, K=256, o_dtype=cg.BF16, path=0, wait_polls=0, x=P, x_st=256, x_scale=2 * P, w=3 * P, w_st=256, w_scale=4 * P,
              o=5 * P, o_st=64, status=0)
ROTARY = dict(n=3, Hq=4, Hk=2, D=64, half=32, dtype=cg.BF16, interleaved=0, scale=1.0, q=P, q_st=256, q_sh=64, k=2 * P, k_st=128, k_sh=64,
              positions=3 * P, freq=4 * P, status=0)
CALLS = {"norm": (layer.NORM, "cgdr_norm"), "quantize": (layer.QUANTIZE, "cgdr_quantize"), "matmul": (layer.MATMUL, "cgdr_matmul"),
         "rotary": (layer.ROTARY, "cgdr_rotary")}


def call(lib, name, good, **kw):
    values = dict(good, **kw)
    block, fn = CALLS[name]
    return getattr(lib, fn)(block.pack(*(values[f] for f, _ in block.fields)), None)


INV, UNS, ALN = cg.ERR_INVALID_ARG, cg.ERR_UNSUPPORTED, cg.ERR_ALIGNMENT


@pytest.mark.parametrize("name,good,kw,code", [
    ("norm", NORM, dict(n=-1), INV), ("norm", NORM, dict(C=0), INV), ("norm", NORM, dict(H=0), INV), ("norm", NORM, dict(x=0), INV),
    ("norm", NORM, dict(o=0), INV), ("norm", NORM, dict(y8=7 * P, y8_st=64, y_scale=P), INV), ("norm", NORM8, dict(y_scale=0), INV),
    ("norm", NORM, dict(C=60), UNS), ("norm", NORM, dict(C=32776), UNS), ("norm", NORM, dict(dtype=2), UNS), ("norm", NORM8, dict(H=2), UNS),
    ("norm", NORM, dict(x=P + 8), ALN), ("norm", NORM, dict(weight=P + 4), ALN), ("norm", NORM, dict(x_st=60), ALN), ("norm", NORM, dict(o_st=68), ALN),
    ("norm", NORM, dict(residual_st=66), ALN), ("norm", NORM8, dict(y8_st=72), ALN),
    ("norm", NORM, dict(o_st=0), INV), ("norm", NORM, dict(residual_st=32), INV), ("norm", NORM8, dict(y8_st=48), INV),     # rows that overlap
    ("norm", NORM, dict(H=2, o_sh=0, o_st=128, x_sh=64, residual_sh=64, residual_st=128), INV),
    ("quantize", QUANTIZE, dict(n=-1), INV), ("quantize", QUANTIZE, dict(C=0), INV), ("quantize", QUANTIZE, dict(x=0), INV),
    ("quantize", QUANTIZE, dict(y_scale=0), INV), ("quantize", QUANTIZE, dict(C=68), UNS), ("quantize", QUANTIZE, dict(block_rows=64), UNS),
    ("quantize", QUANTIZE, dict(dtype=7), UNS), ("quantize", QUANTIZE, dict(n=1 << 29, C=1024, x_st=1024, y8_st=1024), UNS),
    ("quantize", QUANTIZE, dict(x=P + 4), ALN), ("quantize", QUANTIZE, dict(x_st=66), ALN), ("quantize", QUANTIZE, dict(y8_st=72), ALN),
    ("quantize", QUANTIZE, dict(y8_st=32), INV),
    ("matmul", MATMUL, dict(n=-1), INV), ("matmul", MATMUL, dict(N=-1), INV), ("matmul", MATMUL, dict(K=0), INV), ("matmul", MATMUL, dict(path=3), INV),
    ("matmul", MATMUL, dict(path=-1), INV), ("matmul", MATMUL, dict(w=0), INV), ("matmul", MATMUL, dict(x_scale=0), INV), ("matmul", MATMUL, dict(o=0), INV),
    ("matmul", MATMUL, dict(o_st=56), INV), ("matmul", MATMUL, dict(o_dtype=2), UNS), ("matmul", MATMUL, dict(n=1 << 30, N=1 << 30, o_st=1 << 30), UNS),
    ("matmul", MATMUL, dict(x=P + 8), ALN), ("matmul", MATMUL, dict(w_st=264), ALN), ("matmul", MATMUL, dict(x_st=264), ALN), ("matmul", MATMUL, dict(o_st=68), ALN),
    ("matmul", MATMUL, dict(o=P + 8), ALN), ("matmul", MATMUL, dict(status=P + 2), ALN), ("matmul", MATMUL, dict(x_st=128), INV), ("matmul", MATMUL, dict(w_st=0), INV),
    ("rotary", ROTARY, dict(n=-1), INV), ("rotary", ROTARY, dict(Hq=0), INV), ("rotary", ROTARY, dict(half=0), INV), ("rotary", ROTARY, dict(half=33), INV),
    ("rotary", ROTARY, dict(q=0), INV), ("rotary", ROTARY, dict(k=0), INV), ("rotary", ROTARY, dict(positions=0), INV), ("rotary", ROTARY, dict(freq=0), INV),
    ("rotary", ROTARY, dict(k=P), INV), ("rotary", ROTARY, dict(q_sh=0), INV), ("rotary", ROTARY, dict(k_st=64), INV),                                         # heads that overlap
    ("rotary", ROTARY, dict(D=1024, half=512, q_sh=1024, q_st=4096, k_sh=1024, k_st=2048), UNS), ("rotary", ROTARY, dict(dtype=2), UNS),
    ("rotary", ROTARY, dict(Hk=70000, k_st=70000 * 64), UNS), ("rotary", ROTARY, dict(q=P + 2), ALN), ("rotary", ROTARY, dict(q_st=260), ALN),
    ("rotary", ROTARY, dict(freq=P + 4), ALN), ("rotary", ROTARY, dict(k_sh=65, k_st=200), ALN),
])
def test_refusals(lib, name, good, kw, code):
    assert call(lib, name, good, **kw) == code


@pytest.mark.parametrize("name,good,kw", [
    ("norm", NORM, dict(n=0, x=0, o=0)), ("norm", NORM8, dict(n=0, x=0)), ("quantize", QUANTIZE, dict(n=0, x=0, y8=0)),
    ("matmul", MATMUL, dict(n=0, x=0, o=0)), ("matmul", MATMUL, dict(N=0, w=0, o=0)), ("rotary", ROTARY, dict(n=0, q=0, k=0, positions=0))])
def test_nothing_to_do(lib, name, good, kw):
    assert call(lib, name, good, **kw) == cg.OK


def test_null_blocks(lib):
    for _, fn in CALLS.values():
        assert getattr(lib, fn)(None, None) == INV


def test_python_checks_types_and_shapes():
    """What the binding refuses before the library is reached: it has no CPU path, and shapes have to agree."""
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    E = torch.float8_e4m3fn
    with pytest.raises(ValueError, match="CUDA"):
        cg.rms_norm(z(2, 8), z(8))
    with pytest.raises(ValueError, match="n, C"):
        cg.rms_norm(z(8), z(8))
    with pytest.raises(ValueError, match="n, C"):
        cg.rms_norm_fp8(z(1, 2, 8), z(8))
    for eps in (-1e-6, float("nan")):
        with pytest.raises(ValueError, match="eps"):
            cg.rms_norm(z(2, 8), z(8), eps=eps)
    with pytest.raises(ValueError, match="CUDA"):
        cg.fp8_quantize(z(2, 16))
    with pytest.raises(ValueError, match="matrix"):
        cg.fp8_quantize_weight(z(2, 2, 16))
    with pytest.raises(TypeError, match="y must be"):
        cg.fp8_quantize(z(2, 16), z(2, 16))
    with pytest.raises(ValueError, match="y_scale must have shape"):
        cg.fp8_quantize(z(2, 16), z(2, 16, dtype=E), z(2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        cg.fp8_matmul(z(2, 16, dtype=E), z(2, 1), z(4, 16, dtype=E), z(1, 1))
    with pytest.raises(ValueError, match="CUDA"):
        cg.rotary(z(2, 1, 8), None, z(2, dtype=torch.int32), z(4, dtype=torch.float64))


# ------------------------------------------------------------------------------------ frequencies


def test_frequencies_without_scaling():
    freq, scale = cg.rotary_frequencies(8, device="cpu")
    assert scale == 1.0 and freq.dtype == torch.float64
    assert torch.allclose(freq, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)


def test_frequencies_scaled():
    R, factor = 64, 8.0
    plain, _ = cg.rotary_frequencies(R, device="cpu")
    linear, s = cg.rotary_frequencies(R, scaling="linear", factor=factor, device="cpu")
    assert s == 1.0 and torch.allclose(linear, plain / factor, rtol=1e-15)
    base, s = cg.rotary_frequencies(R, scaling="base", factor=factor, device="cpu")
    assert s == 1.0 and base[0] == 1 and abs(float(base[-1] * factor / plain[-1]) - 1) < 1e-12
    for scaling in ("turns", "ramp"):
        some, s = cg.rotary_frequencies(R, scaling=scaling, factor=factor, length=4096, device="cpu")
        assert some[0] == plain[0] and abs(float(some[-1] * factor / plain[-1]) - 1) < 1e-12      # 650 turns; 0.09
        assert (some <= plain).all() and (some >= plain / factor * (1 - 1e-15)).all() and (some[1:] < some[:-1]).all()
        turns = 4096 * plain / (2 * torch.pi)
        between = (turns < 32) & (turns > 1)
        assert between.any() and (some[between] < plain[between]).any()
        assert abs(s - (1.0 if scaling == "turns" else 1 + 0.1 * 2.0794415416798357)) < 1e-15     # 0.1 ln 8
        same, s = cg.rotary_frequencies(R, scaling=scaling, factor=1.0, device="cpu")
        assert torch.equal(same, plain) and s == 1.0


@pytest.mark.parametrize("kw", [dict(R=0), dict(R=7), dict(R=8, base=0.0), dict(R=8, factor=0.5), dict(R=8, scaling="none"), dict(R=8, length=0),
                                dict(R=8, scaling="turns", fast=1.0, slow=1.0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError):
        cg.rotary_frequencies(**kw, device="cpu")
