"""Importing the package, its build module and the C ABI needs no torch; the calls are there when torch is."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = """
import sys
sys.modules["torch"] = None                # importing torch now fails
sys.path.insert(0, sys.argv[1])
from gated_delta_rule_channelwise_gb300 import *
import gated_delta_rule_channelwise_gb300 as cg
from gated_delta_rule_channelwise_gb300 import build
build.build()
assert cg.lib().cgdr_abi_version() > 0 and "cgdr_conv" in dir(cg.lib()) and cg.status_string(cg.OK)
try:
    cg.conv_decode
except ImportError:
    print("fine")
"""
WITH = """
import sys
sys.path.insert(0, sys.argv[1])
import gated_delta_rule_channelwise_gb300 as cg
assert "torch" not in sys.modules          # nor does it load one that is there
assert not hasattr(cg, "no_such_call") and "cache_plan" in dir(cg)
from gated_delta_rule_channelwise_gb300 import *
assert conv_decode is cg.conv_decode is cg.serve.conv_decode and set(cg.__all__) <= set(dir(cg))
print("fine")
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", code, ROOT], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout.split()


def test_without_torch():
    assert run(WITHOUT) == ["fine"]


def test_with_torch():
    assert run(WITH) == ["fine"]
