"""The package on a torch that lacks the element types of the MX formats: it
imports, every call that needs none of them is there, and the ones that do
refuse by name.  Run in a child process, whose torch is stripped before the
package is imported."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys
import torch
saved = {n: getattr(torch, n) for n in sys.argv[1:]}
for n in saved:
    delattr(torch, n)
import sparse_fp8_row_amd as sfr
sfr.load()
assert sfr.default_algo(16, 4096, 4096) >= 0 and callable(sfr.sparse_fp8_rowwise_linear)
x = torch.zeros((4, 64), dtype=torch.bfloat16)
e2m1, e8m0 = saved.get("float4_e2m1fn_x2"), saved.get("float8_e8m0fnu")
# the tables that every call looks its element type up in
assert None not in sfr._MX and None not in sfr._SAVE and e2m1 not in sfr._MX and e2m1 not in sfr._FP4
if e2m1 is not None:
    assert sfr._FP4 == ()
if e8m0 is not None:
    assert sfr._MX == {} and list(sfr._SAVE) == [torch.bfloat16]
else:
    assert sfr._SAVE == {torch.bfloat16: 1, torch.float8_e4m3fn: 2, torch.float8_e5m2: 3}
    assert sfr.MxTensor(x.view(torch.float8_e5m2), None).shape == (4, 128)
for parts in (sfr.MxTensor(x, x), sfr.MxTensor(x.view(torch.uint8).view(e2m1 or torch.float8_e5m2), x)):
    for kinds in (sfr._FP4, sfr._MX):  # what mxfp4_linear and dequantize_mx ask of their operand
        try:
            sfr._mx_parts(parts, "t", 0, kinds)
        except ValueError as e:
            assert "unsupported element type" in str(e) or "scale float8_e8m0fnu" in str(e), e
        else:
            raise AssertionError("not refused")
print("imported")
"""


@pytest.mark.parametrize("missing", [["float4_e2m1fn_x2"], ["float8_e8m0fnu"], ["float4_e2m1fn_x2", "float8_e8m0fnu"]],
                         ids=",".join)
def test_without_mx_types(missing):
    r = subprocess.run([sys.executable, "-c", CHILD, *missing], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr
