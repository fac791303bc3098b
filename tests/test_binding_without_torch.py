"""The ctypes side of the binding (library, exports, structures) needs no torch."""
import os
import subprocess
import sys

from tests._util import ROOT, ensure_built

CODE = """
import ctypes, sys
{block}
from transformer_esm_layer_gb300 import binding
assert {absent}
lib = binding.load_library()
assert all(hasattr(lib, n) for n in binding.EXPORTS)
w = binding.EsmAttnWindow(1, 1, 0)
assert lib.esm_encoder_set_attention_window(None, ctypes.byref(w)) == 1
assert lib.esm_encoder_check(None, None) == 1
{after}
"""


def _run(**parts):
    ensure_built()
    r = subprocess.run([sys.executable, "-c", CODE.format(**parts)], cwd=ROOT, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0, r.stderr


def test_where_torch_cannot_be_imported():
    _run(block="sys.modules['torch'] = None", absent="sys.modules['torch'] is None",
         after="try:\n    binding._stream_ptr(None)\nexcept ImportError:\n    pass\nelse:\n    raise AssertionError")


def test_torch_is_imported_at_its_first_use():
    _run(block="", absent="'torch' not in sys.modules",
         after="try:\n    binding._check_workspace(0, 'x', None)\nexcept ValueError:\n    pass\n"
               "assert binding.torch is sys.modules['torch']")
