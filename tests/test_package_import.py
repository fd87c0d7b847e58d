"""Importing the package, all of its names included, asks for neither torch nor the built binding; a call of a layer operator
without the binding says how to build it (no GPU needed)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_every_name_without_torch():
    python("import sys; sys.modules['torch'] = None\n"
           "from state_space_sequence_ssd_gb300 import *\n"
           "import state_space_sequence_ssd_gb300 as ssd\n"
           "assert all(callable(getattr(ssd, n)) for n in ssd.__all__ if n != 'library_path')\n"
           "assert ssd_conv_forward is ssd.ssd_conv_forward and ssd_conv_forward.__doc__\n")


def test_a_missing_binding_is_named_when_it_is_needed():
    python("from state_space_sequence_ssd_gb300 import *\n"
           "from state_space_sequence_ssd_gb300 import layer\n"
           "layer._BINDING = '/nowhere/ssd_layer_binding.so'\n"
           "try:\n"
           "    ssd_layer_norm_forward(None)\n"
           "except RuntimeError as e:\n"
           "    assert 'build it with' in str(e) and '/nowhere' in str(e)\n"
           "else:\n"
           "    raise AssertionError('no error')\n")
