"""The marshalling module's file: which one is loaded, and when it is built anew."""
import sysconfig

import torch

from fine_grained_moe_gemm_b200 import build


def test_binding_file_names_torch_and_the_interpreter():
    """A second interpreter or torch in the same checkout must not find the other's module fresh and load it."""
    name = build.binding_path()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")      # such as .cpython-312-x86_64-linux-gnu.so
    assert sysconfig.get_config_var("SOABI") in suffix and name.endswith(suffix)
    assert "".join(c if c.isalnum() else "_" for c in torch.__version__) in name
