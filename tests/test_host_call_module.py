"""The marshalling module of the binding (csrc/gdn_call.c): whose it is."""
import importlib.machinery
import os
import sysconfig

from linear_attention_gdn_gb300 import build


def test_the_module_is_named_after_its_interpreter():
    """Another interpreter, whose objects lie otherwise in memory, must not load this one's file."""
    name = os.path.basename(build.CALL)
    assert name == "_gdn_call" + sysconfig.get_config_var("EXT_SUFFIX")
    assert name.endswith(importlib.machinery.EXTENSION_SUFFIXES[0]) and name != "_gdn_call.so"
