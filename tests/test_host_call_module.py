"""The marshalling module of the binding (csrc/gdn_call.c): whose it is, and what happens without it."""
import importlib.machinery
import os
import sysconfig

import pytest

import linear_attention_gdn_gb300 as gdn
from linear_attention_gdn_gb300 import build
from tests import test_host_step_qk
from tests.test_host_step_qk import P


def test_the_module_is_named_after_its_interpreter():
    """Another interpreter, whose objects lie otherwise in memory, must not load this one's file."""
    name = os.path.basename(build.CALL)
    assert name == "_gdn_call" + sysconfig.get_config_var("EXT_SUFFIX")
    assert name.endswith(importlib.machinery.EXTENSION_SUFFIXES[0]) and name != "_gdn_call.so"


def test_the_library_builds_without_python_headers(tmp_path, monkeypatch):
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    assert build.call_job(force=True)
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: paths)
    assert build.call_job(force=True) == []


@pytest.mark.parametrize("module", [True, False])
def test_calls_with_and_without_the_module(module, monkeypatch):
    """The same statuses either way, from entry points of 9, 11 and 14 pointers: addresses, None and a size."""
    if not module:
        monkeypatch.setattr(build, "CALL", build.CALL + ".none")
    monkeypatch.setattr(gdn, "_native", None)
    monkeypatch.setattr(gdn, "_entries", {})
    test_host_step_qk.test_step_with_nothing_to_do()
    assert (gdn._native is gdn._through_ctypes) == (not module)
    test_host_step_qk.test_step_refusals(gdn.gdn_step, {}, dict(beta=P + 4), 1)
    test_host_step_qk.test_step_refusals(gdn.gdn_kda_step, {}, dict(err=None), 1)
    test_host_step_qk.test_conv_step_refusals({}, dict(y=P + 2), 1)
    test_host_step_qk.test_qk_bad_arguments({}, 4, P + 4)
    test_host_step_qk.test_qk_documents_and_workspace()
