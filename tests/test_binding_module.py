"""The binding's compiled module is optional: neither a build without it nor a
module that this interpreter cannot load keeps the library from working."""
import importlib.util
import os
import shutil
import sys
import sysconfig
import warnings

import pytest

import mixed_precision_numerics_amd as amp
from mixed_precision_numerics_amd import build


@pytest.mark.parametrize("compiler", ["/bin/false", "/nonexistent/compiler"])
def test_a_module_that_does_not_build_is_left_out(monkeypatch, tmp_path, compiler):
    stale = tmp_path / "_quick.so"
    stale.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "QUICK", str(stale))
    monkeypatch.setattr(build.shutil, "which", lambda name: compiler)
    with pytest.warns(RuntimeWarning, match="_quick"):
        build._build_quick()
    assert not stale.exists()


def test_the_module_is_named_for_its_interpreter():
    assert os.path.basename(build.QUICK) == "_quick" + sysconfig.get_config_var("EXT_SUFFIX")


def copied(tmp_path):
    """The package's Python part under another name, in a folder of its own."""
    shutil.copy(amp.__file__, tmp_path / "__init__.py")
    spec = importlib.util.spec_from_file_location("amp_copied", tmp_path / "__init__.py", submodule_search_locations=[str(tmp_path)])
    m = importlib.util.module_from_spec(spec)
    sys.modules["amp_copied"] = m
    spec.loader.exec_module(m)
    m._lib, m._current = object(), lambda: (0, 0)       # as once the library and a GPU are in use
    return m


def test_a_module_that_does_not_load_counts_as_absent(tmp_path):
    (tmp_path / "_quick.so").write_bytes(b"of another interpreter")
    try:
        m = copied(tmp_path)
        with pytest.warns(RuntimeWarning, match="_quick"):
            m._bind()
        assert m._plain is None
    finally:
        sys.modules.pop("amp_copied", None)


def test_a_module_that_was_not_built_is_no_cause_for_a_warning(tmp_path):
    try:
        m = copied(tmp_path)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            m._bind()
        assert m._plain is None
    finally:
        sys.modules.pop("amp_copied", None)
