"""How the Python extension of the decoder-layer operators is put in its place."""
import importlib.util
import os
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """The build script with the extension's place in a folder of the test's own."""
    import __graft_entry__

    __graft_entry__.build()  # the library itself is up to date
    spec = importlib.util.spec_from_file_location("_builder", os.path.join(ROOT, "moe_decode_host_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.place = mod.BINDING
    monkeypatch.setattr(mod, "BINDING", str(tmp_path / os.path.basename(mod.BINDING)))
    return mod


def _compiler(tmp_path, monkeypatch, status):
    """A compiler that writes its output file, notes where, and ends with `status`."""
    c = tmp_path / "cxx"
    c.write_text('#!/bin/sh\nfor last; do :; done\necho part > "$last"\necho "$last" > "%s"\nexit %d\n'
                 % (tmp_path / "wrote", status))
    c.chmod(0o755)
    monkeypatch.setenv("CXX", str(c))


def test_the_name_carries_the_interpreter(builder):
    assert os.path.basename(builder.place) == "_decoder_ops" + sysconfig.get_config_var("EXT_SUFFIX")
    from moe_decode_host_gb300 import decoder_ops

    assert os.path.samefile(decoder_ops._decoder_ops.__file__, builder.place)


def test_a_failed_build_leaves_the_extension_as_it_was(builder, tmp_path, monkeypatch):
    with open(builder.BINDING, "w") as f:
        f.write("whole")
    os.utime(builder.BINDING, (0, 0))  # out of date
    _compiler(tmp_path, monkeypatch, 1)
    with pytest.raises(RuntimeError):
        builder.build()
    assert open(builder.BINDING).read() == "whole"
    assert sorted(os.listdir(tmp_path)) == sorted([os.path.basename(builder.BINDING), "cxx", "wrote"])


def test_the_extension_is_written_elsewhere_and_moved(builder, tmp_path, monkeypatch):
    _compiler(tmp_path, monkeypatch, 0)
    builder.build()
    assert open(builder.BINDING).read() == "part\n"
    wrote = (tmp_path / "wrote").read_text().strip()
    assert wrote != builder.BINDING and not os.path.exists(wrote)
    assert os.path.dirname(wrote) == os.path.dirname(builder.BINDING)  # a rename within one file system
