"""The C marshalling of the selector's calls is built for one interpreter and can be missing: the library and the
calls' Python form stand without it."""
import os
import sysconfig
import warnings

import pytest
import torch


@pytest.fixture
def b():
    from mla_latent_cache_attention_gb300 import build
    build.build()
    return build


@pytest.fixture
def m(b, monkeypatch):
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    monkeypatch.setattr(mod, "_marshal", None)      # put back after the test
    return mod


def test_the_file_is_named_for_the_interpreter(b):
    assert b.MARSHAL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.exists(b.MARSHAL)


def test_it_is_built_alone_where_the_library_is_there(b, monkeypatch, tmp_path):
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / os.path.basename(b.MARSHAL)))
    at = os.path.getmtime(b.LIB)
    assert not b.up_to_date()
    assert b.build() == b.LIB
    assert os.path.exists(b.MARSHAL) and os.path.getmtime(b.LIB) == at and b.up_to_date()


@pytest.mark.parametrize("headers", [False, True])
def test_the_library_stands_without_it(b, monkeypatch, tmp_path, headers):
    """No Python headers, or some that do not compile: a warning, and an old file does not stay."""
    if headers:
        (tmp_path / "Python.h").write_text("#error not these\n")
    old = tmp_path / "mla_marshal.so"
    old.write_text("built for another library")
    os.utime(old, (0, 0))
    monkeypatch.setattr(b, "MARSHAL", str(old))
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: paths)
    with pytest.warns(UserWarning, match="Python form"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not old.exists() and not [f for f in os.listdir(tmp_path) if "tmp" in f]


@pytest.mark.parametrize("there", [False, True])
def test_calls_take_the_python_form_without_it(m, b, monkeypatch, tmp_path, there):
    f = tmp_path / "mla_marshal.so"
    if there:
        f.write_text("not a shared object")
    monkeypatch.setattr(b, "MARSHAL", str(f))
    calls = []
    monkeypatch.setattr(m, "_cuda_device", lambda t: t.device)
    monkeypatch.setattr(m, "_call", lambda fn, dev, *args: calls.append(fn.__name__))
    x, lens = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.warns(UserWarning, match="Python form"):
        blocks, _ = m.index_select(x, lens, 3)
    assert blocks.shape == (2, 3) and calls == ["mla_index_select"]
    with warnings.catch_warnings():
        warnings.simplefilter("error")          # once is enough
        m.index_select(x, lens, 3)
    assert len(calls) == 2
