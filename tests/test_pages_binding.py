"""The compiled binding of the shared-prompt calls, without a GPU: the library is built and its calls are
made without the binding too."""
import ctypes
import importlib.metadata
import importlib.util
import os
import sys

import pytest
import torch

import kv_cache_eviction_02_gb300 as package
from kv_cache_eviction_02_gb300 import _build


@pytest.fixture(scope="module")
def api():
    from kv_cache_eviction_02_gb300 import api as a
    _build.build()
    a.lib()
    return a


@pytest.fixture
def small(monkeypatch, tmp_path):
    """build() of a library of one function in an empty folder, with a binding that is a copied file."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(_build, "sources", lambda: [str(src)])
    made = []

    def command(out):
        made.append(out)
        return ["cp", str(src), out]

    monkeypatch.setattr(_build, "binding_command", command)
    return made


def test_a_build_leaves_library_and_binding(small):
    assert ctypes.CDLL(_build.build()).one() == 1
    assert os.path.exists(_build.BINDING) and len(small) == 1
    _build.build()
    assert len(small) == 1  # as it was


@pytest.mark.parametrize("missing", ["compiler", "torch", "metadata"])
def test_the_library_is_built_without_the_binding(small, monkeypatch, capfd, missing):
    """No C++ compiler that takes torch's headers, no torch, a torch without package metadata: the library
    is there, an old binding is not."""
    with open(_build.BINDING, "w") as f:
        f.write("of other sources")
    os.utime(_build.BINDING, (0, 0))
    real, version = importlib.util.find_spec, importlib.metadata.version
    if missing == "compiler":
        monkeypatch.setattr(_build, "binding_command", lambda out: ["false"])
    elif missing == "torch":
        monkeypatch.setattr(_build, "binding_command", COMMAND)
        monkeypatch.setattr(importlib.util, "find_spec",
                            lambda name, *a: None if name == "torch" else real(name, *a))
    else:
        def fails(name):
            if name == "torch":
                raise importlib.metadata.PackageNotFoundError(name)
            return version(name)
        monkeypatch.setattr(importlib.metadata, "version", fails)
    assert ctypes.CDLL(_build.build()).one() == 1
    assert not os.path.exists(_build.BINDING)
    assert "_binding is not built" in capfd.readouterr().err


COMMAND = _build.binding_command


@pytest.mark.parametrize("stamp", ["none", "another"])
def test_a_binding_of_unknown_or_other_versions_is_made_anew(small, stamp):
    """A binding that came without its stamp, or was written when the build was cut off before the stamp,
    may be of any Python and torch."""
    _build.build()
    path = os.path.join(_build.BUILD, "binding.txt")
    if stamp == "none":
        os.remove(path)
    else:
        with open(path, "w") as f:
            f.write("python (3, 0) torch 0")
    _build.build()
    assert len(small) == 2
    _build.build()
    assert len(small) == 2


def test_a_build_cut_off_behind_the_binding_leaves_no_stamp(small, monkeypatch):
    """The stamp of the binding before would vouch for the new one."""
    _build.build()
    path = os.path.join(_build.BUILD, "binding.txt")
    os.utime(_build.BINDING, (0, 0))

    def cut(*a):
        raise OSError("cut off")

    monkeypatch.setattr(_build.os, "replace", cut)
    _build.build()
    assert not os.path.exists(path)


@pytest.fixture
def unbound(api, monkeypatch):
    """The package without its binding."""
    monkeypatch.setattr(api, "_native", None)
    monkeypatch.setitem(sys.modules, package.__name__ + "._binding", None)
    monkeypatch.delattr(package, "_binding", raising=False)
    return api


def test_calls_without_the_binding_reach_the_library_and_its_checks(unbound):
    api = unbound
    pb = api.PgProblem(2, 3, 8, 2, 64, 100, 16, 40, 5, 20, 7, api.KVE_BF16)
    bad = api.PgProblem(2, 3, 9, 2, 64, 100, 16, 40, 5, 20, 7, api.KVE_BF16)
    with pytest.warns(RuntimeWarning, match="_binding"):
        with pytest.raises(api.KveError, match="n_q_heads"):
            api.pg_plan(bad, *[256] * 11)
    with pytest.raises(api.KveError, match="n_q_heads"):
        api.pg_append(bad, *[256] * 5)
    with pytest.raises(api.KveError, match="null"):
        api.pg_attention(pb, None, *[256] * 2, None, *[256] * 6, 256, None, None)
    with pytest.raises(ValueError, match="elements"):
        api.pg_append(pb, torch.zeros(19, 2, 64, dtype=torch.bfloat16), 256, 256, 256, 256)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_without_the_binding_give_what_those_with_it_give(api, request, dtype):
    from test_gpu_pages import DEV, Case

    def step():
        pb = api.PgProblem(1, 3, 8, 2, 64, 50, 4, 20, 4, 5, 1, c.pb.dtype)
        cache = api.PgCache(pb, 1, DEV)
        cache.plan(torch.ones(3, dtype=torch.int32, device=DEV))
        cache.append(0, rows[:, :2], rows[:, 2:])
        return cache.slot_map, cache.K_pages, cache.V_pages

    c = Case(dtype, 2, 3, 8, 2, 64, 120, 8, 40, 2, seed=50, ragged=True, stride=True)
    rows = torch.randn(5, 4, 64, device=DEV).to(c.q.dtype)
    want, stepped = c.run(), step()
    request.getfixturevalue("unbound")
    with pytest.warns(RuntimeWarning, match="_binding"):
        got = c.run()
    assert api._native is api._NoBinding
    for a, b in zip((*want, *stepped), (*got, *step())):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="dtype"):
        api.pg_attention(c.pb, c.q.double(), c.Kp, c.Vp, c.plen, *c.args(), want[0], None, c.ws)
