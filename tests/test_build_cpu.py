"""What build() makes, in which order and when again; compilers are stood in for (CPU)."""
import os
import subprocess
import sysconfig

import pytest
import torch

from combine_router_softmax_top_gb300 import build


class Compilers:
    """Stands in for subprocess.run: every command makes its output, unless it is to fail."""

    def __init__(self):
        self.fails, self.made, self.commands = (), [], []

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        self.commands.append(cmd)
        if any(f in cmd or f == os.path.basename(cmd[0]) for f in self.fails):
            return subprocess.CompletedProcess(cmd, 1, "", "no such compiler or header")
        with open(out, "w") as f:
            f.write("made")
        self.made.append(os.path.basename(out))
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def tools(tmp_path, monkeypatch):
    run = Compilers()
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setenv("CXX", "g++")
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(build, "PY_CALL", str(tmp_path / "_py_call.so"))
    return run


def test_the_library_needs_nvcc_alone(tools):
    """Without g++, torch's or Python's headers there is no _py_call.so, which build() says, but
    the C library is made all the same."""
    tools.fails = ("g++",)
    with pytest.raises(RuntimeError, match="py_call"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.PY_CALL)
    assert not build.up_to_date()


def test_a_missing_torch_does_not_stop_the_library(tools, monkeypatch):
    def absent():
        raise ImportError("no torch")
    monkeypatch.setattr(build, "_torch_dir", absent)
    with pytest.raises(Exception, match="no torch"):
        build.build()
    assert os.path.exists(build.LIB)


def test_a_failing_kernel_leaves_no_library(tools):
    tools.fails = ("nvcc",)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
    assert not os.path.exists(build.LIB) and not os.path.exists(build.PY_CALL)


def test_built_once(tools):
    assert build.build() == build.LIB and build.up_to_date()
    assert {"libmoe.so.tmp", "_py_call.so.tmp"} <= set(tools.made)
    n = len(tools.commands)
    build.build()
    assert len(tools.commands) == n
    build.build(force=True)
    assert len(tools.commands) == 2 * n


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_torch_or_python_makes_the_call_path_again(tools, monkeypatch, what):
    """_py_call.so reads torch's objects by their layout in one version of it."""
    build.build()
    n = len(tools.commands)
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    else:
        get = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var",
                            lambda name: "cpython-999" if name == "SOABI" else get(name))
    assert not build.up_to_date()
    build.build()
    assert build.up_to_date()
    new = tools.commands[n:]
    assert len(new) == 2 and not any(c[0] == "nvcc" for c in new), "the library needs neither"


def test_a_failed_call_path_is_not_taken_for_the_new_one(tools, monkeypatch):
    build.build()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    tools.fails = ("g++",)
    with pytest.raises(RuntimeError, match="py_call"):
        build.build()
    assert not build.up_to_date()


def test_torchs_string_layout_is_passed_on(tools):
    build.build()
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    assert [abi in c for c in tools.commands if build.PY_CALL_SOURCE in c] == [True]


def test_the_call_path_knows_what_it_was_made_for():
    """The real module, built for this torch and this Python; one made for others is not used."""
    import combine_router_softmax_top_gb300 as moe
    build.build()
    from combine_router_softmax_top_gb300 import _py_call
    assert _py_call.built_for == build.built_for()
    made_for = moe._call_spec("moe_permute_fp4", moe._SPEC_PERMUTE4)
    assert made_for[0] is _py_call.call


def test_a_call_path_for_another_torch_is_refused(monkeypatch):
    import combine_router_softmax_top_gb300 as moe
    build.build()
    monkeypatch.setattr(torch, "__version__", "1.0.other")
    with pytest.raises(ImportError, match="1.0.other"):
        moe._call_spec("moe_permute_fp4", moe._SPEC_PERMUTE4)
