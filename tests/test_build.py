"""build.py's host logic, with the compilers replaced by ones that only note their
command and write their output file: what is built, in which order, and what is left
when a part cannot be."""
import os

import pytest

from attention_forward_flashattention_gb300 import build as fabuild


class Tools:
    """Stands in for subprocess: writes the file behind -o, or fails."""

    def __init__(self, monkeypatch, out):
        self.commands, self.broken = [], ()
        monkeypatch.setattr(fabuild, "OUT", str(out))
        monkeypatch.setattr(fabuild, "nvcc_path", lambda: "/opt/cuda/bin/nvcc")
        monkeypatch.setattr(fabuild.subprocess, "Popen", self.popen)
        monkeypatch.setattr(fabuild.subprocess, "run", self.run)

    def act(self, cmd):
        self.commands.append(cmd)
        if any(b in " ".join(cmd) for b in self.broken):
            return 1
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return 0

    def popen(self, cmd, stdout=None, stderr=None):
        if "missing " + cmd[0] in self.broken:
            raise FileNotFoundError(cmd[0])
        rc = self.act(cmd)

        class Done:
            returncode = rc

            def wait(self):
                return rc
        return Done()

    def run(self, cmd, check=False):
        assert check
        assert self.act(cmd) == 0

    def took(self):
        n, self.commands = len(self.commands), []
        return n


@pytest.fixture
def tools(monkeypatch, tmp_path):
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1'\n")
    t = Tools(monkeypatch, tmp_path / "out")
    t.torch = torch_dir

    class Spec:
        submodule_search_locations = [str(torch_dir)]
    t.spec = Spec
    monkeypatch.setattr(fabuild.importlib.util, "find_spec", lambda name: t.spec)
    return t


def built():
    return {n for n in os.listdir(fabuild.OUT) if n.endswith(".so")}


LIBS = {fabuild.LIB_NAME, fabuild.SELFTEST_NAME}


def test_everything_once(tools):
    fabuild.build()
    assert built() == LIBS | {fabuild.TORCH_NAME}
    # the module is linked against the library, so behind it
    last = [c for c in tools.commands if "-shared" in c]
    assert [os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in last] == [
        fabuild.LIB_NAME, fabuild.SELFTEST_NAME, fabuild.TORCH_NAME]
    tools.took()
    fabuild.build()
    assert tools.took() == 0


def test_the_libraries_need_no_pytorch(tools):
    tools.spec = None
    assert fabuild.build() == (fabuild.lib_path(), fabuild.selftest_path())
    assert built() == LIBS
    tools.took()
    fabuild.build()
    assert tools.took() == 0


@pytest.mark.parametrize("broken", [("missing g++",), (fabuild.TORCH_UNIT,)])
def test_a_module_that_does_not_compile_leaves_the_libraries(tools, broken):
    tools.broken = broken
    with pytest.raises(RuntimeError, match="fa_cache_torch"):
        fabuild.build()
    assert built() == LIBS
    tools.broken = ()
    tools.took()
    fabuild.build()
    assert built() == LIBS | {fabuild.TORCH_NAME} and tools.took() == 2


def test_another_pytorch_rebuilds_the_module_alone(tools):
    fabuild.build()
    tools.took()
    (tools.torch / "version.py").write_text("__version__ = '2'\n")
    fabuild.build()
    assert tools.took() == 2        # compiled and linked
    fabuild.build()
    assert tools.took() == 0


def test_a_unit_that_does_not_compile_is_named(tools):
    tools.broken = ("fa_bwd_d64.cu",)
    with pytest.raises(RuntimeError, match="fa_bwd_d64.cu"):
        fabuild.build()
    assert built() == set()
