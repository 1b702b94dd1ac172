"""When the compiled wrappers are built again: after a change of their sources, and for another interpreter or torch."""
import os

import pytest

from fp8_block_scaled_13_b200 import build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """The built files in a folder of their own, and a compiler that only writes its output file."""
    built = []

    def run(cmd, check):
        built.append(os.path.basename(cmd[cmd.index("-o") + 1]).split(".tmp")[0])
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    for name in ("LIB_PATH", "BINDING_PATH", "BINDING_TARGET_PATH"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))), raising=False)
    monkeypatch.setattr(build.subprocess, "run", run)
    return built, tmp_path


def test_built_once(sandbox):
    built, _ = sandbox
    build.build()
    assert built == ["libpuro_fp8.so", "_binding.so"]
    build.build()
    assert len(built) == 2


def test_another_torch_or_interpreter(sandbox, monkeypatch):
    built, _ = sandbox
    build.build()
    version = build.importlib.metadata.version
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: version(name) + ".1")
    build.build()
    assert built[2:] == ["_binding.so"]
    abi = build.sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: str(abi(name)) + "x")
    build.build()
    assert built[3:] == ["_binding.so"]
    build.build()
    assert len(built) == 4


def test_a_module_of_unknown_origin(sandbox):
    built, folder = sandbox
    build.build()
    os.remove(folder / "_binding.target")
    build.build()
    assert built[2:] == ["_binding.so"]
