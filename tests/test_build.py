"""How the library and the compiled calls are built and loaded (no GPU needed)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_non_uniform_b200 import build
    build.build()


def python(code, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, **env},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_importing_the_package_does_not_load_the_library():
    """A process that builds the library imports the package first: had that
    loaded the old libcq.so, its lib() would get that one again, whatever the
    build put in its place."""
    out = python("""
import bit_non_uniform_b200 as cq
from bit_non_uniform_b200 import build
def mapped():
    with open("/proc/self/maps") as f:
        return sorted({l.split("/")[-1].strip() for l in f if "libcq" in l or "_cq_torch" in l})
print(mapped(), cq._direct)
cq.lib()
print(mapped(), cq._direct is not None)
""")
    assert out.splitlines() == ["[] None", "['_cq_torch.so', 'libcq.so'] True"]


@pytest.fixture
def compiles(monkeypatch, tmp_path):
    """build.py with the extension's place in a new folder; what it would run."""
    from bit_non_uniform_b200 import build
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "_cq_torch.so"))
    calls = []

    def check_call(cmd):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    return build, calls


def test_an_extension_of_another_torch_is_built_again(compiles):
    build, calls = compiles
    for text, runs in ((f"x {build.built_for()} y", 0), ("torch 1.0, python 3.12", 1)):
        with open(build.TORCH_LIB, "w") as f:
            f.write(text)
        build.build_torch()
        assert len(calls) == runs
    assert f'-DCQ_BUILT_FOR="{build.built_for()}"' in calls[0]
    with open(build.TORCH_LIB) as f:
        assert f.read() == "new"


def test_an_extension_of_another_torch_is_not_loaded():
    code = """
import sys, types
if {fake}:
    sys.modules["bit_non_uniform_b200._cq_torch"] = types.SimpleNamespace(**{fake})
import bit_non_uniform_b200 as cq
cq.lib()
print(cq._direct is None)
"""
    for fake in (dict(built_for="torch 1.0"), dict(older=1)):
        assert python(code.format(fake=fake)).strip() == "True"
    assert python(code.format(fake={})).strip() == "False"


@pytest.mark.parametrize("error", [FileNotFoundError("no compiler"),
                                   subprocess.CalledProcessError(1, "g++")])
def test_the_library_is_built_without_the_extension(compiles, monkeypatch, capfd, error):
    build, calls = compiles
    with open(build.TORCH_LIB, "w") as f:
        f.write("older")

    def check_call(cmd):
        raise error

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.TORCH_LIB)
    assert "_cq_torch.so was not built" in capfd.readouterr().err
