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
