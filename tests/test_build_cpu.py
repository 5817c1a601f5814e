"""The library and the tensor front end are built and loaded apart: the library
needs nvcc alone, the operators of the C ABI need no front extension, and the
front extension follows the torch and the Python it is built for (no GPU)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    from lightning_indexer_cross_b200 import build
    build.build()


def _run(code):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)


def test_ops_of_the_library_need_no_front_extension(built):
    """Without _front.so the operators of libindexcache.so are there; those of the front end say what is missing."""
    r = _run("import sys\n"
             "sys.modules['lightning_indexer_cross_b200._front'] = None\n"
             "import torch\n"
             "from lightning_indexer_cross_b200 import ops\n"
             "try:\n    ops.topk(torch.zeros(1, 8), 4)\nexcept ValueError as e:\n    print('older', e)\n"
             "f, _ = ops.rope_frequencies(64, device='cpu')\n"
             "try:\n    ops.rope(torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int64), f)\n"
             "except ImportError as e:\n    print('new', e)\n")
    assert r.returncode == 0, r.stderr
    lines = r.stdout.splitlines()
    assert lines[0].startswith("older") and "CUDA" in lines[0]
    assert lines[1].startswith("new") and "lightning_indexer_cross_b200.build" in lines[1]


def test_a_front_extension_for_another_torch_is_not_called(built):
    r = _run("import sys, types\n"
             "m = types.ModuleType('lightning_indexer_cross_b200._front')\n"
             "m.torch_version = '1.0'\n"
             "m.set_error = m.rope = lambda *a: print('called')\n"
             "sys.modules[m.__name__] = m\n"
             "import torch\n"
             "from lightning_indexer_cross_b200 import ops\n"
             "f, _ = ops.rope_frequencies(64, device='cpu')\n"
             "try:\n    ops.rope(torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int64), f)\n"
             "except ImportError as e:\n    print(e)\n")
    assert r.returncode == 0, r.stderr
    assert "1.0" in r.stdout and "called" not in r.stdout


@pytest.fixture
def fake_build(tmp_path, monkeypatch):
    """build.py with fake compilers that write their outputs; returns (module, commands so far)."""
    from lightning_indexer_cross_b200 import build as b
    for name, path in (("BUILD", "_build"), ("LIB", "libindexcache.so"), ("FRONT", "_front.so"),
                       ("FRONT_FOR", "_build/front.txt")):
        monkeypatch.setattr(b, name, str(tmp_path / path))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "nvcc", lambda: "/fake/bin/nvcc")
    return b, ran


def test_the_library_builds_where_torch_is_missing(fake_build, monkeypatch, capsys):
    b, ran = fake_build
    real = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda n: None if n == "torch" else real(n))
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.FRONT)
    assert all(c[0] == "/fake/bin/nvcc" for c in ran)
    assert "torch" in capsys.readouterr().err
    n = len(ran)
    assert not b.needs_build() and b.build() == b.LIB and len(ran) == n


def test_a_replaced_torch_or_python_rebuilds_the_front_extension_alone(fake_build, monkeypatch):
    b, ran = fake_build
    b.build()
    assert os.path.exists(b.FRONT) and not b.needs_build()
    n = len(ran)
    real = b.importlib.metadata.version
    monkeypatch.setattr(b.importlib.metadata, "version", lambda n: "99.0" if n == "torch" else real(n))
    assert b.needs_build()
    b.build()
    assert len(ran) == n + 1 and ran[-1][0] != "/fake/bin/nvcc" and not b.needs_build()
    os.remove(b.FRONT)
    assert b.needs_build()


def test_a_torch_without_a_package_record_builds(fake_build, monkeypatch):
    b, ran = fake_build

    def version(name):
        raise b.importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(b.importlib.metadata, "version", version)
    assert b.build() == b.LIB and os.path.exists(b.FRONT) and not b.needs_build()
