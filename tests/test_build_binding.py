"""The binding module is built on torch's headers: it is rebuilt for another torch, and says so when
it is loaded beside one that it was not built for.  No GPU needed."""
import importlib.metadata
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def made(monkeypatch, tmp_path):
    """build_binding into an empty folder, with a compiler that writes an empty file."""
    from sparse_graph_causal_b200 import build as b
    runs = []

    def run(cmd, check):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "BIND", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(b, "OBJ", str(tmp_path / "objects"))
    monkeypatch.setattr(b.subprocess, "run", run)

    def call():
        before = len(runs)
        b.build_binding()
        return len(runs) - before
    return call


def test_rebuilt_for_another_torch(made, monkeypatch):
    assert made() == 1
    assert made() == 0
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version",
                        lambda name: "9.8.7" if name == "torch" else real(name))
    assert made() == 1
    assert made() == 0
    monkeypatch.setattr(importlib.metadata, "version", real)
    assert made() == 1


@pytest.mark.parametrize("version, ok", [(None, True), ("9.8.7", False)])
def test_loaded_beside_another_torch(version, ok):
    code = "import torch\n"
    if version:
        code += f"torch.__version__ = torch.torch_version.TorchVersion({version!r})\n"
    code += ("import sparse_graph_causal_b200 as sa\n"
             "try:\n    print(sa._paged.decode)\n"
             "except ImportError as e:\n    print('refused:', e)\n"
             "    try:\n        print(sa._paged.decode)\n"
             "    except ImportError as e:\n        print('again:', e)\n")
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    if ok:
        assert "built-in" in p.stdout
    else:
        lines = p.stdout.splitlines()
        assert [x.split(":")[0] for x in lines] == ["refused", "again"]
        assert all(version in x and "sparse_graph_causal_b200.build" in x for x in lines)
