"""How the grouped operators are reached and built, on the host (CPU only)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code, folder):
    """Run with `folder` as the working folder, first in sys.path."""
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=folder,
                          timeout=300)


def test_star_import_loads_neither_torch_nor_a_library(tmp_path):
    # A torch that cannot be imported, and a package directory without built files.
    (tmp_path / "torch.py").write_text("raise ImportError('not here')\n")
    package = tmp_path / "tiled_matrix_multiply_gb300"
    package.mkdir()
    source = os.path.join(ROOT, "tiled_matrix_multiply_gb300")
    for name in os.listdir(source):
        if name.endswith(".py"):
            (package / name).write_text(open(os.path.join(source, name)).read())
    run = python("from tiled_matrix_multiply_gb300 import *\n"
                 "import tiled_matrix_multiply_gb300 as tmm\n"
                 "assert callable(gemm_f32) and issubclass(TmmError, Exception)\n"
                 "assert {'gemm_grouped', 'group_rows', 'gemm_lora'} <= set(dir(tmm))\n"
                 "assert tmm.__file__.startswith(%r)" % str(tmp_path), tmp_path)
    assert run.returncode == 0, run.stderr
