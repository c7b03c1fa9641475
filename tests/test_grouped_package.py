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


def test_the_library_is_built_without_the_headers_of_python(tmp_path, monkeypatch):
    from tiled_matrix_multiply_gb300 import build
    built = []
    monkeypatch.setattr(build, "_build", lambda path, *_: built.append(path) or path)
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build(force=True) == build.LIB_PATH
    assert built == [build.LIB_PATH]


def test_calls_go_through_ctypes_where_the_module_cannot_be_built(tmp_path):
    code = ("import sys; sys.path.insert(0, %r)\n"
            "from tiled_matrix_multiply_gb300 import build\n"
            "build.build()\n"
            "build.CALL_PATH += '.absent'\n"
            "build.sysconfig.get_paths = lambda: {'include': '/nowhere'}\n"
            "import torch, tiled_matrix_multiply_gb300 as tmm\n"
            "i = torch.zeros(3, dtype=torch.int32)\n"
            "for fn, args in ((tmm.group_rows, (i, 2)), (tmm.gemm_grouped, (i, i, i)),\n"
            "                 (tmm.gemm_grouped_wgrad, (i, i, i)), (tmm.gemm_lora, (i,) * 6)):\n"
            "    try: fn(*args)\n"
            "    except (TypeError, ValueError): pass\n"
            "    else: raise AssertionError(fn)\n" % ROOT)
    run = python(code, tmp_path)
    assert run.returncode == 0, run.stderr


def test_the_module_is_named_for_its_interpreter():
    import importlib.machinery
    from tiled_matrix_multiply_gb300 import build
    name = os.path.basename(build.CALL_PATH)
    suffix = name[len("grouped_call"):]
    assert name.startswith("grouped_call.") and suffix in importlib.machinery.EXTENSION_SUFFIXES
    assert sys.implementation.cache_tag.replace("-", "") in suffix.replace("-", "")
