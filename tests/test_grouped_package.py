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


BLOCKING = """
#include <stddef.h>
#include <time.h>
/* Stands for every entry point (the callers of both kinds pass integers and pointers only). */
int blocking(void) {
  struct timespec t = {0, 400 * 1000 * 1000};
  nanosleep(&t, NULL);
  return 0;
}
size_t no_workspace(void) { return 0; }
"""


class FakeTensor:
    """What the marshalling module asks of a CUDA tensor; its memory is never touched."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, *shape, dtype):
        self.shape, self.dtype = shape, dtype

    def stride(self):
        out, step = [], 1
        for n in reversed(self.shape):
            out.insert(0, step)
            step *= n
        return tuple(out)

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x7F0000001000


def test_other_threads_run_while_a_call_blocks(tmp_path):
    # The module handed an entry point that sleeps: a thread that counts goes on meanwhile.
    import ctypes
    import importlib.util
    import shutil
    import threading
    import time
    from tiled_matrix_multiply_gb300 import build
    source, lib = tmp_path / "blocking.c", tmp_path / "blocking.so"
    source.write_text(BLOCKING)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(source)], check=True)
    # A copy: the module's functions are its own, not those of the package's.
    copy = shutil.copy(build.build_call(), tmp_path / "copied.so")
    spec = importlib.util.spec_from_file_location("grouped_call", copy)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    fake = ctypes.CDLL(str(lib))
    entry = ctypes.cast(fake.blocking, ctypes.c_void_p).value
    size = ctypes.cast(fake.no_workspace, ctypes.c_void_p).value
    module.start((FakeTensor, lambda shape, dtype, device: FakeTensor(*shape, dtype=dtype),
                  lambda device: 0, lambda: 0, lambda *a: a, "u8", "i32", "i64", "f32", "f32",
                  "bf16", "f16"), (entry, size) * 4)

    def t(*shape, dtype="f32"):
        return FakeTensor(*shape, dtype=dtype)
    off, i = t(3, dtype="i32"), t(4, 1, dtype="i32")
    calls = [lambda: module.group_rows(i, 2), lambda: module.grouped(t(4, 8), t(2, 8, 8), off, None),
             lambda: module.wgrad(t(4, 8), t(4, 8), off, None),
             lambda: module.lora(t(4, 8), t(8, 8), t(2, 8, 2), t(2, 2, 8), t(2), off, None)]
    for call in calls:
        stop, ticks = threading.Event(), []

        def count():
            while not stop.wait(0.02):
                ticks.append(time.perf_counter())
        thread = threading.Thread(target=count)
        thread.start()
        began = time.perf_counter()
        assert call() is not None
        ended = time.perf_counter()
        stop.set()
        thread.join()
        assert ended - began >= 0.4
        assert sum(began < at < ended for at in ticks) >= 3
