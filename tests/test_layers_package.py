"""How routing, log probabilities and linear layers are reached, on the host (CPU only)."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from test_grouped_package import FakeTensor  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = {"route_rows", "RowRoutes", "route_rows_grad", "logprob_rows", "RowLogprobs",
         "logprob_rows_grad", "gemm_bias_act", "gemm_bias_act_grad", "LinearGrads"}


def test_the_package_offers_them():
    import tiled_matrix_multiply_gb300 as tmm
    assert NAMES <= set(dir(tmm))
    for name in NAMES:
        assert getattr(tmm, name).__doc__


def test_calls_go_through_ctypes_where_the_module_cannot_be_built(tmp_path):
    code = ("import sys; sys.path.insert(0, %r)\n"
            "from tiled_matrix_multiply_gb300 import build\n"
            "build.build()\n"
            "build.CALL_PATH += '.absent'\n"
            "build.sysconfig.get_paths = lambda: {'include': '/nowhere'}\n"
            "import torch, tiled_matrix_multiply_gb300 as tmm\n"
            "x = torch.zeros(3, 4)\n"
            "for fn, args in ((tmm.route_rows, (x, 2)), (tmm.route_rows_grad, (x, x, x)),\n"
            "                 (tmm.logprob_rows, (x,)), (tmm.logprob_rows_grad, (x, None, x)),\n"
            "                 (tmm.gemm_bias_act, (x, x.t())), (tmm.gemm_bias_act_grad, (x, x, x))):\n"
            "    try: fn(*args)\n"
            "    except (TypeError, ValueError): pass\n"
            "    else: raise AssertionError(fn)\n" % ROOT)
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=tmp_path,
                         timeout=300)
    assert run.returncode == 0, run.stderr


RECORDING = """
#include <stddef.h>
#include <stdint.h>
static int calls;
int recorded(void) { return ++calls, 0; }
int refused(void) { return -1; }
int count(void) { return calls; }
size_t no_workspace(void) { return 0; }
"""


@pytest.fixture
def module(tmp_path):
    """A copy of the marshalling module, its entry points stand-ins that count their calls."""
    import ctypes
    import importlib.util
    import shutil
    from tiled_matrix_multiply_gb300 import build
    source, lib = tmp_path / "recorded.c", tmp_path / "recorded.so"
    source.write_text(RECORDING)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(source)], check=True)
    copy = shutil.copy(build.build_call(), tmp_path / "copied.so")
    spec = importlib.util.spec_from_file_location("grouped_call", copy)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    fake = ctypes.CDLL(str(lib))

    def address(name):
        return ctypes.cast(getattr(fake, name), ctypes.c_void_p).value
    entry, size = address("recorded"), address("no_workspace")
    FakeTensor.t = lambda self: FakeTensor(*reversed(self.shape), dtype=self.dtype)
    m.start((FakeTensor, lambda shape, dtype, device: FakeTensor(*shape, dtype=dtype),
             lambda device: 0, lambda: 0, lambda *a: a, "u8", "i32", "i64", "f32", "f32",
             "bf16", "f16"), (entry, size) * 4)

    def start(entry):
        m.start_scores((lambda *a: a, lambda *a: a), (entry,) * 4)
        m.start_linear((lambda *a: a,), (entry, size) * 2)
    start(entry)
    m.refuse = lambda: start(address("refused"))
    m.count = fake.count
    return m


def t(*shape, dtype="f32"):
    return FakeTensor(*shape, dtype=dtype)


def usual(m):
    x, v = t(4, 8, dtype="bf16"), t(4)
    tokens, ids = t(4, dtype="i64"), t(4, 2, dtype="i32")
    return {
        "route": lambda: m.route(x, 2, t(8), 0, 1, 1, 1, True, 1.0),
        "route_grad": lambda: m.route_grad(t(4, 2), x, ids, 0, True, 1.0),
        "logprob": lambda: m.logprob(x, tokens, 3, 1.0),
        "logprob_plain": lambda: m.logprob(x, None, 0, 1.0),
        "logprob_grad": lambda: m.logprob_grad(x, tokens, v, v, v, v, ids, t(4, 2), 1.0),
        "linear": lambda: m.linear(x, t(8, 6, dtype="bf16"), t(6), 1, t(4, 6, dtype="bf16"), True),
        "linear_plain": lambda: m.linear(x, t(8, 6, dtype="bf16"), None, 0, None, False),
        "linear_grad": lambda: m.linear_grad(t(4, 6, dtype="bf16"), x, t(8, 6, dtype="bf16"),
                                             t(4, 6, dtype="bf16"), 2, True)}


def test_usual_calls_are_marshalled(module):
    shapes = {"route": [(4, 2), (4, 2)], "route_grad": (4, 8),
              "logprob": [(4,), (4,), (4,), (4, 3), (4, 3)],
              "logprob_plain": [None, (4,), (4,), None, None], "logprob_grad": (4, 8),
              "linear": [(4, 6), (4, 6)], "linear_plain": (4, 6),
              "linear_grad": [(4, 8), (8, 6), (6,)]}
    for i, (name, call) in enumerate(usual(module).items()):
        out = call()
        assert module.count() == i + 1, name
        got = [o and o.shape for o in out] if isinstance(out, tuple) else out.shape
        assert got == shapes[name], name


def test_unusual_calls_are_left_to_python(module):
    x, w = t(4, 8, dtype="bf16"), t(8, 6, dtype="bf16")
    ids = t(4, 2, dtype="i32")
    for call in (lambda: module.route(x, 99, None, 0, 1, 1, 1, True, 1.0),
                 lambda: module.route(x, 2, t(7), 0, 1, 1, 1, True, 1.0),
                 lambda: module.route(x, 2, t(8, dtype="bf16"), 0, 1, 1, 1, True, 1.0),
                 lambda: module.route(x, 2.0, None, 0, 1, 1, 1, True, 1.0),
                 lambda: module.route(x, 2, None, 0, 1, 1, 1, "yes", 1.0),
                 lambda: module.route("x", 2, None, 0, 1, 1, 1, True, 1.0),
                 lambda: module.route(x, 1 << 70, None, 0, 1, 1, 1, True, 1.0),
                 lambda: module.route_grad(t(4, 3), x, ids, 0, True, 1.0),
                 lambda: module.route_grad(t(5, 2), x, ids, 0, True, 1.0),
                 lambda: module.logprob(x, t(3, dtype="i64"), 0, 1.0),
                 lambda: module.logprob(x, t(4, dtype="u8"), 0, 1.0),
                 lambda: module.logprob(x, None, 33, 1.0),
                 lambda: module.logprob(t(4, 8, dtype="f64"), None, 0, 1.0),
                 lambda: module.logprob_grad(x, None, t(4), t(4), None, None, None, None, 1.0),
                 lambda: module.logprob_grad(x, None, t(4), None, None, t(4), None, None, 1.0),
                 lambda: module.logprob_grad(x, None, t(3), None, None, None, None, None, 1.0),
                 lambda: module.logprob_grad(x, None, t(4), None, None, None, None, ids, 1.0),
                 lambda: module.linear(x, t(7, 6, dtype="bf16"), None, 0, None, False),
                 lambda: module.linear(x, t(8, 6), None, 0, None, False),
                 lambda: module.linear(x, w, t(6, dtype="f16"), 0, None, False),
                 lambda: module.linear(x, w, None, 0, t(4, 5, dtype="bf16"), False),
                 lambda: module.linear(x, w, None, 0, None, t(4, 6, dtype="bf16")),
                 lambda: module.linear_grad(t(4, 5, dtype="bf16"), x, w, None, 0, False),
                 lambda: module.linear_grad(t(4, 6, dtype="bf16"), x, w, None, 1, False),
                 lambda: module.linear_grad(t(4, 6, dtype="bf16"), x, w, None, 0, t(6))):
        assert call() is None
    assert module.count() == 0


def test_refused_calls_are_left_to_python(module):
    module.refuse()
    for name, call in usual(module).items():
        assert call() is None, name
