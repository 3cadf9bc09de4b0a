"""Tensors inside torch's function transforms (vmap, grad, jvp, functionalize)
have the plain tensor type and no memory.  The compiled way into the norm and decoding calls
must leave them to the Python functions, which raise.

On the CPU: a copy of csrc/s2_torch.cpp with its device conditions taken out
and C calls that do nothing, in a process of its own (a wrong binding ends
it).  On the GPU: the public calls."""
import os
import re
import subprocess
import sys

import pytest
import torch

import sparse_attention_attn_b200 as s2
from sparse_attention_attn_b200 import api, build
from tests.test_binding import NAMES, _args, _public, _Without

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# operand of each call that the transform takes (the plan has whole numbers alone: vmap only)
CASES = [(n, i, how) for n, ops in (("qknorm_fwd", (0, 3)), ("qknorm_bwd", (0, 5)), ("cache_append", (0, 6)),
                                    ("cache_attention", (0, 2))) for i in ops for how in ("vmap", "grad", "jvp")]
CASES += [("cache_attention", 6, "functionalize"), ("cache_append", 8, "functionalize"), ("cache_append", 9, "functionalize"),
          ("cache_plan", 6, "functionalize")]  # (the C calls refuse the address 0 of the other operands)
CASES += [("cache_plan", 0, "vmap"), ("cache_plan", 2, "vmap"), ("cache_attention", 4, "vmap")]


def _transformed(call, x, how):
    if how == "vmap":
        return torch.vmap(call)(torch.stack([x, x]))
    if how == "functionalize":  # its tensors have the address 0
        return torch.func.functionalize(call)(x)
    if how == "grad":
        return torch.func.grad(call)(x)
    return torch.func.jvp(call, (x,), (torch.ones_like(x),))


CHILD = r'''
import ctypes, sys, torch
sys.path[:0] = [sys.argv[1], sys.argv[2]]
import _relaxed
from tests.test_binding import NAMES, _args
from tests.test_binding_transforms import CASES, _transformed
lib = ctypes.CDLL(sys.argv[1] + "/fake.so")
at = lambda n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
_relaxed.bind(*(at(n) for n in ("ok", "ok", "bytes", "ok", "ok", "ok", "bytes")))
for n in NAMES:
    assert getattr(_relaxed, n)(*_args("cpu")[n]) is not None, n   # a usual call is taken
for n, i, how in CASES:
    a, fn, seen = _args("cpu")[n], getattr(_relaxed, n), []
    def call(x):
        seen.append(fn(*a[:i], x, *a[i + 1:]))
        return x.float().sum()
    _transformed(call, a[i], how)
    assert seen and seen[0] is None, (n, i, how)
    print(n, i, how, flush=True)
print("done")
'''


def test_transformed_tensors_are_left_to_python(tmp_path):
    with open(build.BINDING_SOURCE) as fh:
        src = fh.read()
    for old, new in ((r"!t->is_cuda\(\) \|\| ", ""), (r" \|\| t->get_device\(\) != c10::cuda::current_device\(\)", ""),
                     (r"at::detail::empty_cuda\(shape, type, dev, std::nullopt\)", "at::empty(shape, at::TensorOptions(type))"),
                     (r"return c10::cuda::getCurrentCUDAStream[^;]*;", "return t.defined() ? nullptr : nullptr;"),
                     (r"_s2torch\b", "_relaxed")):
        src, n = re.subn(old, new, src)
        assert n > 0, old
    src = src.replace("PyInit__s2torch", "PyInit__relaxed")
    (tmp_path / "relaxed.cpp").write_text(src)
    (tmp_path / "fake.c").write_text("int ok(void) { return 0; }\nunsigned long bytes(void) { return 64; }\n")
    cmd = build.binding_command(str(tmp_path / "relaxed.cpp"), str(tmp_path / "_relaxed.so"), "-O0")
    if cmd is None:
        pytest.skip("no compiler or no torch headers")
    subprocess.run(cmd, check=True)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "fake.so"), str(tmp_path / "fake.c")], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, str(tmp_path), ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), (r.returncode, r.stdout[-300:], r.stderr[-2000:])


def test_an_operand_without_memory_is_not_an_absent_one():
    x = torch.zeros(3)
    assert api._optional("mask", None) is None and api._optional("mask", x) == x.data_ptr()
    with pytest.raises(ValueError, match="mask has no memory"):
        torch.func.functionalize(lambda t: api._optional("mask", t))(x)


@pytest.mark.gpu
@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_public_calls_raise_under_transforms(monkeypatch, name, compiled):
    if compiled:
        pytest.importorskip("sparse_attention_attn_b200._s2torch")
    else:
        monkeypatch.setattr(api, "_fast", _Without())
    for n, i, how in CASES:
        if n != name:
            continue
        a = _args("cuda")[n]
        with pytest.raises((RuntimeError, ValueError), match="storage|data pointer|INVALID_ARG|no memory"):
            _transformed(lambda x: _public(n, [*a[:i], x, *a[i + 1:]])[0].float().sum(), a[i], how)
    want = _public(name, _args("cuda")[name])  # and the next usual call is as ever
    torch.cuda.synchronize()
    assert s2.device_status() == 0 and all(x is None or torch.isfinite(x.float()).all() for x in want)
