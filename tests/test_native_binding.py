"""The native part of the binding is a short cut: without it, or with one that
does not load here, every call works through Python, and a build puts it back.
On a copy of the package, with a compiler that hands out the built files."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "quantized_fp8_attention_b200"

PROBE = """
import warnings, torch
import quantized_fp8_attention_b200 as f
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    assert f.version() >> 16 == 1
native = f._native is not f._CheckedWay
assert native == (not [x for x in w if "_binding.so" in str(x.message)])
for call in (lambda: f.mx_quantize(torch.zeros(4, 64), "mxfp8"), lambda: f.rotary(torch.zeros(1, 1, 1, 128), None, None)):
    try:
        call()
    except (ValueError, TypeError) as e:
        assert "CUDA" in str(e) or "Rotary" in str(e)
    else:
        raise AssertionError
print("native" if native else "checked")
"""


@pytest.fixture(scope="module")
def built():
    from quantized_fp8_attention_b200 import build
    build.build()
    return build


@pytest.fixture
def copy(built, tmp_path):
    shutil.copytree(os.path.join(ROOT, NAME), tmp_path / NAME, ignore=shutil.ignore_patterns("__pycache__", "*.tmp*"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    for tool, source in (("cxx", built.BINDING), ("nvcc", built.LIB)):
        script = tmp_path / "bin" / tool
        script.parent.mkdir(exist_ok=True)
        script.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\ncp "%s" "$2"\n' % source)
        script.chmod(0o755)
    return tmp_path


def run(copy, *args, cxx="cxx"):
    env = dict(os.environ, PYTHONPATH=str(copy), CXX=str(copy / "bin" / cxx),
               PATH=f"{copy / 'bin'}{os.pathsep}{os.environ['PATH']}")
    got = subprocess.run([sys.executable, *args], cwd=copy, env=env, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]
    return got.stdout.strip().splitlines()[-1]


def spoil(path, how):
    data = path.read_bytes()
    if how == "absent":
        path.unlink()
    elif how == "no library":
        path.write_bytes(b"not a library\n")
    elif how == "cut short":
        path.write_bytes(data[: len(data) // 2])
    else:
        at = data.rfind(b"\n")
        line = data[at + 1:].split(b" ")
        line[1 if how == "another torch" else 2] += b"x"
        path.write_bytes(data[: at + 1] + b" ".join(line))


@pytest.mark.parametrize("how", ["absent", "no library", "cut short", "another torch", "another Python"])
def test_calls_work_without_it_and_a_build_restores_it(copy, how):
    spoil(copy / NAME / "_binding.so", how)
    assert run(copy, "-c", PROBE + f"from {NAME} import build; build.build()") == "checked"
    assert run(copy, "-c", PROBE) == "native"


def test_a_build_leaves_what_fits(copy):
    before = (copy / NAME / "_binding.so").stat().st_mtime_ns
    run(copy, "-m", NAME + ".build")
    assert (copy / NAME / "_binding.so").stat().st_mtime_ns == before
    assert run(copy, "-c", PROBE) == "native"


def test_the_library_is_built_where_the_binding_cannot_be(copy):
    (copy / NAME / "_binding.so").unlink()
    (copy / NAME / "libfqa.so").unlink()
    run(copy, "-m", NAME + ".build", cxx="no such compiler")
    assert (copy / NAME / "libfqa.so").exists() and not (copy / NAME / "_binding.so").exists()
    assert run(copy, "-c", PROBE) == "checked"
    (copy / "bin" / "bad").write_text("#!/bin/sh\nexit 1\n")
    (copy / "bin" / "bad").chmod(0o755)
    run(copy, "-m", NAME + ".build", cxx="bad")
    assert run(copy, "-c", PROBE) == "checked"


def test_the_stand_in_answers_none_to_every_call():
    import quantized_fp8_attention_b200 as f
    from quantized_fp8_attention_b200 import _binding
    for name in ("quantize", "dequantize", "rms_norm", "matmul", "rotate"):
        assert callable(getattr(_binding, name)) and getattr(f._CheckedWay, name)(1, 2, 3, 4) is None
