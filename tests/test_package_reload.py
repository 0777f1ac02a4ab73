"""The package in a tree whose operand-check extension is not built yet, as a
build finds it: imported without it, loaded again without it and, once it is
there, with it; and a build that cannot make the extension.  A copy of the
package in a process of its own."""

import os
import shutil
import subprocess
import sys
import textwrap

import pytest

PACKAGE = "fp8_tensor_scaled_amd"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EXTENSION = os.path.join(ROOT, PACKAGE, "_fp8binding.so")


@pytest.fixture
def bare(tmp_path):
    """A folder with the package's sources and no compiled file."""
    shutil.copytree(os.path.join(ROOT, PACKAGE), tmp_path / PACKAGE,
                    ignore=shutil.ignore_patterns("*.so*", "_build", "__pycache__"))
    return tmp_path


def python(folder, program):
    env = dict(os.environ, PYTHONDONTWRITEBYTECODE="1")
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(program)], cwd=folder, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


REFUSAL = """
    import torch

    def refuses(f):
        try:
            f.fp8_act_fwd(torch.zeros(2, 8), 2, 8, f.ACT_SILU, False, torch.zeros(2, 7))
        except ValueError as e:
            assert "out: 14 elements" in str(e), e
        else:
            raise AssertionError("a short buffer went through")
"""


def test_without_the_extension(bare):
    python(bare, REFUSAL + """
    import importlib, os
    import fp8_tensor_scaled_amd as f
    assert os.path.dirname(f.__file__) == os.path.join(os.getcwd(), "fp8_tensor_scaled_amd")
    for again in range(3):
        assert f._take is f._take_slow
        refuses(f)
        importlib.reload(f)
    """)


def test_extension_built_meanwhile(bare):
    if not os.path.exists(EXTENSION):
        pytest.skip("the extension is not built here")
    python(bare, REFUSAL + f"""
    import importlib, shutil
    import fp8_tensor_scaled_amd as f
    assert f._take is f._take_slow
    shutil.copy({EXTENSION!r}, "fp8_tensor_scaled_amd")
    importlib.invalidate_caches()
    for again in range(3):
        importlib.reload(f)
        assert f._take is f._fp8binding.take and f._take is not f._take_slow
        refuses(f)
    """)


@pytest.mark.parametrize("cxx", ["missing", "failing"])
def test_library_built_without_the_extension(bare, cxx):
    """A machine without a host compiler, or whose compiler fails: the library is
    linked, the build says what is missing, an extension of older sources goes
    and the package takes the Python form.  (hipcc is a stub that makes its
    output file.)"""
    for name, text in (("hipcc", "while [ \"$1\" != -o ]; do shift; done; : > \"$2\""),
                       ("failing", "echo no headers here >&2; exit 1")):
        (bare / name).write_text(f"#!/bin/sh\n{text}\n")
        (bare / name).chmod(0o755)
    (bare / PACKAGE / "_fp8binding.so").write_bytes(b"of older sources")
    python(bare, REFUSAL + f"""
    import os, warnings
    os.environ.update(HIPCC=os.path.abspath("hipcc"), CXX=os.path.abspath({cxx!r}))
    from fp8_tensor_scaled_amd import build
    with warnings.catch_warnings(record=True) as seen:
        warnings.simplefilter("always")
        lib = build.build()
    assert os.path.exists(lib) and os.path.exists(build.BENCH_LIB)
    said = [str(w.message) for w in seen if "_fp8binding" in str(w.message)]
    assert len(said) == 1 and {"no headers here" if cxx == "failing" else "missing"!r} in said[0]
    assert not os.path.exists(build.BINDING_LIB)
    """)
    python(bare, REFUSAL + """
    import fp8_tensor_scaled_amd as f
    assert f._take is f._take_slow
    refuses(f)
    """)
