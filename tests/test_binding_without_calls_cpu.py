"""The binding where the native marshalling of the 4-bit cache's per-token calls is
missing, is another interpreter's or does not load: the library and every other
call work, and those calls say what is missing."""
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

from conftest import ROOT

PKG = "gqa_attention_preallocated_qa_gb300"


@pytest.fixture(scope="module")
def build():
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    return _build


@pytest.fixture
def copy(build, tmp_path):
    """The package without the module, beside the real library."""
    there = tmp_path / PKG
    there.mkdir()
    for name in os.listdir(os.path.join(ROOT, PKG)):
        if name.endswith(".py"):
            shutil.copy(os.path.join(ROOT, PKG, name), there / name)
    os.symlink(build.LIB, there / os.path.basename(build.LIB))
    return there


def run(copy, code):
    out = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=copy.parent, capture_output=True, text=True,
                         timeout=300, env={**os.environ, "PYTHONPATH": str(copy.parent)})
    assert out.returncode == 0, out.stdout + out.stderr
    return out.stdout


USE = """
    from gqa_attention_preallocated_qa_gb300 import binding as qa
    assert qa.qa_abi_version() > 0
    try:
        qa.qa_decode_step(None, 0, 1, 16, 16, 16, 16, 16, 16, stream=0)
    except qa.QaError as e:
        assert e.status == 1
    try:
        qa.qa_q4_cache_set_window(None, 0, 1)   # through ctypes, like all calls that are not made per token
    except qa.QaError as e:
        assert e.status == 1
    said = set()
    for call in (lambda: qa.qa_q4_append(None, 0, [0], [1], 16, 16, stream=0),
                 lambda: qa.qa_q4_read(None, 0, [0], [1], 16, 16, stream=0),
                 lambda: qa.qa_q4_prefill(None, 0, [0], [1], 16, 16, 16, 16, 16, 16, stream=0),
                 lambda: qa.qa_q4_decode_step(None, 0, [0], 16, 16, 16, 16, 16, 16, stream=0),
                 lambda: qa.qa_q4_decode_step_device_positions(None, 0, 1, 16, 16, 16, 16, 16, 16, 16, stream=0)):
        try:
            call()
        except ImportError as e:
            said.add(str(e))
    assert len(said) == 1 and "_q4calls" in said.pop()
"""


def test_the_module_is_missing(copy):
    run(copy, USE)


def test_an_untagged_module_is_not_taken_for_this_interpreters(copy):
    (copy / "_q4calls.so").write_bytes(b"built by another interpreter")
    (copy / "_q4calls.cpython-399-other.so").write_bytes(b"another one")
    run(copy, USE)


def test_a_module_that_does_not_load(copy, build):
    (copy / os.path.basename(build.CALLS)).write_bytes(b"no shared library")
    run(copy, USE)


def test_the_module_is_used_where_it_is(copy, build):
    shutil.copy(build.CALLS, copy / os.path.basename(build.CALLS))
    run(copy, """
        from gqa_attention_preallocated_qa_gb300 import binding as qa
        try:
            qa.qa_q4_append(None, 0, [0], [1], 16, 16, stream=0)
        except qa.QaError as e:
            assert e.status == 1
        else:
            raise SystemExit(1)
    """)


def test_the_module_is_named_for_the_interpreter_and_its_machine(build):
    import sysconfig
    assert os.path.basename(build.CALLS) == "_q4calls" + sysconfig.get_config_var("EXT_SUFFIX")


def test_without_a_compiler_or_headers_the_library_is_up_to_date(build, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "none.so"))
    assert build.stale()                        # it can be built, and is not there
    monkeypatch.setattr(build.sysconfig, "get_path", lambda name: str(tmp_path))
    assert not build.can_build_calls() and not build.stale()
    monkeypatch.undo()
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "none.so"))
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert not build.can_build_calls() and not build.stale()
