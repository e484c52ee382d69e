"""Host-only checks of the speculative-decoding operators at the edges of what their
documentation allows."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

from long_context_fp8_b200 import build as dsa_build

OK, INVALID, UNSUP, WS = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x1000)           # never dereferenced: every call is refused
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_fp8_b200", "csrc")


def _code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_tree_attention_has_no_unbounded_wait_in_its_roles():
    """After a wait that ran out, warps leave their loops one by one, so nothing inside them may wait for a number
    of threads: a named barrier there could wait for warps that have left, for ever.  (Named barriers
    would be the only such wait besides __syncthreads, which stands before and behind the loops.)"""
    code = _code("tree_attn.cu")
    assert not re.search(r"\bbar(rier)?(\.cta)?\.(sync|red|arrive)\b", code)
    body = code[code.index("void tree_attn_body("):code.index("void __launch_bounds__(TA_THREADS")]
    roles = body[body.index("if (warp < 4 || warp >= 12)"):body.rindex("if (ctl->abort)")]
    assert roles.count("__syncthreads") == 1 and roles.rindex("__syncthreads") > roles.rindex("mbar_arrive(&oempty")
    assert "mbar_wait(" not in roles and "mbar_try_wait(" not in roles


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    from long_context_fp8_b200 import dsa
    return dsa.load()


def test_tree_attention_refuses_contexts_whose_last_block_passes_32_bits(lib):
    """Positions are counted in 32 bits up to the end of the last block of 128, which may lie past 2^31 where a
    block table allows it (its pages may repeat)."""
    def call(pages, ps, max_context, ws):
        return lib.dsa_tree_attn(FAKE, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, 20, pages, ps, 2, 10, 8, max_context,
                                 16, 1, 128, 0.1, FAKE, None, FAKE, ws, None)

    last = 2 ** 31 - 128
    pages = (2 ** 31 - 16) // 16
    for max_context in (2 ** 31 - 16, last + 1, 2 ** 40):
        assert call(pages, 16, max_context, 0) == UNSUP, max_context
    # one block less is refused for its workspace alone
    assert call(pages, 16, last, 0) == WS
    assert call(last // 16, 16, 2 ** 40, 0) == WS


# ------------------------------------------------------------------ the build

def test_library_is_built_first_and_without_torch(monkeypatch, capsys):
    """The C library needs nvcc alone: it is built whether or not the Python binding can be."""
    done = []
    monkeypatch.setattr(dsa_build, "up_to_date", lambda: False)
    monkeypatch.setattr(dsa_build, "binding_up_to_date", lambda: False)
    monkeypatch.setattr(dsa_build, "build_library", lambda *a: done.append("library"))

    def binding(*a):
        done.append("binding")
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(dsa_build, "build_binding", binding)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):        # loud, with the library in place
        dsa_build.build()
    assert done == ["library", "binding"]
    done.clear()
    monkeypatch.setattr(dsa_build.importlib.util, "find_spec", lambda name: None)
    assert dsa_build.build() == dsa_build.LIB
    assert done == ["library"] and "not built" in capsys.readouterr().err


def test_build_runs_without_torch(tmp_path):
    """The build script as a C user runs it, in an interpreter that has no torch."""
    code = """
import sys
sys.path.insert(0, %r)
from long_context_fp8_b200 import build
build.BIND = %r                          # a binding that is not there yet
print(build.build())
""" % (dsa_build.ROOT, str(tmp_path / "_bind.so"))
    # -S: no site-packages, and so no torch
    r = subprocess.run([sys.executable, "-S", "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == dsa_build.LIB and not (tmp_path / "_bind.so").exists()


def test_binding_is_compiled_again_for_another_torch_or_interpreter(lib, monkeypatch):
    """The binding's file says nothing about the torch and the interpreter it was compiled against."""
    import sysconfig

    import torch
    assert dsa_build.binding_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0")
        assert not dsa_build.binding_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch.version, "git_version", "another commit")
        assert not dsa_build.binding_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-39-x86_64-linux-gnu")
        assert not dsa_build.binding_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(dsa_build, "nvcc", lambda: "/opt/another-cuda/bin/nvcc")
        assert not dsa_build.binding_up_to_date()
    assert dsa_build.binding_up_to_date()
