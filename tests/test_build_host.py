"""What the in-tree build needs and redoes: the library without torch, the
library where the binding fails, and nothing that is current already."""
import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# One small translation unit in place of the library's, in a folder of its own.
SETUP = """
import os, sys
tmp = sys.argv[1]
{before}
from variable_length_batching_gb300 import build as b
src = os.path.join(tmp, "one.cu")
if not os.path.exists(src):
    open(src, "w").write("__global__ void k() {{}}\\n")
b.sources = lambda: [src]
b.BUILD = tmp
b.LIB, b.BINDING = os.path.join(tmp, "libone.so"), os.path.join(tmp, "binding.so")
b.STAMP, b.BINDING_STAMP = os.path.join(tmp, "stamp"), os.path.join(tmp, "binding_stamp")
"""


def _run(tmp, code, before=""):
    r = subprocess.run([sys.executable, "-c", SETUP.format(before=before) + textwrap.dedent(code), str(tmp)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_library_without_torch(tmp_path):
    _run(tmp_path, """
        b.build()
        assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
        assert "torch" not in sys.modules or sys.modules["torch"] is None
    """, before="sys.modules['torch'] = None            # import torch raises ImportError")


def test_library_stands_where_the_binding_fails(tmp_path):
    _run(tmp_path, """
        def fail(*_):
            raise RuntimeError("g++ failed")
        b._compile_binding = fail
        try:
            b.build()
            raise SystemExit("no error")
        except RuntimeError as e:
            assert "g++" in str(e)
        assert os.path.exists(b.LIB)
    """)


def test_each_part_is_redone_by_itself(tmp_path):
    _run(tmp_path, """
        import torch
        done = []
        compile_one = b._compile
        b._compile = lambda *a: done.append("library") or compile_one(*a)
        b._compile_binding = lambda *a: done.append("binding") or open(b.BINDING, "w").close()
        b.build()
        assert sorted(done) == ["binding", "library"]
        b.build()
        assert len(done) == 2
        torch.__version__ = "another"
        b.build()
        assert done[2:] == ["binding"]
        open(src, "a").write("// changed\\n")
        b.build()
        assert done[3:] == ["library"]
        b.build(force=True)
        assert sorted(done[4:]) == ["binding", "library"]
    """)
