"""The torch binding next to the library: what works without it, and when it is built."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_monarch_attention_needs_no_binding():
    """Without the binding the Monarch entry points import as ever; the others say what is
    missing."""
    r = python("""
import structured_attention_video_b200 as pkg
from structured_attention_video_b200 import build
build.BINDING = "/nonexistent/monarch_torch.so"
pkg.monarch_attention, pkg.workspace_bytes, pkg.kernel_path, pkg.Rotary
from structured_attention_video_b200.attention import monarch_attention_backward
for name in ("window_attention", "paged_attention", "rotary"):
    try:
        getattr(pkg, name)
    except ImportError as e:
        assert "is not built" in str(e), e
    else:
        raise AssertionError(name + " without a binding")
""")
    assert r.returncode == 0, r.stderr


# A process that finds another version of torch installed than the one that runs.
UPGRADED = """
import importlib.metadata
installed = importlib.metadata.version
importlib.metadata.version = lambda name: "99.1+cu999" if name == "torch" else installed(name)
from structured_attention_video_b200 import build
"""


def test_binding_of_another_torch_is_not_loaded():
    """The binding is compiled against one torch's headers: after an upgrade it counts as not
    built, whatever its age, and the Monarch entry points work meanwhile."""
    r = python(UPGRADED + """
import structured_attention_video_b200 as pkg
pkg.monarch_attention
try:
    pkg.window_attention
except ImportError as e:
    assert "is not built" in str(e) and "99.1" in str(e), e
else:
    raise AssertionError("loaded a binding of another torch")
""")
    assert r.returncode == 0, r.stderr


def test_binding_of_another_torch_is_built_anew():
    r = python(UPGRADED + """
targets = []
class Done:
    returncode = 0
build.subprocess.run = lambda cmd, **kw: targets.append(cmd) or Done()
build.os.replace = lambda a, b: targets.append(b)
build._build_binding(False)
assert targets and targets[-1] == build.BINDING, targets
""")
    assert r.returncode == 0, r.stderr


def test_library_builds_where_the_binding_cannot(tmp_path):
    """Without torch, without a C++ compiler or with headers that do not fit: the library is
    there, the reason is said, and no module that is older than its source stays."""
    for broken in ('sys.modules["torch"] = None',
                   'build.subprocess.run = fails',
                   'build.subprocess.run = missing'):
        r = python("""
import os, subprocess, sys
from structured_attention_video_b200 import build
real, out = build.BINDING, %r
build.BINDING = os.path.join(out, "binding.so")
open(build.BINDING, "w").close()
os.utime(build.BINDING, (0, 0))
older = build._stale
build._stale = lambda target, deps: target != build.LIB and older(target, deps)   # it is built
def fails(cmd, **kw):
    return subprocess.CompletedProcess(cmd, 1, "", "headers do not fit")
def missing(cmd, **kw):
    raise FileNotFoundError("g++")
%s
assert build.build() == build.LIB and os.path.exists(build.LIB)
assert not os.path.exists(build.BINDING)
""" % (str(tmp_path), broken))
        assert r.returncode == 0, r.stderr
        assert "was not built" in r.stderr
