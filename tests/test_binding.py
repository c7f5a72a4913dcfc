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
