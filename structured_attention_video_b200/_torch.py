"""Loads the torch binding: argument checks and marshalling of the window attention, the
paged attention and the rotary positions (csrc/torch_binding.cpp).  Importing this module
fails with an ImportError when it has not been built for the installed torch."""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch  # noqa: F401  (its libraries come first)

from . import _lib
from . import build as _build

if not os.path.exists(_build.BINDING):
    raise ImportError("the torch binding is not built (%s); run "
                      "`python -m structured_attention_video_b200.build`" % _build.BINDING)

_loader = importlib.machinery.ExtensionFileLoader("monarch_torch", _build.BINDING)
native = importlib.util.module_from_spec(
    importlib.util.spec_from_file_location("monarch_torch", _build.BINDING, loader=_loader))
_loader.exec_module(native)
native.set_status_error(_lib.MonarchError)
