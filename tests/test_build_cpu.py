"""An edit of any file that a unit includes makes the unit's object stale."""
import os
import re

import pytest

from block_scaled_fp8_w8a8_gb300 import build


def included(path, seen):
    """The files that `path` includes by a quoted name, and those that they include."""
    for name in re.findall(r'^\s*#\s*include\s+"([^"]+)"', open(path).read(), re.M):
        dep = os.path.normpath(os.path.join(os.path.dirname(path), name))
        if dep not in seen:
            seen.add(dep)
            included(dep, seen)
    return seen


@pytest.mark.parametrize("unit", build.UNITS)
def test_an_edited_include_makes_its_units_stale(unit, monkeypatch, tmp_path):
    src, obj = os.path.join(build.SRC, unit), str(tmp_path / "unit.o")
    open(obj, "w").close()
    deps = included(src, set())
    assert deps
    edited = None
    monkeypatch.setattr(build.os.path, "getmtime", lambda p: 2.0 if os.path.normpath(p) == edited else 1.0)
    assert not build._stale(obj, src)
    for edited in sorted(deps) + [src]:
        assert build._stale(obj, src), edited
