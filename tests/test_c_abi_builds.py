"""The sanitizer builds of tests/c_abi compile again when any file that goes into them has changed: each names every header
that its sources include, directly or through another (CPU)."""
import importlib.util
import os
import re

import pytest

from block_table_contiguous_amd import build as B

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi")


def included(path, seen):
    """The headers of this repository that a source includes."""
    with open(path) as f:
        names = re.findall(r'^\s*#\s*include\s+"([^"]+)"', f.read(), re.M)
    for name in names:
        for folder in (os.path.dirname(path), B.INCLUDE, B.CSRC):
            header = os.path.join(folder, name)
            if os.path.exists(header):
                if header not in seen:
                    seen.add(header)
                    included(header, seen)
                break
        else:
            raise AssertionError(f"{path}: no {name}")
    return seen


@pytest.mark.parametrize("name", ["build_attention", "build_fp4"])
def test_a_changed_header_is_compiled(name):
    script = os.path.join(HERE, name + ".py")
    if not os.path.exists(script):
        pytest.skip("the sanitizer build script is not available")
    spec = importlib.util.spec_from_file_location(name, script)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    needed = set()
    for source in mod.SOURCES:
        included(source, needed)
    missing = {os.path.basename(p) for p in needed} - {os.path.basename(p) for p in mod.HEADERS}
    assert needed and not missing, f"{name}.py does not look at {sorted(missing)}"
