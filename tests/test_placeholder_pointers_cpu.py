"""Tests that call the library with addresses that are no memory never run where a kernel could be launched (no GPU).

A child process runs those files with torch reporting a GPU: every test that takes the library has to be skipped there.
"""

import ast
import os
import subprocess
import sys

import pytest

from conftest import PLACEHOLDER_POINTER_FILES

HERE = os.path.dirname(os.path.abspath(__file__))
CHILD = """
import sys
import pytest
import torch
torch.cuda.is_available = lambda: True
sys.exit(pytest.main([*sys.argv[1:], "-v", "-p", "no:cacheprovider", "-p", "no:xdist"]))
"""


def library_tests(path):
    with open(path) as f:
        tree = ast.parse(f.read())
    return {n.name for n in tree.body if isinstance(n, ast.FunctionDef) and n.name.startswith("test_")
            and any(a.arg == "lib" for a in n.args.args)}


@pytest.mark.parametrize("name", PLACEHOLDER_POINTER_FILES)
def test_skipped_where_there_is_a_gpu(name):
    path = os.path.join(HERE, name)
    wanted = library_tests(path)
    assert len(wanted) > 5
    res = subprocess.run([sys.executable, "-c", CHILD, path], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                         timeout=600, cwd=os.path.dirname(HERE))
    assert res.returncode == 0, res.stdout[-3000:]
    seen = set()
    for line in res.stdout.splitlines():
        if "::" in line and any(word in line for word in ("PASSED", "FAILED", "SKIPPED", "ERROR")):
            test = line.split("::", 1)[1].split("[")[0].split(" ")[0]
            if test in wanted:
                seen.add(test)
                assert "SKIPPED" in line, line
    assert seen == wanted
