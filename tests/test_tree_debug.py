"""The draft-tree entry points on the debug build (every global access that a
kernel derives from lengths, slots, nodes or page ids is checked): no check may
fire, and every byte and output is the release build's."""
import os
import subprocess
import sys

import numpy as np
import pytest

from test_debug_build import _build_debug

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def _run(tmp_path, debug):
    out = tmp_path / ("debug.npz" if debug else "release.npz")
    subprocess.run([sys.executable, os.path.join(HERE, "tree_debug_cases.py"), str(out)],
                   env=dict(os.environ, TBQ4_DEBUG="1" if debug else "0"), check=True, timeout=600)
    return np.load(out)


def test_debug_build_matches_release_bit_for_bit(tmp_path):
    _build_debug()
    rel, dbg = _run(tmp_path, False), _run(tmp_path, True)
    assert int(rel["debug"]) == 0 and int(dbg["debug"]) == 1
    assert int(rel["status"]) == 0
    assert int(dbg["status"]) == 0, "a bounds check of the debug build fired"
    keys = [k for k in rel.files if k not in ("debug", "lib")]
    assert len(keys) == 2 * 5 + 1
    for k in keys:
        np.testing.assert_array_equal(rel[k], dbg[k], err_msg=k)
