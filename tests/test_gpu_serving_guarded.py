"""The serving operators' later GPU tests again under the guarded build, which
refuses and reports every access out of range."""
import os
import re
import subprocess
import sys

import pytest

from conftest import ROOT
from recurrence_augmented_dilated_chunked_b200 import build as B_

pytestmark = pytest.mark.gpu


def test_later_serving_tests_under_the_guarded_build():
    env = dict(os.environ, RATP_LIBRARY=B_.build_library(guarded=True))
    env["PYTHONPATH"] = ROOT + os.pathsep + env.get("PYTHONPATH", "")
    files = ["tests/test_gpu_%s.py" % n for n in ("cache_q4_long", "cache_q4_edges", "cache_handoff", "padded_batch",
                                                  "cache_lengths", "norm_rope_f32", "linear_attn_infinite",
                                                  "linear_attn_state")]
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider"] + files,
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert res.returncode == 0, "\n".join((res.stdout + res.stderr).splitlines()[-30:])
    m = re.search(r"(\d+) passed", res.stdout)
    assert m and int(m.group(1)) >= 50, res.stdout[-500:]
