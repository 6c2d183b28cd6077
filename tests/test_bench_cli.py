"""bench.py's command line on the CPU: more than one GPU is refused with a
message (the code runs on one GPU), before any device work."""

import json
import os
import re
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_more_than_one_gpu_is_refused():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--gpus", "2"],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 2
    msg = json.loads(r.stdout.strip().splitlines()[-1])
    assert msg["n_gpus_requested"] == 2 and "one GPU" in msg["error"]


def test_the_head_source_hash_covers_what_the_head_includes():
    """Sources left out of the hash that a measurement is filed under are
    included by each other alone."""
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    import bench
    csrc = os.path.join(ROOT, "lm_output_head_amd", "csrc")
    for name in os.listdir(csrc):
        if name in bench.SERVE_SOURCES:
            continue
        with open(os.path.join(csrc, name)) as f:
            included = re.findall(r'#include "([^"]+)"', f.read())
        assert not set(included) & set(bench.SERVE_SOURCES), name
