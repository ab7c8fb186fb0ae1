"""A planner without host memory returns a status; no exception leaves the C entry points."""
import os
import subprocess
import sys

import pytest

import paged_kv_decode_host_gb300 as pkd

PROGRAM = """
import ctypes, resource
import numpy as np
import paged_kv_decode_host_gb300 as pkd
lib = pkd.load()
heads, kv_heads, dim, flags = {case}
batch = 1 << 30          # 8 GB of lengths, before the table is read
cfg = pkd.make_config(heads, kv_heads, dim, 16, batch, 16, 16, num_ctas=8, flags=flags)
some = np.zeros(64, np.int32).ctypes.data_as(ctypes.c_void_p)
resource.setrlimit(resource.RLIMIT_AS, (4 << 30, 4 << 30))
print("status", lib.pkd_plan_host(ctypes.byref(cfg), some, some, some, batch, some, 1 << 60, None))
"""


@pytest.mark.parametrize("case", [(32, 8, 128, 0), (128, 1, 512, pkd.FLAG_LATENT)])
def test_host_plan_without_memory(case):
    pkd.load()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(case=case)], cwd=root, capture_output=True,
                       text=True, timeout=120)
    assert r.stdout.strip() == "status -7" and r.returncode == 0, (r.returncode, r.stderr[-500:])
