"""Counts that the paged kernels could step past in 32 bits are refused (no GPU).  The
addresses are made up, so the calls run in a child process that sees no device."""
import json
import os
import subprocess
import sys

from mlx_grouped_affine_gb300 import qmm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 1024
CHILD = """
import json, sys
from mlx_grouped_affine_gb300 import qmm
L, A = qmm.lib(), 1 << 44
at = lambda i: A + (i << 36)
cache = qmm.PagedCache(at(1), at(2), qmm.QMM_BF16, 10, 16, 2, 64, 2048, 1024, 64)
got = []
for what, n in json.load(sys.stdin):
    if what == "plan":
        s = L.qmm_page_plan(at(3), at(4), n, at(5), 9, None, 16, at(6), 1, 5, at(7), at(8), at(9), at(10), at(11), 0)
    else:
        t, b = (n, 3) if what == "tokens" else (3, n)
        s = L.qmm_paged_attention(at(3), 256, t, 4, cache, at(4), 8, at(5), at(6), b, 1, 1.0, 1, 0, at(7), 256, None,
                                  at(8), qmm.QMM_ATTENTION_WORKSPACE_BYTES, 0)
    got.append((s, qmm.qmm_last_error()))
print(json.dumps(got))
"""


def test_counts_within_a_block_of_2_to_the_31():
    calls = [(w, n) for w in ("plan", "tokens", "requests") for n in (MOST + 1, 2 ** 31 - 1)]
    fine = [(w, MOST) for w in ("plan", "tokens", "requests")]
    run = subprocess.run([sys.executable, "-c", CHILD], input=json.dumps(calls + fine), text=True, check=True,
                         capture_output=True, cwd=ROOT, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    got = json.loads(run.stdout)
    for (what, n), (status, message) in zip(calls, got):
        assert status == qmm.QMM_ERR_INVALID_ARG and "2^31 - 1024" in message, (what, n, message)
    for status, message in got[len(calls):]:
        assert status == qmm.QMM_ERR_CUDA, message  # past the checks there is no device to run on
