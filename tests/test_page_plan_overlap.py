"""qmm_page_plan refuses outputs over inputs or over other outputs (no GPU).  The
addresses are made up, so the calls run in a child process that sees no device."""
import json
import os
import subprocess
import sys

import pytest

from mlx_grouped_affine_gb300 import qmm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ["past_lens", "new_lens", "free_pages", "next_free", "block_table", "starts", "seq_lens", "positions",
         "slots", "next_free_out"]
INPUTS = NAMES[:4]
REQUESTS, STRIDE, TOKENS, FREE = 40, 8, 600, 50
COUNT = dict(past_lens=REQUESTS, new_lens=REQUESTS, free_pages=FREE, next_free=1, block_table=REQUESTS * STRIDE,
             starts=REQUESTS + 1, seq_lens=REQUESTS, positions=TOKENS, slots=TOKENS, next_free_out=1)
CHILD = """
import json, sys
from mlx_grouped_affine_gb300 import qmm
got = []
for a, stride in json.load(sys.stdin):
    status = qmm.lib().qmm_page_plan(a["past_lens"], a["new_lens"], %d, a["free_pages"], %d, a["next_free"], 16,
                                     a["block_table"], stride, %d, a["starts"], a["seq_lens"], a["positions"],
                                     a["slots"], a["next_free_out"], 0)
    got.append((status, qmm.qmm_last_error()))
print(json.dumps(got))
""" % (REQUESTS, FREE, TOKENS)


def apart():
    return {n: (1 << 20) + (1 << 16) * i for i, n in enumerate(NAMES)}


def end(n):
    """The last 16-byte boundary inside array n."""
    return (4 * COUNT[n] - 1) // 16 * 16


@pytest.fixture(scope="module")
def calls():
    """(first array, second array, addresses) of every overlap, and of none."""
    got = []
    for i, a in enumerate(NAMES):
        for b in NAMES[i + 1:]:
            if a in INPUTS and b in INPUTS:
                continue
            same = apart()
            same[b] = same[a]
            tail, head = apart(), apart()
            tail[b] = tail[a] + end(a)
            head[a] = head[b] + end(b)
            got += [(a, b, c, STRIDE) for c in (same, tail, head) if (a, b) != ("past_lens", "seq_lens") or c is not same]
    # A table wider than what 64 bits count reaches everything behind it.
    wide = apart()
    got.append(("block_table", "starts", wide, 1 << 62))
    fine = len(got)
    ones = apart()
    ones["seq_lens"] = ones["past_lens"]
    close, at = {}, 1 << 20
    for n in NAMES:
        close[n] = at
        at += (4 * COUNT[n] + 15) // 16 * 16
    shared = apart()
    shared["new_lens"] = shared["past_lens"]
    got += [("", "", c, STRIDE) for c in (apart(), ones, close, shared)]
    run = subprocess.run([sys.executable, "-c", CHILD], input=json.dumps([(c, s) for _, _, c, s in got]), text=True,
                         capture_output=True, cwd=ROOT, check=True, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    answers = json.loads(run.stdout)
    return list(zip(got, answers))[:fine], answers[fine:]


def test_overlaps_are_refused(calls):
    refused, _ = calls
    assert len(refused) > 100
    for (a, b, _, _), (status, message) in refused:
        assert status == qmm.QMM_ERR_INVALID_ARG and message.startswith("qmm_page_plan:"), (a, b, message)
        if (a, b) != ("next_free", "next_free_out"):  # one address: its own message
            assert a in message and b in message, (a, b, message)


def test_arrays_apart_lengths_in_place_and_shared_inputs_are_taken(calls):
    """Past the checks there is no device to run on."""
    for status, message in calls[1]:
        assert status == qmm.QMM_ERR_CUDA, message
