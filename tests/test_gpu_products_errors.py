"""Every set of product kernels has an error word of its own: each is reported, once, and cleared."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_word_is_reported_and_cleared():
    """The bounds-checked build sets the words by hand; no wait runs out."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g.build()
    code = ("import torch, asynchronous_expert_execution_gb300 as moe\n"
            "from asynchronous_expert_execution_gb300 import _native as N\n"
            "x = torch.ones((8, 64), dtype=torch.bfloat16, device='cuda')\n"
            "moe.linear(x, x); moe.linear_backward(x[:, :8].contiguous(), x, x); moe.ops_sync()\n"
            "latch = N.load().moe_async_debug_latch_ops_word\n"
            "for words in ((0,), (1,), (2,), (0, 1), (1, 2), (0, 2), (0, 1, 2)):\n"
            "    for stream in (None, torch.cuda.Stream()):\n"
            "        for w in words:\n"
            "            N.check(latch(w, None), 'latch')\n"
            "        torch.cuda.synchronize()\n"
            "        try:\n"
            "            moe.ops_sync(stream=stream)\n"
            "            raise SystemExit(f'{words} not reported')\n"
            "        except moe.MoEError as e:\n"
            "            assert e.status == N.MOE_ERR_TIMEOUT\n"
            "        moe.ops_sync(); moe.ops_sync(stream=stream)\n"
            "assert latch(3, None) == latch(-1, None) == N.MOE_ERR_INVALID\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, "MOE_DEBUG_BOUNDS": "1"}, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
