"""Page allocation at the batch sizes where its shared memory passes 48 KB, each in a process of its own: what
an earlier call has asked for must not matter."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [(6111,), (6112,), (6113,), (6127,), (6128,), (6143,), (6144, 6130), (16384, 6128)])
def test_alloc_of_many_requests(sizes):
    body = "from tests.test_gpu_q8 import run_alloc\n" + "".join(
        f"run_alloc(16, [i % 40 for i in range({b})], [(i * 7) % 5 for i in range({b})])\n" for b in sizes)
    r = subprocess.run([sys.executable, "-c", body], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
