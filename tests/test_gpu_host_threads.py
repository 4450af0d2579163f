"""Calls from several host threads at once, each with its own stream, workspace and results, on the GPU."""
import threading

import pytest
import torch

from block_diffusion_moe_gb300 import clover as C
from tests.test_gpu_attention import DEV, Case

pytestmark = pytest.mark.gpu


def _at_once(makers, times):
    """Each maker gives a call; all are made in turn, then `times` times at once, and must give what they gave alone."""
    failed = []

    def work(call, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(times):
                    got = call()
                    if i % 100 == 99:
                        torch.cuda.current_stream().synchronize()
                        if not torch.equal(got, want):
                            failed.append("results differ")
        except Exception as e:  # noqa: BLE001
            failed.append(str(e))

    calls = [m() for m in makers]
    wants = [c().clone() for c in calls]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=x) for x in zip(calls, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[:3]


@pytest.mark.parametrize("many,few", [(1024, 200), (160, 1)])  # a piece per warp, a team per SM
def test_cached_attention_of_different_batches(many, few):
    """The kernel's shared memory goes by the number of sequences."""
    def maker(n):
        def make():
            c = Case([1] * n, [20] * n, 32, 1, 64, seed=n)
            q, cache, args = c.q(4).to(DEV), c.cache(), c.args()
            ws = C.workspace(C.kv_attention_workspace_bytes(cache, c.rows, 4, *args[2].shape))
            out = torch.empty_like(q)
            return lambda: C.kv_attention(q, cache, *args, ws=ws, out=out)
        return make

    _at_once([maker(many), maker(few)] * 2, 3000)
