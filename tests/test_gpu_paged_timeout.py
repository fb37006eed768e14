"""The waits of the kernels over pages give up too: after their limit, and at once where another
warp of the block has given up.  (kvd_debug_wait_timeout runs each form once, none of which can
end by its barrier; the limit is given, no fault or endless loop is involved.)"""
import time

import pytest
import torch

import long_context_decode_kv_gb300 as kvd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [2000, 100000])
def test_every_form_of_wait_runs_out(limit_us):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvd.debug_wait_timeout(status, 1)               # loads the kernel
    torch.cuda.synchronize()
    status.zero_()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    kvd.debug_wait_timeout(status, limit_us)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert kvd.STATUS[int(status.item())] == "KVD_ERR_TIMEOUT"
    # two waits take the limit each; the third, with 2 s to go, sees the flag
    assert 1.9e-6 * limit_us <= elapsed < 2e-6 * limit_us + 1.0
