"""The error path of the kernels' bounded waits, exercised without a GPU
fault.  pa_test_decode_timeout runs pa_decode with every wait of the
partition kernel limited to a couple of milliseconds and with each CTA's
producer leaving one tile's shared-memory stage unfilled, as if its load had
never arrived (a flag that nothing sets).  The waits on that stage run out:
the kernel must flag PA_DEVERR_TIMEOUT, let the loads it did issue land and
return, and the next ordinary call on the same context must match the oracle.
"""
import time

import numpy as np
import pytest
import torch

from pagedattention_paged_kv_pa_b200 import workloads as W
from tests import parity as P

pytestmark = pytest.mark.gpu

PA_DEVERR_TIMEOUT = 4


@pytest.fixture(scope="module")
def B(cuda_device):
    from pagedattention_paged_kv_pa_b200 import binding
    return binding


@pytest.mark.parametrize("kv_dt", [W.BF16, W.FP8_E4M3])
def test_a_wait_that_runs_out_is_flagged_and_the_context_stays_usable(B, cuda_device, kv_dt):
    # partitions of 64-128 blocks, one of 13 blocks and one of 5 (which never
    # reaches the skipped tile 5 and completes normally)
    ctx = np.array([3000, 200, 1100], np.int32)
    spec = W.DecodeSpec("timeout", 3, 16, 2, 128, W.BF16, kv_dt, "fixed", (ctx,), max_ctx=3072,
                        seed=501)
    inp = W.make_decode_inputs(spec, ctx=ctx)
    d = inp.to(cuda_device)
    out = torch.empty_like(d.q)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    t0 = time.monotonic()
    B.pa_test_decode_timeout(out, d.q, d.k_pool, d.v_pool, d.block_tables, d.context_lens,
                             d.scale, skip_tile=5, wait_limit_us=2000, k_scale=d.k_scale,
                             v_scale=d.v_scale, dev_err=err)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 30
    assert int(err.item()) & PA_DEVERR_TIMEOUT
    gpu, e2 = P.run_decode(inp, cuda_device)
    assert e2 == 0
    P.assert_close(gpu, P.oracle_decode(inp), W.BF16, kv_dt, "decode after a timed-out call")


def test_the_hook_refuses_bad_arguments(B, cuda_device):
    spec = W.DecodeSpec("timeout_args", 1, 8, 2, 128, W.BF16, W.BF16, "fixed",
                        (np.array([40], np.int32),), max_ctx=64)
    d = W.make_decode_inputs(spec).to(cuda_device)
    out = torch.empty_like(d.q)
    for skip, limit in ((-1, 2000), (0, 0), (0, 2_000_000)):
        with pytest.raises(B.PAError):
            B.pa_test_decode_timeout(out, d.q, d.k_pool, d.v_pool, d.block_tables,
                                     d.context_lens, d.scale, skip_tile=skip,
                                     wait_limit_us=limit)


# The same of whole-prompt and tree attention, whose CTAs have a dozen warps or
# more that wait on one another: whichever waits for the missing tile gives up
# first and the others follow it.

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("skip", [0, 1, 4, 7])
def test_prompt_waits_that_run_out(B, cuda_device, d, skip):
    # prompts of 1 to 6 key tiles, each with a last V tile whose end is zeroed
    from tests import test_prefill_packed_gpu as T
    lens = [700, 90, 300, 1, 650, 128]
    q, k, v, start = T.make(lens, 16, 2, d, torch.bfloat16, cuda_device, seed=502)
    want, err = T.run(B, q, k, v, start, 0.09)
    assert err == 0
    out = torch.empty_like(want)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    t0 = time.monotonic()
    B.pa_test_prefill_packed_timeout(out, q, k, v, start, 0.09, skip_tile=skip,
                                     wait_limit_us=2000, dev_err=err)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 30
    assert int(err.item()) == PA_DEVERR_TIMEOUT
    got, err = T.run(B, q, k, v, start, 0.09)
    assert err == 0 and torch.equal(got, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [6, 40])  # one tile of rows, and two
@pytest.mark.parametrize("skip", [0, 3])
def test_tree_waits_that_run_out(B, cuda_device, fp8, d, nodes, skip):
    from tests import test_decode_tree_gpu as T
    c = T.Case([9000, 200, 6100, 77] * 4, nodes, 16, 4, d, torch.bfloat16, fp8, cuda_device,
               seed=503)
    want = c.run(B)
    a, k = c.args()
    out = torch.empty_like(want)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    t0 = time.monotonic()
    B.pa_test_decode_tree_timeout(out, *a, skip_tile=skip, wait_limit_us=2000, dev_err=err, **k)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 30
    assert int(err.item()) == PA_DEVERR_TIMEOUT
    assert torch.equal(c.run(B), want)


def test_the_attention_hooks_refuse_bad_arguments(B, cuda_device):
    from tests import test_decode_tree_gpu as T
    from tests import test_prefill_packed_gpu as TP
    q, k, v, start = TP.make([40], 4, 2, 64, torch.bfloat16, cuda_device)
    c = T.Case([40], 3, 4, 2, 64, torch.bfloat16, False, cuda_device)
    a, kw = c.args()
    for skip, limit in ((-1, 2000), (0, 0), (0, 2_000_000)):
        with pytest.raises(B.PAError):
            B.pa_test_prefill_packed_timeout(torch.empty_like(q.contiguous()), q, k, v, start, 0.1,
                                             skip_tile=skip, wait_limit_us=limit)
        with pytest.raises(B.PAError):
            B.pa_test_decode_tree_timeout(torch.empty_like(c.q), *a, skip_tile=skip,
                                          wait_limit_us=limit, **kw)
