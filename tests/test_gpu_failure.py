"""Failure detection on the GPU without a fault: the bounded wait of the staged
kernels is made to run out (a barrier nothing completes), and the host reads the
status it leaves; the context is then used again."""
import time

import numpy as np
import pytest
import torch

import kv_cache_compression_calib_b200 as tri
import synth
from tests import harness as H
from tests.test_gpu_parity import PRE, gpu_score, oracle_centres, oracle_scores, to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_staged_wait_times_out_and_the_context_stays_usable():
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    limit_ns = 20_000_000  # 20 ms
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    tri.tri_selftest_wait_timeout(ws, limit_ns)
    st, flags = tri.tri_status_check(ws)
    elapsed = time.perf_counter() - t0
    assert st == tri._abi.TRI_ERR_DEVICE_FLAG and flags == tri.TRI_FLAG_STAGE_TIMEOUT
    assert elapsed >= limit_ns * 1e-9
    st, flags = tri.tri_status_check(ws)  # the flag word was cleared
    assert st == 0 and flags == 0
    # the context still works: a staged scoring call meets the oracle
    wl = synth.WORKLOADS["single_layer_4k"].with_(name="after", batch=2, n_calib=32)
    host = synth.make_contig(wl, "cpu", lens=[700, 129], rotate=False)
    cs, ms = oracle_centres(host)
    got = gpu_score(to_dev(host), cs, ms, key_mode=PRE).cpu().numpy().astype(np.float64)
    ref, bound = oracle_scores(host, cs, ms, post_rope=False, tier="collapsed")
    assert H.score_error(got[:host.total], ref, bound) <= 1e-4


@pytest.mark.parametrize("elem,layout,bs", [("bf16", "contig", 16), ("bf16", "paged", 16), ("bf16", "paged", 4),
                                            ("fp8", "paged", 16), ("fp8", "paged", 2)])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("new,old", [([700, 900, 300, 5], [0, 300, 3000, 40]), ([1, 3, 2, 1] * 12, [3000, 9, 7000, 12000] * 12)])
def test_prompt_attention_gives_up_in_the_middle(elem, layout, bs, d, new, old):
    """Waits of prompt attention that give up after few tries, with copies, products, claims of items and the other
    warps' waits under way: the block ends, says so, and the next call has the results it always had.  Unseen values
    that are NaN send tiles through the mending warps."""
    from tests.prompt_ref import Batch

    b = Batch(new, old, hq=8, h=4, d=d, elem=elem, layout=layout, bs=bs, dev=DEV, junk=float("nan"), seed=d)
    kv, ws = b.kv(), tri.alloc_prefill_attention_workspace(b.m, b.S, b.T)

    def run(tries=None):
        out = torch.full((b.L, b.T, b.hq, b.d), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((b.L, b.T, b.hq), 7.0, device=DEV)
        args = (b.m, kv, b.K, b.V, b.q, b.tok_off, d ** -0.5, out, lse, ws)
        if tries is None:
            tri.tri_prefill_attention(*args)
        else:
            tri.tri_selftest_prefill_timeout(*args, tries)
        return out, lse, tri.tri_status_check(ws)[1]

    want, want_lse, flags = run()
    assert flags == 0
    got, got_lse, flags = run(1 << 26)  # the same kernels, with time enough
    assert flags == 0 and torch.equal(got, want) and torch.equal(got_lse, want_lse)
    gave_up = 0
    for tries in (1, 2, 3, 5, 9, 20, 50, 150, 400, 1000, 4000):
        t0 = time.perf_counter()
        got, got_lse, flags = run(tries)
        assert time.perf_counter() - t0 < 1.5  # a copy or product that was waited for in vain takes 2 s
        assert flags in (0, tri.TRI_FLAG_STAGE_TIMEOUT)
        gave_up += flags != 0
        if flags == 0:
            assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
        again, again_lse, flags = run()
        assert flags == 0 and torch.equal(again, want) and torch.equal(again_lse, want_lse)
    assert gave_up > 0
