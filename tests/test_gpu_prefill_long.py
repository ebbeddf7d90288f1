"""tri_prefill_attention over rows of 2^31 16-byte chunks and more: a paged row may name the
same block many times, so the pool stays small.  The softmax in 64 bits weighs each record by
how often the table names it.  Tolerance: as in test_gpu_prefill, with the fp32 sums' error
from the additions really made one after another (of a thread's key tiles: half of a split's
where both warpgroups take the same rows; eight per tile in the product with V, whose adder may
truncate)."""
import numpy as np
import pytest
import torch

import kv_cache_compression_calib_b200 as tri
from tests.test_gpu_prefill import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_rows_past_31_bits_of_chunks(d):
    bs, n, tail = 1024, 3, 133
    full = (1 << 31) // (d // 8) // bs + 1
    slots = full * bs + tail
    g = torch.Generator().manual_seed(d)
    table = torch.randint(0, 3, (1, full + 1), generator=g, dtype=torch.int32)
    table[0, full] = 3
    K, V = (torch.randn(1, 4, bs, 1, d, generator=g).to(torch.bfloat16) for _ in range(2))
    V = (V.float() + 1).to(torch.bfloat16)
    K[0, 3, tail:], V[0, 3, tail:] = float("nan"), float("nan")  # behind the row's end, in its last page
    q = torch.randn(1, n, 1, d, generator=g).to(torch.bfloat16)
    m, scale = tri.model(1, 1, 1, 1e4, d), d ** -0.5
    kv = tri.kv_paged(1, torch.tensor([0, slots], device=DEV), slots, table.to(DEV), bs, 4)
    out, lse = torch.empty(1, n, 1, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, n, 1, device=DEV)
    ws = tri.alloc_prefill_attention_workspace(m, 1, n)
    tri.tri_prefill_attention(m, kv, K.to(DEV), V.to(DEV), q.to(DEV), torch.tensor([0, n], device=DEV), scale, out, lse, ws)
    assert tri.tri_status_check(ws) == (0, 0)

    named = np.bincount(table[0].numpy(), minlength=4).astype(np.float64)
    k, v = K.double().view(-1, d).numpy(), V.double().view(-1, d).numpy()
    splits = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = slots / (64 if d == 256 else 128) / splits
    sums = (tiles + 128 + splits) * 2.0 ** -24
    adds = (8 * tiles + splits) * 2.0 ** -23
    rel = 2.0 ** -19 + sums
    for i in range(n):
        seen = 3 * bs + tail - n + i + 1
        times = np.repeat(named, bs)[:seen]
        times[3 * bs:] = 1.0
        qi = q[0, i, 0].double().numpy()
        s = scale * (k[:seen] @ qi)
        w = times * np.exp(s - s.max())
        total = w.sum()
        ref, mag = w @ v[:seen] / total, w @ np.abs(v[:seen]) / total
        eps = 4 * d * 2.0 ** -24 * scale * np.linalg.norm(qi) * np.linalg.norm(k[:seen], axis=-1).max()
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * eps + 2 * rel + adds) * mag
        assert (np.abs(out[0, i, 0].double().cpu().numpy() - ref) <= tol).all(), i
        rlse = s.max() + np.log(total)
        assert abs(lse[0, i, 0].item() - rlse) <= eps + rel + 2.0 ** -23 * abs(rlse)
