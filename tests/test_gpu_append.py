"""tri_append against the rotation and the slot rule in 64 bits.

Tolerance: the angle is reduced exactly to 2^-33 turns, rounded to fp32 as a part of
pi (pi 2^-24) and its sine and cosine are good to 2 ulp (2^-23): with two products and
a sum in fp32 (3 * 2^-24) each part of a pair is within 6e-7 |pair| of the exact turn,
then rounded once, by half a step of the stored type (bf16 2^-8, e4m3 2^-4 relative, or
2^-10 absolute among e4m3's subnormals)."""
import numpy as np
import pytest
import torch

import kv_cache_compression_calib_b200 as tri
from tests.prompt_ref import DTYPE, Batch, bytes_of, turned64

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {"bf16": (2.0 ** -8, 0.0), "fp8": (2.0 ** -4, 2.0 ** -10)}


def make_tokens(b, fused=False, far=0, seed=5, q=True):
    """Token tensors of batch b (fused: columns of one projection), positions around ``far``."""
    g = torch.Generator().manual_seed(seed)
    heads = b.hq + 2 * b.h
    x = (b.amp * torch.randn(b.L, b.T, heads, b.d, generator=g)).to(torch.bfloat16).to(b.dev)
    parts = [x[:, :, :b.hq], x[:, :, b.hq:b.hq + b.h], x[:, :, b.hq + b.h:]]
    if not fused:
        parts = [p.contiguous() for p in parts]
    pos = torch.randint(max(far - 50000, -2 ** 31), far + 50000, (b.T,), generator=g).clamp(max=2 ** 31 - 1).int().to(b.dev)
    return parts[0] if q else None, parts[1], parts[2], pos


def near(got, want, pair, elem, what):
    rel, sub = HALF_STEP[elem]
    fine = 6e-7 * pair
    tol = (want.abs() + fine) * rel + sub + fine
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), (got.double() - want).abs().max())


def pair_size(x, il):
    z = x.double()
    d = x.shape[-1]
    re, im = (z[..., 0::2], z[..., 1::2]) if il else (z[..., :d // 2], z[..., d // 2:])
    m = torch.hypot(re, im)
    return m.repeat_interleave(2, -1) if il else torch.cat((m, m), -1)


def check(b, q, k, v, pos, q_out, K, V, P, rotate=True, K0=None, V0=None):
    """Everything the call may write, and that it wrote nothing else."""
    n = int(b.tok[-1])
    if q is not None:
        near(q_out[:, :n], turned64(q[:, :n], pos[:n], b.theta, b.il), pair_size(q[:, :n], b.il), "bf16", "q")
    want_k = turned64(k, pos, b.theta, b.il) if rotate else k.double()
    pair = pair_size(k, b.il) if rotate else torch.zeros_like(want_k)
    held = (lambda x: x) if b.elem == "bf16" else (lambda x: x.clamp(-448, 448))
    left = torch.ones(K.numel() // b.d, dtype=torch.bool, device=b.dev)
    Kr, Vr, Pr = b.rows64(K), b.rows64(V), P.view(-1)
    for l in range(b.L):
        for s, ns in enumerate(b.new):
            for x in range(b.h):
                rec = b.rec((l * b.S + s) * b.h + x)
                i0 = max(0, ns - len(rec))
                rec = rec[len(rec) - (ns - i0):]
                toks = np.arange(int(b.tok[s]) + i0, int(b.tok[s + 1]))[rec >= 0]
                rec = torch.as_tensor(rec[rec >= 0]).to(b.dev)
                toks = torch.as_tensor(toks).to(b.dev)
                near(Kr[rec], held(want_k[l, toks, x]), pair[l, toks, x], b.elem, ("K", l, s, x))
                near(Vr[rec], held(v[l, toks, x].double()), torch.zeros_like(Vr[rec]), b.elem, ("V", l, s, x))
                assert torch.equal(Pr[rec], pos[toks]), (l, s, x)
                left[rec] = False
    for t, t0 in ((K, K0), (V, V0)):
        a, c = bytes_of(t).view(-1, b.d)[left], bytes_of(t0).view(-1, b.d)[left]
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
    assert (Pr[left] == -7).all()


def run(b, fused=False, far=0, mode=tri.TRI_KEYS_POST_ROPE, expect=0, with_q=True, kv=None, stream=None):
    q, k, v, pos = make_tokens(b, fused, far, q=with_q)
    q_out = torch.full((b.L, b.T, b.hq, b.d), 5.0, dtype=torch.bfloat16, device=DEV) if with_q else None
    K, V, P = b.K.clone(), b.V.clone(), b.pos.clone()
    ws = tri.alloc_append_workspace()
    tri.tri_append(b.m, kv or b.kv(), tri.tokens(k, v, b.tok_off, pos, q=q), mode, q_out, K, V, P, ws)
    st, flags = tri.tri_status_check(ws)
    assert flags == expect, flags
    check(b, q, k, v, pos, q_out, K, V, P, mode == tri.TRI_KEYS_POST_ROPE, b.K, b.V)
    if with_q:
        assert (q_out[:, int(b.tok[-1]):] == 5.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("elem", ["bf16", "fp8"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("layout", ["paged", "contig"])
def test_append(d, elem, il, layout):
    b = Batch([3, 0, 1, 40], [0, 9, 21, 5], hq=6, h=2, d=d, elem=elem, il=il, layout=layout, pad=3, dev=DEV, amp=2.0)
    run(b, fused=True)


@pytest.mark.parametrize("L,hq,h,bs,new", [(3, 4, 4, 1, [2, 5]), (1, 7, 1, 2, [1]), (2, 16, 8, 128, [300, 1, 77]),
                                            (1, 32, 8, 1024, [1100]), (1, 8, 8, 16, [1] * 70)])
def test_append_shapes(L, hq, h, bs, new):
    """Layers, groups, block sizes from 1 to 1024, more sequences than a warp has lanes."""
    b = Batch(new, [(7 * s + 3) % 29 for s in range(len(new))], L=L, hq=hq, h=h, bs=bs, dev=DEV)
    run(b, fused=False)


def test_append_many_tokens():
    """Enough tokens for whole tiles per block, the last one ragged."""
    run(Batch([4001, 1, 2000], [0, 5, 100], hq=2, h=1, dev=DEV, junk=0.0), fused=True)


@pytest.mark.parametrize("far", [0, 1 << 20, 2 ** 31 - 1, -2 ** 31])
def test_append_far_positions(far):
    run(Batch([65, 3], [1, 2], dev=DEV, theta=1e6), far=far)


def test_append_pre_rope_keys_and_no_queries():
    b = Batch([5, 6], [1, 0], dev=DEV)
    run(b, mode=tri.TRI_KEYS_PRE_ROPE)
    run(b, with_q=False)


def test_append_fp8_saturates_and_keeps_nan():
    b = Batch([4], [3], hq=1, h=1, d=64, elem="fp8", dev=DEV)
    k = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    v[0, 0, :6] = torch.tensor([1e6, -1e6, float("inf"), float("-inf"), float("nan"), 448.0])
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    ws = tri.alloc_append_workspace()
    K, V = b.K.clone(), b.V.clone()
    tri.tri_append(b.m, b.kv(), tri.tokens(k, v, b.tok_off, pos), tri.TRI_KEYS_POST_ROPE, None, K, V, None, ws)
    got = V.float().view(-1, 64)[int(b.rec(0)[3])]
    assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and torch.isnan(got[4]) and got[5] == 448.0


def test_append_in_place_queries_equal():
    b = Batch([9, 2], [0, 4], dev=DEV)
    q, k, v, pos = make_tokens(b)
    q = q.contiguous()
    out, ws = torch.empty_like(q), tri.alloc_append_workspace()
    K, V = b.K.clone(), b.V.clone()
    tri.tri_append(b.m, b.kv(), tri.tokens(k, v, b.tok_off, pos, q=q), tri.TRI_KEYS_POST_ROPE, out, K, V, None, ws)
    tri.tri_append(b.m, b.kv(), tri.tokens(k, v, b.tok_off, pos, q=q), tri.TRI_KEYS_POST_ROPE, q, K, V, None, ws)
    assert torch.equal(q, out)


def test_append_reports_what_it_cannot_place():
    """A sequence with more tokens than slots, a block id out of the pool, a table too short: flagged, skipped,
    the rest written."""
    b = Batch([6, 5], [0, 0], h=2, dev=DEV, row_len=[4, 6, 5, 5])
    run(b, expect=tri.TRI_FLAG_ROW_OFFSETS)
    b = Batch([40, 5], [0, 0], dev=DEV)
    b.table_np[0, 1] = b.nb
    run(b, expect=tri.TRI_FLAG_BLOCK_TABLE)
    b = Batch([40, 5], [0, 0], dev=DEV)
    b.table_np = np.ascontiguousarray(b.table_np[:, :2])
    run(b, expect=tri.TRI_FLAG_BLOCK_TABLE)


def test_append_inconsistent_token_offsets():
    b = Batch([4, 4], [0, 0], dev=DEV)
    q, k, v, pos = make_tokens(b)
    for bad in ([0, 4, 100], [0, 9, 8], [2, 1, 8]):
        ws = tri.alloc_append_workspace()
        tri.tri_append(b.m, b.kv(), tri.tokens(k, v, torch.tensor(bad, device=DEV), pos, q=q), tri.TRI_KEYS_POST_ROPE,
                       torch.empty_like(q.contiguous()), b.K.clone(), b.V.clone(), None, ws)
        assert tri.tri_status_check(ws)[1] == tri.TRI_FLAG_ROW_OFFSETS, bad


def test_append_on_another_stream_and_in_a_graph():
    b = Batch([3, 17], [2, 0], dev=DEV)
    q, k, v, pos = make_tokens(b)
    s = torch.cuda.Stream()
    K, V, P = b.K.clone(), b.V.clone(), b.pos.clone()
    q_out = torch.empty(b.L, b.T, b.hq, b.d, dtype=torch.bfloat16, device=DEV)
    kv, toks = b.kv(), tri.tokens(k, v, b.tok_off, pos, q=q)
    ws = tri.alloc_append_workspace()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tri.tri_append(b.m, kv, toks, tri.TRI_KEYS_POST_ROPE, q_out, K, V, P, ws)
    s.synchronize()
    check(b, q, k, v, pos, q_out, K, V, P, True, b.K, b.V)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tri.tri_append(b.m, kv, toks, tri.TRI_KEYS_POST_ROPE, q_out, K, V, P, ws)
    for new in range(2):  # the replay reads what the tensors then hold
        k.copy_(torch.randn(k.shape, device=DEV))
        K.copy_(b.K), V.copy_(b.V)
        g.replay()
        torch.cuda.synchronize()
        check(b, q, k, v, pos, q_out, K, V, P, True, b.K, b.V)
    del g


def test_append_to_a_pool_past_32_bit_offsets():
    """Blocks whose elements lie beyond 2^31 from the pool's start."""
    bs, h, d = 16, 8, 128
    nb = (1 << 31) // (bs * h * d) + 9
    K = torch.zeros(1, nb, bs, h, d, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    m = tri.model(1, 8, 8, 1e4)
    table = torch.tensor([[3, nb - 1, nb - 2]], dtype=torch.int32, device=DEV)
    row_off = torch.arange(h + 1, device=DEV) * 40
    kv = tri.kv_paged(1, row_off, 40 * h, table, bs, nb)
    k, v = (torch.randn(30, h, d, device=DEV).to(torch.bfloat16) for _ in range(2))
    ws = tri.alloc_append_workspace()
    tri.tri_append(m, kv, tri.tokens(k, v, torch.tensor([0, 30], device=DEV), torch.zeros(30, dtype=torch.int32, device=DEV)),
                   tri.TRI_KEYS_POST_ROPE, None, K, V, None, ws)
    assert tri.tri_status_check(ws) == (0, 0)
    for i in range(30):
        j = 10 + i
        blk = int(table[0, j // bs])
        assert torch.equal(K[0, blk, j % bs], k[i]) and torch.equal(V[0, blk, j % bs], v[i]), i
    assert DTYPE["bf16"] == K.dtype and not K[0, 4:nb - 2].any()


def test_append_wrong_caches_and_devices_are_refused():
    b = Batch([3, 2], [1, 0], dev=DEV)
    q, k, v, pos = make_tokens(b)
    ws = tri.alloc_append_workspace()
    t = tri.tokens(k, v, b.tok_off, pos, q=q)
    out = torch.empty_like(q.contiguous())
    for K, V, o, P in ((b.K.to(torch.float8_e4m3fn), b.V, out, None), (b.K, b.V[:, 1:].contiguous(), out, None),
                       (b.K, b.V, out[:, 1:], None), (b.K, b.V, out.float(), None), (b.K, b.V, out, b.pos.long()),
                       (b.K.cpu(), b.V, out, None), (b.K, b.V.transpose(1, 2), out, None)):
        with pytest.raises(ValueError):
            tri.tri_append(b.m, b.kv(), t, tri.TRI_KEYS_POST_ROPE, o, K, V, P, ws)
    with pytest.raises(ValueError):
        tri.tokens(k, v, b.tok_off, pos.cpu(), q=q)
    with pytest.raises(ValueError):
        tri.tri_append(tri.model(2, b.hq, b.h, 1e4), b.kv(), t, tri.TRI_KEYS_POST_ROPE, out, b.K, b.V, None, ws)
