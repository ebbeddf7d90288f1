"""tri_prefill_attention against the causal softmax in 64 bits.

Tolerance, with w the softmax weights: the output is rounded once (half a bf16 step,
2^-8 |out|); the weights enter the product with V rounded to bf16 (2^-8 sum w|v|); an
fp32 score is within eps = 4 d 2^-24 scale |q||k| and moves out by at most 2 eps
sum w|v|; exponentials (2^-19 relative) and fp32 sums over n keys (n 2^-24) add as much
of sum w|v|.  lse moves by eps, by the exponentials' and the sum's relative error, and
is rounded to fp32."""
import math

import numpy as np
import pytest
import torch

import kv_cache_compression_calib_b200 as tri
import oracle
from tests.prompt_ref import Batch, attend64, score_error

pytestmark = pytest.mark.gpu
DEV = "cuda"


def call(b, scale, out=None, lse=None, ws=None, kv=None, with_lse=True):
    out = torch.full((b.L, b.T, b.hq, b.d), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full((b.L, b.T, b.hq), 7.0, device=DEV) if lse is None and with_lse else lse
    ws = tri.alloc_prefill_attention_workspace(b.m, b.S, b.T) if ws is None else ws
    tri.tri_prefill_attention(b.m, kv or b.kv(), b.K, b.V, b.q, b.tok_off, scale, out, lse, ws)
    return out, lse, ws


def check(b, scale=None, expect=0):
    scale = b.d ** -0.5 if scale is None else scale
    out, lse, ws = call(b, scale)
    st, flags = tri.tri_status_check(ws)
    assert flags == expect, flags
    compare(b, scale, out, lse)
    return out, lse


def compare(b, scale, out, lse, rule=attend64):
    ref, rlse, mag = rule(b, scale)
    n = int(b.tok[-1])
    longest = int(np.diff(b.row_off_np).max()) if len(b.row_off_np) > 1 else 0
    eps = score_error(b, scale)
    rel = 2.0 ** -19 + longest * 2.0 ** -24
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * eps + 2 * rel) * mag
    got = out.double()
    bad = ~((got - ref).abs() <= tol)[:, :n]
    assert not bad.any(), (int(bad.sum()), (got - ref).abs()[:, :n].max(), torch.nonzero(bad)[:4])
    inf = torch.isinf(rlse[:, :n])
    assert torch.equal(torch.isinf(lse[:, :n]) & (lse[:, :n] < 0), inf)
    d = (lse.double() - rlse)[:, :n][~inf].abs()
    assert (d <= eps + rel + 2.0 ** -23 * rlse[:, :n][~inf].abs()).all(), d.max()
    assert (out[:, n:] == 7.0).all() and (lse[:, n:] == 7.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("elem", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["paged", "contig"])
def test_prefill(d, elem, layout):
    check(Batch([3, 0, 1, 150, 70], [0, 9, 300, 5, 259], hq=4, h=2, d=d, elem=elem, layout=layout, pad=3, dev=DEV))


@pytest.mark.parametrize("hq,h", [(1, 1), (6, 2), (5, 1), (16, 1), (24, 8), (40, 1), (130, 1)])
def test_prefill_groups(hq, h):
    """Groups that do not divide a tile's rows, one wider than a tile."""
    check(Batch([61, 2], [3, 140], hq=hq, h=h, d=64, dev=DEV))


@pytest.mark.parametrize("bs", [1, 2, 4, 8, 32, 64, 128, 512, 1024])
def test_prefill_block_sizes(bs):
    check(Batch([37, 140], [0, 111], hq=2, h=2, d=128, bs=bs, dev=DEV))


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385])
def test_prefill_lengths_around_tiles(n):
    check(Batch([n], [0], hq=1, h=1, dev=DEV))
    check(Batch([1], [n - 1], hq=1, h=1, dev=DEV, layout="contig"))


@pytest.mark.parametrize("old,new", [(4000, 1), (9000, 3), (5000, 40)])
@pytest.mark.parametrize("elem,d", [("bf16", 128), ("fp8", 64), ("bf16", 256)])
def test_prefill_few_tokens_over_long_rows(old, new, elem, d):
    """Rows long enough to be split over the keys and joined."""
    check(Batch([new, 1], [old, 0], hq=8, h=2, d=d, elem=elem, dev=DEV))


def test_prefill_layers_and_many_sequences():
    check(Batch([(3 * s) % 7 for s in range(45)], [s % 5 for s in range(45)], L=2, hq=2, h=1, d=64, dev=DEV))


def test_prefill_rows_of_unlike_lengths():
    """Row lengths of their own, shorter than the tokens and empty ones among them."""
    b = Batch([5, 6, 3], [0, 0, 0], hq=4, h=2, layout="contig", dev=DEV, row_len=[5, 3, 0, 200, 1, 3], pad=2)
    check(b)


@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("elem", ["bf16", "fp8"])
@pytest.mark.parametrize("which", ["K", "V"])
def test_prefill_nothing_of_later_tokens(layout, elem, which):
    """NaN in a later token's key or value (and in every record outside the rows) reaches no earlier token, and
    reaches every later one."""
    b = Batch([200, 30], [77, 0], hq=2, h=1, d=128, layout=layout, elem=elem, dev=DEV, junk=float("nan"))
    scale = b.d ** -0.5
    clean, clean_lse, _ = call(b, scale)
    at = int(b.rec(0)[77 + 150])
    t = getattr(b, which)
    t.view(torch.uint8 if elem == "fp8" else torch.bfloat16).view(-1, b.d)[at] = 0x7F if elem == "fp8" else float("nan")
    out, lse, _ = call(b, scale)
    assert torch.equal(out[0, :150], clean[0, :150]) and torch.equal(out[0, 200:], clean[0, 200:])
    assert torch.equal(lse[0, :150], clean_lse[0, :150])
    assert torch.isnan(out[0, 150:200]).all()


def test_prefill_infinite_values_of_later_tokens():
    b = Batch([140], [0], hq=2, h=1, d=64, layout="contig", dev=DEV)
    clean, _, _ = call(b, 0.125)
    b.V.view(-1, 64)[100, 3] = float("inf")
    b.V.view(-1, 64)[120, 3] = float("-inf")
    b.V.view(-1, 64)[110, 5] = float("-inf")
    out, _, _ = call(b, 0.125)
    assert torch.equal(out[0, :100], clean[0, :100])
    assert (out[0, 100:120, :, 3] == float("inf")).all() and torch.isnan(out[0, 120:140, :, 3]).all()
    assert torch.isfinite(out[0, 100:110, :, 5]).all() and (out[0, 110:140, :, 5] == float("-inf")).all()
    rest = [x for x in range(64) if x not in (3, 5)]
    assert torch.equal(out[0, :140][..., rest], clean[0, :140][..., rest])


def test_prefill_scores_far_apart():
    """Large scores of both signs, whose maximum keeps growing along the row."""
    b = Batch([300], [200], hq=2, h=1, d=128, dev=DEV, amp=0.5, layout="contig")
    K = b.rows64(b.K)
    ramp = torch.linspace(-60, 60, 500, device=DEV)[:, None].double()
    q = torch.ones(128, device=DEV).double() / 8
    K[:500] = K[:500] * 0.1 + ramp * q
    b.K.copy_(K.view(b.K.shape))
    b.q.copy_((torch.ones_like(b.q.float()) / 8 + 0.01 * b.q.float()).to(torch.bfloat16))
    check(b, scale=4.0)
    check(b, scale=1e-3)
    b.K.copy_(-b.K.float())
    check(b, scale=4.0)


def test_prefill_masks_and_scores_that_vanish():
    """Keys of negative infinity score: weight zero; a row of nothing else has no weight at all."""
    b = Batch([20], [30], hq=1, h=1, d=64, dev=DEV, layout="contig")
    b.q.fill_(1.0)
    Kr = b.K.view(-1, 64)
    Kr[10:40] = 0
    Kr[10:40, 0] = float("-inf")
    out, lse, _ = call(b, 0.125)
    keep = torch.ones(50, dtype=torch.bool)
    keep[10:40] = False
    for i in range(20):
        seen = keep.clone()
        seen[30 + i + 1:] = False
        s = 0.125 * Kr[:50][seen].double().sum(-1)
        w = torch.softmax(s, 0)
        v = b.V.view(-1, 64)[:50][seen.to(DEV)].double()
        assert (out[0, i, 0].double() - w @ v).abs().max() <= 2.0 ** -7 * (w @ v.abs()).max()
        assert abs(lse[0, i, 0].item() - torch.logsumexp(s, 0).item()) < 1e-4


def test_prefill_skips_blocks_it_cannot_place():
    b = Batch([70, 20], [100, 4], hq=2, h=2, dev=DEV)
    b.table_np[0, 2] = b.nb + 5
    b.table_np[0, 10] = -3
    check(b, expect=tri.TRI_FLAG_BLOCK_TABLE)
    b = Batch([70, 20], [100, 4], hq=2, h=2, dev=DEV)
    b.table_np = np.ascontiguousarray(b.table_np[:, :9])  # 144 of 170 slots have a table entry
    check(b, expect=tri.TRI_FLAG_BLOCK_TABLE)


def test_prefill_inconsistent_offsets():
    b = Batch([8, 8], [0, 30], dev=DEV)
    for bad in ([0, 8, 90], [0, 12, 8], [-3, 8, 16]):
        b.tok_off = torch.tensor(bad, device=DEV)
        _, _, ws = call(b, 0.1)
        assert tri.tri_status_check(ws)[1] == tri.TRI_FLAG_ROW_OFFSETS, bad
    b = Batch([8, 8], [0, 30], dev=DEV, layout="contig")
    good = b.row_off.clone()
    for at, x in ((1, -5), (2, 10 ** 9), (1, 60)):
        b.row_off = good.clone()
        b.row_off[at] = x
        _, _, ws = call(b, 0.1)
        assert tri.tri_status_check(ws)[1] == tri.TRI_FLAG_ROW_OFFSETS, (at, x)


def test_prefill_same_bits_every_time_and_without_lse():
    b = Batch([130, 3], [4000, 9], hq=8, h=2, dev=DEV)
    a, la, _ = call(b, 0.1)
    c, lc, _ = call(b, 0.1)
    d, _, _ = call(b, 0.1, with_lse=False)
    assert torch.equal(a, c) and torch.equal(la, lc) and torch.equal(a, d)


def test_prefill_two_streams_and_a_graph():
    """Two calls that overlap with a workspace each; a captured call replayed on new contents."""
    x, y = Batch([90, 5], [700, 0], dev=DEV, seed=1), Batch([1, 1], [3000, 2000], hq=8, dev=DEV, seed=2)
    keep = []
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for st, b in zip(s, (x, y)):
        with torch.cuda.stream(st):
            kv = b.kv()
            out = torch.full((b.L, b.T, b.hq, b.d), 7.0, dtype=torch.bfloat16, device=DEV)
            lse = torch.full((b.L, b.T, b.hq), 7.0, device=DEV)
            ws = tri.alloc_prefill_attention_workspace(b.m, b.S, b.T)
            keep.append((b, kv, out, lse, ws))
    for _ in range(5):
        for st, (b, kv, out, lse, ws) in zip(s, keep):
            with torch.cuda.stream(st):
                tri.tri_prefill_attention(b.m, kv, b.K, b.V, b.q, b.tok_off, 0.1, out, lse, ws)
    torch.cuda.synchronize()
    for b, kv, out, lse, ws in keep:
        compare(b, 0.1, out, lse)
    b, kv, out, lse, ws = keep[1]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tri.tri_prefill_attention(b.m, kv, b.K, b.V, b.q, b.tok_off, 0.1, out, lse, ws)
    b.q.copy_(torch.randn(b.q.shape, device=DEV))
    g.replay()
    torch.cuda.synchronize()
    compare(b, 0.1, out, lse)
    del g


def test_prefill_pool_past_32_bit_offsets():
    bs, h, d = 16, 8, 128
    nb = (1 << 31) // (bs * h * d) + 9
    K = torch.zeros(1, nb, bs, h, d, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    table = torch.tensor([[3, nb - 1, nb - 2]], dtype=torch.int32, device=DEV)
    k, v = (torch.randn(40, h, d, device=DEV).to(torch.bfloat16) for _ in range(2))
    for j in range(40):
        K[0, int(table[0, j // bs]), j % bs], V[0, int(table[0, j // bs]), j % bs] = k[j], v[j]
    m = tri.model(1, h, h, 1e4)
    kv = tri.kv_paged(1, torch.arange(h + 1, device=DEV) * 40, 40 * h, table, bs, nb)
    q = torch.randn(1, 2, h, d, device=DEV).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(1, 2, h, device=DEV)
    ws = tri.alloc_prefill_attention_workspace(m, 1, 2)
    tri.tri_prefill_attention(m, kv, K, V, q, torch.tensor([0, 2], device=DEV), 0.1, out, lse, ws)
    assert tri.tri_status_check(ws) == (0, 0)
    for i in range(2):
        for x in range(h):
            s = 0.1 * (k[:39 + i, x].double() @ q[0, i, x].double())
            w = torch.softmax(s, 0)
            vv = v[:39 + i, x].double()
            assert (out[0, i, x].double() - w @ vv).abs().max() <= 2.0 ** -6.9 * (w @ vv.abs()).max()


def test_prompt_then_decode():
    """A prompt appended and attended to, its cache scored and compacted, the next token appended to the compacted
    blocks and attended to by both attention calls, which agree with the oracle."""
    lens, B, W, bs, h, hq, d = [700, 300], 256, 32, 16, 2, 8, 128
    b = Batch(lens, [0, 0], hq=hq, h=h, d=d, dev=DEV, theta=1e6)
    g = torch.Generator().manual_seed(3)
    rnd = lambda *n: torch.randn(*n, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    T, S, scale = sum(lens), 2, d ** -0.5
    qkv = rnd(T, hq + 2 * h, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
    pos = torch.cat([torch.arange(n) for n in lens]).int().to(DEV)
    wsa = tri.alloc_append_workspace()
    b.q = torch.empty(1, T, hq, d, dtype=torch.bfloat16, device=DEV)
    tri.tri_append(b.m, b.kv(), tri.tokens(k, v, b.tok_off, pos, q=q), tri.TRI_KEYS_POST_ROPE, b.q, b.K, b.V, b.pos, wsa)
    assert tri.tri_status_check(wsa) == (0, 0)
    check(b)
    # calibrate on the prompt's own queries, score and compact into fresh blocks with room for one more token
    qcal = q[:256].permute(1, 0, 2)[None].contiguous()
    c, n = torch.empty(1, hq, d // 2, 2, device=DEV), torch.empty(1, hq, d // 2, device=DEV)
    tri.tri_calib(b.m, qcal, 256, c, n)
    ob = B // bs + 1
    table = torch.randperm(S * ob, generator=g).view(S, ob).int().to(DEV)
    Ko = torch.zeros(1, S * ob, bs, h, d, dtype=torch.bfloat16, device=DEV)
    Vo, Po = torch.zeros_like(Ko), torch.zeros(1, S * ob, bs, h, dtype=torch.int32, device=DEV)
    ws = tri.alloc_workspace(b.m, S, B)
    p_now = torch.tensor(lens, device=DEV)
    tri.tri_score_compact(b.m, b.kv(), b.K, b.V, b.pos, c, n, p_now, [1, 2, 4, 8], tri.TRI_KEYS_POST_ROPE, B, W, max(lens),
                          tri.out_paged(table, bs, S * ob), Ko, Vo, Po, None, None, None, ws)
    assert tri.tri_status_check(ws) == (0, 0)
    # the next token of each sequence: slot B, position lens[s]
    kv = tri.kv_paged(S, torch.arange(S * h + 1, device=DEV) * (B + 1), S * h * (B + 1), table, bs, S * ob)
    x = rnd(S, hq + 2 * h, d)
    one = torch.arange(S + 1, device=DEV)
    qd = torch.empty(1, S, hq, d, dtype=torch.bfloat16, device=DEV)
    before = Ko.clone()
    tri.tri_append(b.m, kv, tri.tokens(x[:, hq:hq + h], x[:, hq + h:], one, p_now.int(), q=x[:, :hq]), tri.TRI_KEYS_POST_ROPE,
                   qd, Ko, Vo, Po, wsa)
    assert tri.tri_status_check(wsa) == (0, 0)
    changed = (before != Ko).any(-1).view(-1, h).any(-1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted(int(table[s, B // bs]) * bs for s in range(S))
    out, lse = torch.empty(1, S, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, S, hq, device=DEV)
    wsp = tri.alloc_prefill_attention_workspace(b.m, S, S)
    tri.tri_prefill_attention(b.m, kv, Ko, Vo, qd, one, scale, out, lse, wsp)
    out2, lse2 = torch.empty(1, S, hq, d, device=DEV), torch.empty(1, S, hq, device=DEV)
    wsd = tri.alloc_attention_workspace(b.m, S)
    tri.tri_decode_attention(b.m, kv, Ko, Vo, qd, scale, out2, lse2, wsd)
    assert tri.tri_status_check(wsp) == (0, 0) and tri.tri_status_check(wsd) == (0, 0)
    for s in range(S):
        j = np.arange(B + 1)
        rec = table[s].cpu().numpy()[j // bs].astype(np.int64) * bs + j % bs
        for e in range(hq):
            kk, vv = (t.double().view(-1, h, d)[:, e // (hq // h)].cpu().numpy()[rec] for t in (Ko, Vo))
            ref, rlse = oracle.attention(qd[0, s, e].double().cpu().numpy(), kk, vv, scale)
            mag = np.abs(vv).max()
            assert np.abs(out2[0, s, e].double().cpu().numpy() - ref).max() <= 1e-4 * mag
            assert np.abs(out[0, s, e].double().cpu().numpy() - ref).max() <= 2.0 ** -6.9 * mag
            assert abs(lse[0, s, e].item() - rlse) <= 1e-4 and abs(lse2[0, s, e].item() - rlse) <= 1e-4
    assert math.isfinite(lse.sum().item())


@pytest.mark.parametrize("layout,bs", [("contig", 16), ("paged", 16), ("paged", 4)])
@pytest.mark.parametrize("new,old,h", [(200, 4000, 2), (2, 4000, 64), (1, 3000, 1)])
@pytest.mark.parametrize("elem", ["fp8", "bf16"])
def test_prefill_values_behind_a_sink(elem, layout, bs, new, old, h):
    """One key far above all others, whose value is zero in half the dims: what those dims hold comes from thousands
    of keys 15.8 to 17.9 nats below it.  Weights 2^-26 of the largest are within half a bf16 step in either type."""
    b = Batch([new], [old], hq=2 * h, h=h, d=64, elem=elem, layout=layout, bs=bs, dev=DEV, seed=new, v_mean=1.0)
    K, V = b.rows64(b.K).clone(), b.rows64(b.V).clone()
    g = torch.Generator().manual_seed(h)
    # by the first two dims: scores of -1 .. 1, and 16.875 of the sink
    small = (torch.randint(-16, 17, (K.shape[0],), generator=g).double() / 16 * 4).to(DEV)
    small = small.to(torch.float8_e4m3fn).double()
    K[:] = 0
    K[:, 0] = small
    for x in range(h):
        rec = int(b.rec(x)[5])
        K[rec, 0], K[rec, 1] = 0, 18
        V[rec, :32] = 0
    b.K.copy_(K.view(b.K.shape))
    b.V.copy_(V.view(b.V.shape))
    b.q.zero_()
    b.q[..., 0], b.q[..., 1] = 0.25, 0.9375
    check(b, scale=1.0)
