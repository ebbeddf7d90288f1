"""tri_prefill_attention where a block takes several items of unlike kinds: more pieces of
work than the GPU has SMs, long and short rows, few and many tokens, special values in
some of them.  Tolerances as in test_gpu_prefill."""
import random

import pytest
import torch

import kv_cache_compression_calib_b200 as tri
from tests.prompt_ref import Batch, attend64_rows
from tests.test_gpu_prefill import call, compare

pytestmark = pytest.mark.gpu
DEV = "cuda"


def mixed(seed, S, new, old):
    r = random.Random(seed)
    return [r.choice(new)(r) for _ in range(S)], [r.choice(old)(r) for _ in range(S)]


def check(b, times=2):
    scale = b.d ** -0.5
    for _ in range(times):
        out, lse, ws = call(b, scale)
        assert tri.tri_status_check(ws) == (0, 0)
        compare(b, scale, out, lse, rule=attend64_rows)


few = [lambda r: 1, lambda r: r.randint(1, 9), lambda r: r.randint(10, 60), lambda r: 0]
many = [lambda r: r.randint(100, 500), lambda r: r.randint(1, 40), lambda r: r.randint(500, 900)]
short = [lambda r: 0, lambda r: r.randint(1, 300)]
both = [lambda r: 0, lambda r: r.randint(1, 200), lambda r: r.randint(900, 4000)]


@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("elem", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_items_of_few_tokens(layout, elem, d):
    new, old = mixed(d, 50, few, both)
    check(Batch(new, old, L=2, hq=8, h=4, d=d, elem=elem, layout=layout, dev=DEV, pad=5, seed=d))


@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("elem", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_items_of_whole_prompts(layout, elem, d):
    new, old = mixed(d + 1, 20, many, short)
    check(Batch(new, old, L=2, hq=16, h=8, d=d, elem=elem, layout=layout, dev=DEV, seed=d))


@pytest.mark.parametrize("d", [64, 128])
def test_items_of_long_and_short_pages(d):
    """Long paged rows between short ones; with few tokens, whose values come by a warp of their own, on blocks that
    take many items."""
    new, old = [300, 40, 700, 3, 280, 1, 200, 17], [20000, 0, 16000, 19000, 30, 21000, 15000, 0]
    check(Batch(new, old, L=2, hq=16, h=8, d=d, dev=DEV, seed=d), times=3)
    new, old = [70, 3, 150, 1, 1, 2, 90, 1, 1, 5, 1, 64], [9000, 12000, 0, 11000, 8, 700, 9000, 400, 10000, 0, 13000, 600]
    check(Batch(new * 3, old * 3, L=1, hq=16, h=8, d=d, dev=DEV, seed=d), times=3)


@pytest.mark.parametrize("hq,bs", [(24, 16), (40, 16), (16, 4), (24, 2)])
@pytest.mark.parametrize("elem", ["bf16", "fp8"])
def test_items_without_tma(hq, bs, elem):
    """Groups that do not divide a query tile, and pages smaller than a swizzle atom."""
    new, old = mixed(hq + bs, 12, many + few, short)
    check(Batch(new, old, hq=hq, h=8, d=128, bs=bs, elem=elem, dev=DEV, seed=bs))


def test_thousands_of_sequences():
    check(Batch([1] * 1500 + [0, 3] * 100, [s % 7 for s in range(1700)], hq=2, h=1, d=64, dev=DEV), times=1)


@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("elem", ["bf16", "fp8"])
@pytest.mark.parametrize("size", ["few", "prompts"])
def test_special_values_stay_in_their_items(layout, elem, size):
    """NaN in the values of some sequences' last tokens: those tokens and no others have them, bit for bit, whatever
    items ran before and after on the same block."""
    new, old = mixed(7, 40, [lambda r: r.randint(2, 40)] if size == "few" else many, both if size == "few" else short)
    new = [max(2, n) for n in new]
    b = Batch(new, old, hq=8, h=4, d=128, elem=elem, layout=layout, dev=DEV, junk=float("nan"), seed=9)
    scale = b.d ** -0.5
    clean, clean_lse, _ = call(b, scale)
    hit = torch.zeros(b.T, b.hq, dtype=torch.bool, device=DEV)
    V = b.V.view(torch.uint8 if elem == "fp8" else torch.bfloat16).view(-1, b.d)
    for s in range(0, len(new), 3):
        x = s % b.h
        rec = b.rec(s * b.h + x)
        back = 1 + s % min(2, new[s])  # tokens from the sequence's end that see it
        V[int(rec[len(rec) - back]), 5 * s % b.d] = 0x7F if elem == "fp8" else float("nan")
        hit[int(b.tok[s + 1]) - back:int(b.tok[s + 1]), x * 2:x * 2 + 2] = True
    for _ in range(3):
        out, lse, ws = call(b, scale)
        assert tri.tri_status_check(ws) == (0, 0)
        nan = torch.isnan(out[0]).any(-1)
        assert torch.equal(nan, hit)
        assert torch.equal(lse, clean_lse)
        same = out[0].clone()
        same[torch.isnan(same)] = clean[0][torch.isnan(same)]
        assert torch.equal(same, clean[0])


def test_output_on_a_16_byte_boundary():
    """Rows of out that no 32-byte store may write."""
    b = Batch([200, 3], [50, 4000], hq=4, h=2, d=128, dev=DEV)
    n = b.L * b.T * b.hq * b.d
    buf = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8:n + 8].view(b.L, b.T, b.hq, b.d)
    assert out.data_ptr() % 32 == 16
    want, _, _ = call(b, 0.1)
    call(b, 0.1, out=out)
    assert torch.equal(out, want) and (buf[:8] == 7.0).all() and (buf[n + 8:] == 7.0).all()


def test_wrong_device_type_and_size_are_refused():
    b = Batch([4], [4], dev=DEV)
    ws = tri.alloc_prefill_attention_workspace(b.m, 1, 4)
    out, lse = torch.empty_like(b.q), torch.empty(1, 4, b.hq, device=DEV)
    args = dict(K=b.K, V=b.V, q=b.q, tok_off=b.tok_off, softmax_scale=0.1, out=out, lse=lse, ws=ws)
    for bad in (dict(K=b.K.cpu()), dict(out=out.float()), dict(lse=lse[:, :2]), dict(tok_off=b.tok_off.int()),
                dict(q=b.q.transpose(1, 2)), dict(out=out[:, :3])):
        with pytest.raises(ValueError):
            tri.tri_prefill_attention(b.m, b.kv(), **{**args, **bad})
    with pytest.raises(tri.TriError):
        tri.tri_prefill_attention(b.m, b.kv(), **{**args, "ws": ws[:256]} if ws.numel() > 256 else {**args, "ws": ws[:128]})


@pytest.mark.parametrize("layout", ["paged", "contig"])
@pytest.mark.parametrize("old", [[5, 3000], [0, 0]])
def test_no_sequence_has_tokens(layout, old):
    """A padded batch of nothing: no row is written, nothing is flagged."""
    b = Batch([0, 0], old, layout=layout, pad=6, dev=DEV)
    out, lse, ws = call(b, 0.1)
    assert tri.tri_status_check(ws) == (0, 0)
    assert (out == 7.0).all() and (lse == 7.0).all()
    out, _, _ = call(b, 0.1, with_lse=False)
    assert (out == 7.0).all()


def test_workspace_is_reused_by_calls_of_other_shapes():
    """One workspace, large enough for each, in stream order: split rows, then whole ones, then split ones."""
    shapes = [Batch([1], [9000], hq=8, h=2, dev=DEV, seed=1), Batch([300, 200], [0, 50], hq=8, h=2, dev=DEV, seed=2),
              Batch([4, 2], [5000, 7000], hq=8, h=2, d=64, dev=DEV, seed=3)]
    n = max(tri.tri_prefill_attention_ws_size(b.m, b.S, b.T) for b in shapes)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    tri.tri_workspace_init(ws)
    got = [call(b, b.d ** -0.5, ws=ws)[:2] for b in shapes + shapes]
    assert tri.tri_status_check(ws) == (0, 0)
    for b, (out, lse) in zip(shapes + shapes, got):
        compare(b, b.d ** -0.5, out, lse, rule=attend64_rows)


def test_workspace_of_the_largest_batch_serves_smaller_ones():
    """Allocated once for the largest batch (whose rows are not split), then used by calls of fewer tokens (whose
    rows are): results and flags as with a workspace of their own, and nothing behind its end written."""
    batches = [Batch([900, 700, 300, 200], [0, 50, 9, 3000], hq=16, h=8, dev=DEV, seed=4),
               Batch([1], [9000], hq=16, h=8, dev=DEV, seed=5), Batch([5, 1, 3], [5000, 9000, 20], hq=16, h=8, dev=DEV, seed=6)]
    n = tri.tri_prefill_attention_ws_size(batches[0].m, batches[0].S, batches[0].T)
    buf = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    ws = buf[:n]
    tri.tri_workspace_init(ws)
    for b in batches:
        out, lse, _ = call(b, 0.1, ws=ws)
        assert tri.tri_status_check(ws) == (0, 0)
        compare(b, 0.1, out, lse, rule=attend64_rows)
    assert (buf[n:] == 0x5A).all()


@pytest.mark.parametrize("elem,bs", [("bf16", 16), ("fp8", 16), ("bf16", 4), ("fp8", 64)])
@pytest.mark.parametrize("new,old", [([300, 70, 1], [3000, 5000, 9000]), ([2, 1, 3, 1], [6000, 9000, 7000, 300])])
def test_unnamed_blocks_that_the_copies_meet_tiles_ahead(elem, bs, new, old):
    """Blocks that the table does not name, in tiles that the copies reach while the softmax is tiles behind: skipped
    and flagged, the same bits every time."""
    b = Batch(new, old, hq=8, h=2, d=64, elem=elem, bs=bs, dev=DEV, seed=bs)
    for s in range(len(new)):
        there = (new[s] + old[s]) // bs
        b.table_np[s, [there // 5, there // 2, there // 2 + 1, there - 3]] = [-1, b.nb, -7, b.nb + 9]
    scale, seen = b.d ** -0.5, None
    for _ in range(4):
        out, lse, ws = call(b, scale)
        assert tri.tri_status_check(ws)[1] == tri.TRI_FLAG_BLOCK_TABLE
        if seen is None:
            seen = (out, lse)
            compare(b, scale, out, lse, rule=attend64_rows)
        assert torch.equal(out, seen[0]) and torch.equal(lse, seen[1])
