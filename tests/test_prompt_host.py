"""Host checks of tri_append and tri_prefill_attention: every refusal comes before any
CUDA call, so these run without a GPU (the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import kv_cache_compression_calib_b200 as tri
from kv_cache_compression_calib_b200 import _abi

A = 1 << 20
M = tri.model(1, 32, 8, 1e6)
BAD, UNSUP, ALIGN, SMALL = (_abi.TRI_ERR_INVALID_ARG, _abi.TRI_ERR_UNSUPPORTED, _abi.TRI_ERR_ALIGNMENT,
                            _abi.TRI_ERR_WORKSPACE_TOO_SMALL)


def kv(layout=0, n_seqs=1, total=4096, row_off=A, table=None, max_blocks=0, bs=0, nb=0, elem=0):
    return _abi.TriKvDesc(layout, n_seqs, total, row_off, table, max_blocks, bs, nb, elem, 0)


def append(m=M, kv_=None, T=4, tok_off=A, positions=A, q=16 * A, k=32 * A, v=48 * A, qs=32 * 128, ks=8 * 128, vs=8 * 128,
           mode=0, q_out=64 * A, K=80 * A, V=96 * A, pos=None, ws=A, ws_bytes=256, toks=True):
    t = _abi.TriTokenDesc(T, tok_off, positions, q, k, v, qs, ks, vs)
    return _abi.load().tri_append(ctypes.byref(m), ctypes.byref(kv_ or kv()), ctypes.byref(t) if toks else None, mode, q_out,
                                  K, V, pos, ws, ws_bytes, None)


def prefill(m=M, kv_=None, K=A, V=2 * A, q=3 * A, tok_off=A, T=4, scale=0.1, out=5 * A, lse=None, ws=A, ws_bytes=1 << 40):
    return _abi.load().tri_prefill_attention(ctypes.byref(m), ctypes.byref(kv_ or kv()), K, V, q, tok_off, T, scale, out, lse,
                                             ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(toks=False), BAD), (dict(T=-1), BAD), (dict(tok_off=None), BAD), (dict(positions=None), BAD), (dict(k=None), BAD),
    (dict(v=None), BAD), (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(K=None), BAD), (dict(V=None), BAD),
    (dict(V=80 * A), BAD), (dict(mode=2), BAD), (dict(ws=None), BAD), (dict(ws_bytes=255), SMALL), (dict(ws=A + 64), ALIGN),
    (dict(T=1 << 31), UNSUP), (dict(qs=32 * 128 - 8), BAD), (dict(ks=8 * 128 - 8), BAD), (dict(vs=0), BAD),
    (dict(ks=-8 * 128), BAD), (dict(qs=1 << 55), BAD), (dict(vs=1 << 62), BAD), (dict(T=1 << 30, ks=1 << 27), BAD), (dict(qs=32 * 128 + 4), ALIGN), (dict(ks=8 * 128 + 2), ALIGN),
    (dict(q=16 * A + 2), ALIGN), (dict(k=32 * A + 8), ALIGN), (dict(q_out=64 * A + 8), ALIGN), (dict(K=80 * A + 8), ALIGN),
    (dict(V=96 * A + 2), ALIGN), (dict(tok_off=A + 4), ALIGN), (dict(positions=A + 2), ALIGN), (dict(pos=A + 1), ALIGN),
    # q_out over the queries (but not exactly in place), over the keys, over the values
    (dict(q_out=16 * A, qs=48 * 128), BAD), (dict(q_out=16 * A + 16), BAD), (dict(q_out=32 * A), BAD), (dict(q_out=48 * A), BAD),
    (dict(m=tri.model(1, 32, 8, 1e6, head_dim=96)), UNSUP), (dict(m=tri.model(1, 1 << 21, 8, 1e6), qs=1 << 28), UNSUP),
    (dict(kv_=kv(n_seqs=0)), BAD), (dict(kv_=kv(elem=3)), BAD), (dict(kv_=kv(layout=1, table=A, max_blocks=2, bs=12, nb=3)), UNSUP),
])
def test_append_refuses(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=None), BAD), (dict(V=None), BAD), (dict(q=None), BAD), (dict(tok_off=None), BAD), (dict(out=None), BAD),
    (dict(out=3 * A), BAD), (dict(T=-1), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(K=A + 8), ALIGN), (dict(V=A + 8), ALIGN), (dict(q=A + 8), ALIGN), (dict(out=A + 4), ALIGN),
    (dict(tok_off=A + 4), ALIGN), (dict(lse=A + 2), ALIGN), (dict(ws=A + 16), ALIGN), (dict(ws=None), BAD), (dict(ws_bytes=255), SMALL),
    (dict(T=1 << 31), UNSUP), (dict(m=tri.model(1, 32, 8, 1e6, head_dim=32)), UNSUP), (dict(kv_=kv(total=-1)), BAD),
    (dict(kv_=kv(layout=1)), BAD), (dict(out=3 * A + 4096), BAD), (dict(out=3 * A - 32 * 128 * 8 + 16), BAD), (dict(scale=3e38), BAD),
    (dict(m=tri.model(1, 128, 1, 1e6), T=1 << 25), UNSUP), (dict(m=tri.model(1 << 20, 8, 8, 1e6), kv_=kv(n_seqs=64), T=64), UNSUP),
])
def test_prefill_refuses(kw, status):
    assert prefill(**kw) == status


def test_no_tokens_is_no_work():
    assert append(T=0, q=None, q_out=None, k=None, v=None, K=None, V=None, tok_off=None, positions=None) == 0
    assert prefill(T=0, K=None, V=None, q=None, out=None, tok_off=None) == 0


def test_prefill_workspace_size():
    n = tri.tri_prefill_attention_ws_size
    assert n(M, 1, 0) >= 256 and n(M, 0, 4) == 0 and n(M, 1, -1) == 0
    assert n(tri.model(1, 32, 8, 1e6, head_dim=80), 1, 4) == 0
    for m in (M, tri.model(64, 64, 8, 1e6), tri.model(1, 8, 8, 1e4, head_dim=256)):
        for S, T in ((1, 1), (16, 16), (3, 5000), (64, 100000)):
            assert 256 <= n(m, S, T) <= 256 << 20 and n(m, S, T) % 256 == 0


class _Fake:
    """A CUDA tensor as far as tokens() looks at one (there is no device here)."""
    is_cuda, device, dtype = True, "cuda:0", torch.bfloat16

    def __init__(self, t):
        self.t = t
        self.shape, self.numel, self.stride, self.dim = t.shape, t.numel, t.stride, t.dim

    def data_ptr(self):
        return 64 + 2 * self.t.storage_offset()


def test_token_rows_of_fused_projections():
    x = torch.zeros(3, 5, 10, 64, dtype=torch.bfloat16)
    rows = lambda t: tri._token_rows(_Fake(t), "x")  # noqa: E731
    assert rows(x) == (64, 640)
    assert rows(x[:, :, 4:6]) == (64 + 2 * 4 * 64, 640)
    assert rows(x[1, :, 4:6])[1] == 640
    assert rows(x[:, :1, 4:6].contiguous())[1] == 128
    for bad in (x.transpose(2, 3), x.transpose(0, 1), x[..., ::2], x[:, :, ::2], x[:, :4]):
        with pytest.raises(ValueError):
            rows(bad)
    with pytest.raises(ValueError):
        tri._token_rows(x, "x")  # not on a GPU
    with pytest.raises(ValueError):
        tri._token_rows(_Fake(x[0, 0]), "x")


class _Device:
    """Stands in for a CUDA tensor of this many elements (there is no device here)."""
    is_cuda, device = True, torch.device("cuda:0")

    def __init__(self, dtype, *shape):
        self.t, self.dtype, self.shape = torch.empty(shape, device="meta"), dtype, torch.Size(shape)
        self.numel, self.stride, self.dim, self.is_contiguous = self.t.numel, self.t.stride, self.t.dim, self.t.is_contiguous

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def get_device(self):
        return 0

    def data_ptr(self):
        return A


class _Calls:
    """Stands in for the library and counts the calls that reach it."""

    def __init__(self):
        self.n = 0

    def tri_append(self, *a):
        self.n += 1
        return 0


@pytest.fixture
def reached(monkeypatch):
    calls = _Calls()
    monkeypatch.setattr(tri, "_L", calls)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(tri, "_s", lambda stream: 0)
    return calls


def append_call(layout, S=2, T=5, L=2, h=2, hq=4, d=64, offsets=None, positions=0):
    """tri_append of T tokens of S sequences into a cache of 100 (contiguous) or 3 * 16 * h * L (paged) records."""
    i64, i32, bf16 = torch.int64, torch.int32, torch.bfloat16
    t = tri.tokens(_Device(bf16, L, T, h, d), _Device(bf16, L, T, h, d), _Device(i64, offsets or S + 1), _Device(i32, T))
    n = 3 * 16 * h * L if layout == "paged" else 100
    if layout == "paged":
        kv = tri.kv_paged(S, _Device(i64, L * S * h + 1), 100, _Device(i32, S, 3), 16, 3)
    else:
        kv = tri.kv_contig(S, _Device(i64, L * S * h + 1), 100)
    pos = None if positions is None else _Device(i32, n + positions)
    tri.tri_append(tri.model(L, hq, h, 1e4, d), kv, t, 0, None, _Device(bf16, n, d), _Device(bf16, n, d), pos,
                   _Device(torch.uint8, 256))


@pytest.mark.parametrize("layout", ["contig", "paged"])
def test_append_refuses_offsets_and_positions_of_other_sizes(reached, layout):
    """Fewer token offsets than the kernel reads, or positions than it may write: refused before the library is called."""
    for good in (dict(), dict(positions=7), dict(positions=None)):
        append_call(layout, **good)
    assert reached.n == 3
    for bad in (dict(offsets=2), dict(offsets=1), dict(offsets=4), dict(positions=-1), dict(positions=-90)):
        with pytest.raises(ValueError):
            append_call(layout, **bad)
    assert reached.n == 3


def test_append_refuses_tokens_made_by_hand(reached):
    """A descriptor without its tensors, which have to be checked, is refused by name."""
    kv_, m = tri.kv_contig(2, _Device(torch.int64, 5), 100), tri.model(1, 4, 2, 1e4, 64)
    made = _abi.TriTokenDesc(5, A, A, None, A, A, 0, 128, 128)
    with pytest.raises(ValueError, match="tokens"):
        tri.tri_append(m, kv_, made, 0, None, _Device(torch.bfloat16, 100, 64), _Device(torch.bfloat16, 100, 64), None,
                       _Device(torch.uint8, 256))
    assert reached.n == 0


@pytest.mark.parametrize("m", [M, tri.model(1, 8, 1, 1e4), tri.model(2, 40, 40, 1e4, 64), tri.model(3, 27, 27, 1e4), tri.model(1, 1, 1, 1e4),
                               tri.model(1, 64, 2, 1e4, 256), tri.model(64, 64, 8, 1e6), tri.model(1, 300, 1, 1e4)])
def test_prefill_workspace_serves_smaller_calls(m):
    """A workspace of n_seqs sequences and total_tokens tokens is enough for every call of at most as many."""
    sizes = [(s, t) for s in (1, 2, 3, 4, 9, 16, 64) for t in (1, 2, 4, 16, 40, 129, 512, 2000, 8192, 100000)]
    most = {x: tri.tri_prefill_attention_ws_size(m, *x) for x in sizes}
    for S, T in sizes:
        for s, t in sizes:
            if s <= S and t <= T:
                assert most[S, T] >= most[s, t]
                # the size is looked at before the addresses (a missing one here), so no kernel is launched
                assert prefill(m=m, kv_=kv(n_seqs=s), T=t, K=None, ws_bytes=most[S, T]) == BAD


def test_prefill_workspace_of_one_call():
    """What a call of many tokens needs is its flag word alone, as a workspace made for it alone always was."""
    assert prefill(kv_=kv(n_seqs=1), T=8192, K=None, ws_bytes=256) == BAD
    assert prefill(kv_=kv(n_seqs=1), T=1, K=None, ws_bytes=256) == SMALL
    assert prefill(kv_=kv(n_seqs=1), T=1 << 62, K=None, ws_bytes=256) == BAD


def test_prefill_selftest_rejects_bad_arguments():
    def f(tries, d=64, ws_bytes=1 << 40, K=A):
        m = tri.model(1, 32, 8, 1e6, head_dim=d)
        return _abi.load().tri_selftest_prefill_timeout(ctypes.byref(m), ctypes.byref(kv()), K, 2 * A, 3 * A, A, 4, 0.1, 5 * A, None,
                                                        A, ws_bytes, tries, None)

    assert f(0) == BAD and f((1 << 26) + 1) == BAD and f(9, K=None) == BAD
    assert f(9, d=128) == UNSUP and f(9, ws_bytes=255) == SMALL


@pytest.mark.parametrize("layout", ["contig", "paged"])
def test_append_and_prefill_refuse_descriptors_of_other_sizes(reached, layout):
    """Row offsets, block tables and devices are compared with the model's: a descriptor made for fewer layers or heads, or
    on another device, is refused before the library is called."""
    reached.tri_prefill_attention = reached.tri_append
    i64, i32, bf16 = torch.int64, torch.int32, torch.bfloat16
    S, T, h, d = 3, 5, 2, 64
    n = 4 * 16 * h * 2

    def calls(offsets, tables=S, device=0):
        off, tab = _Device(i64, offsets), _Device(i32, tables, 4)
        off.get_device = tab.get_device = lambda: device
        off.device = tab.device = torch.device("cuda", device)
        kv_ = tri.kv_paged(S, off, n, tab, 16, 4) if layout == "paged" else tri.kv_contig(S, off, n)
        m, ws = tri.model(2, 4, h, 1e4, d), _Device(torch.uint8, 256)
        K, V, tok = _Device(bf16, n, d), _Device(bf16, n, d), _Device(i64, S + 1)
        t = tri.tokens(_Device(bf16, 2, T, h, d), _Device(bf16, 2, T, h, d), tok, _Device(i32, T))
        q = _Device(bf16, 2, T, 4, d)
        return (lambda: tri.tri_append(m, kv_, t, 0, None, K, V, None, ws),
                lambda: tri.tri_prefill_attention(m, kv_, K, V, q, tok, 0.1, q, None, ws))

    for call in calls(2 * S * h + 1) + calls(2 * S * h + 9):
        call()
    assert reached.n == 4
    wrong = [dict(offsets=2 * S * h), dict(offsets=S * h + 1), dict(offsets=2 * S * h + 1, device=1)]
    if layout == "paged":
        wrong.append(dict(offsets=2 * S * h + 1, tables=2))
    for kw in wrong:
        for call in calls(**kw):
            with pytest.raises(ValueError):
                call()
    assert reached.n == 4


def test_kv_paged_refuses_tensors_on_two_devices():
    a, b = _Device(torch.int64, 5), _Device(torch.int32, 1, 4)
    b.device = torch.device("cuda:1")
    with pytest.raises(ValueError):
        tri.kv_paged(1, a, 4, b, 16, 4)
