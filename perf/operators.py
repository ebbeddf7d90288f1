"""The two prompt-side operators of the cache, as measured cases.

``append``: new tokens enter the cache.  Their queries and keys are rotated by
their positions (RoPE), keys, values and positions are written to the cache
slots the tokens take, contiguous or paged, bf16 or fp8 e4m3.

``attend``: causal softmax attention of those tokens' queries over the cache
they were appended to: the last ``n`` of a sequence's ``N`` slots are the new
tokens, and token ``i`` of them sees slots ``0 .. N - n + i``.

``run`` computes them from elementary torch operations, or, where ``own`` is
true, by the package's calls.
"""
import math
import random

import torch

own = False

# Shapes: 32 query / 8 KV heads of dim 128 at theta 1e6 (the Qwen3-8B-shaped cache of
# the synthetic workloads), 64 / 8 (the Qwen3-32B-shaped one), and the variant
# head dims 64 and 256 at theta 1e4, rotate-half and interleaved.


def _case(op, name=None, **kw):
    c = {"op": op, "layout": "paged", "elem": "bf16", "d": 128, "hq": 32, "h": 8, "il": False, "theta": 1e6, "bs": 16,
         "seqs": 1, "new_lo": 1, "new_hi": 1, "old_lo": 0, "old_hi": 0, "pad": 0, "far": 0, "lens_seed": 1}
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of the paged serving batch: 16 sequences, one token each, 2048 kept
        # keys and up to 128 decoded since; latency counts
        _case("append", "append_step_16seq", seqs=16, old_lo=2048, old_hi=2175, far=32768),
        # ragged prompts of a serving batch into 16-token blocks
        _case("append", "append_prompts_paged", seqs=16, new_lo=200, new_hi=2000),
        # the interleaved head-dim-64 variant into an fp8 cache behind a cached prefix, odd
        # lengths, a padded token batch
        _case("append", "append_fp8_d64", seqs=5, new_lo=333, new_hi=1777, old_lo=1, old_hi=999, elem="fp8", d=64, hq=64,
              il=True, theta=1e4, pad=37),
        # a 32K prompt of the 64-query-head shape into a contiguous cache
        _case("append", "append_prompt_32k", layout="contig", new_lo=32768, new_hi=32768, hq=64),
        # one decode step over the compacted paged cache: 16 sequences, one token each
        _case("attend", "attend_step_16seq", seqs=16, old_lo=2047, old_hi=2174),
        # a few tokens per sequence (drafted tokens being checked) over long caches: few
        # rows, long rows
        _case("attend", "attend_draft_long", seqs=4, new_lo=3, new_hi=5, old_lo=20000, old_hi=32763),
        # a 512-token chunk of a prompt behind 32256 cached keys
        _case("attend", "attend_chunk_512", new_lo=512, new_hi=512, old_lo=32256, old_hi=32256),
        # ragged packed prompts, contiguous cache, a padded token batch
        _case("attend", "attend_prompts_ragged", layout="contig", seqs=16, new_lo=100, new_hi=4096, pad=11),
        # a whole 32K prompt: the largest
        _case("attend", "attend_prompt_32k", layout="contig", new_lo=32768, new_hi=32768),
        # prompt chunks over an fp8 paged cache
        _case("attend", "attend_fp8_chunks", seqs=4, new_lo=700, new_hi=1100, old_lo=1000, old_hi=9000, elem="fp8"),
        # head dim 64, every query head with its own KV head's group of 2
        _case("attend", "attend_d64_prompts", seqs=8, new_lo=500, new_hi=3000, d=64, hq=16, il=True, theta=1e4),
        # head dim 256, one KV head shared by 8 query heads
        _case("attend", "attend_d256_prompt", layout="contig", new_lo=5000, new_hi=5000, d=256, hq=16, h=2, theta=1e4),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    most = {o: max(_cost(c) for c in listed() if c["op"] == o) for o in ("append", "attend")}
    while True:
        d = rng.choice([64, 128, 128, 128, 256])
        h = rng.choice([1, 2, 4, 8, 8])
        new = _spread(rng, 1, 16384)
        old = rng.choice([0, _spread(rng, 1, 32768)])
        c = _case(rng.choice(["append", "attend", "attend"]), layout=rng.choice(["paged", "contig"]),
                  elem=rng.choice(["bf16", "bf16", "fp8"]), d=d, h=h, hq=h * rng.choice([1, 2, 3, 4, 8, 8]),
                  il=rng.choice([False, True]), theta=1e6 if d == 128 else 1e4, bs=rng.choice([8, 16, 16, 32, 64]),
                  seqs=_spread(rng, 1, 24), new_lo=max(1, int(new * rng.uniform(0.2, 1.0))), new_hi=new,
                  old_lo=int(old * rng.uniform(0.3, 1.0)), old_hi=old, pad=rng.choice([0, 0, rng.randrange(1, 50)]),
                  far=rng.choice([0, 0, 1 << 20]), lens_seed=rng.randrange(1 << 30))
        new_of, old_of = _lens(c)
        cells = sum(n + o for n, o in zip(new_of, old_of)) * c["h"] * d
        if _cost(c) <= most[c["op"]] / 3 and cells <= 1 << 29:
            return c


def _cost(c):
    w = work(c)
    return w["bytes"] if c["op"] == "append" else w["flops"]


def _lens(c):
    """Per sequence: new tokens, and slots cached before them."""
    r = random.Random(c["lens_seed"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    old = [r.randint(c["old_lo"], c["old_hi"]) for _ in range(c["seqs"])]
    return new, old


def work(case):
    new, old = _lens(case)
    t, d, hq, h = sum(new), case["d"], case["hq"], case["h"]
    e = 2 if case["elem"] == "bf16" else 1
    if case["op"] == "append":
        # queries read and written; keys and values read in bf16, written as the cache holds
        # them; positions read, and written per head.  Six operations per rotated pair.
        return {"bytes": t * (hq * d * 4 + h * (2 * d * 2 + 2 * d * e + 4) + 4), "flops": t * (hq + h) * d * 3}
    pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
    keys = sum(n + o for n, o in zip(new, old))
    return {"bytes": t * hq * (4 * d + 4) + keys * h * 2 * d * e, "flops": 4 * d * hq * pairs}


def _to_elem(x, elem):
    """fp32 values as the cache holds them: bf16, or e4m3 with values beyond +-448 held at the ends."""
    return x.to(torch.bfloat16) if elem == "bf16" else x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _turned(x, pos, il, theta):
    """Pairs of the last dim of x [tokens, heads, d] turned by pos * theta^(-2f/d); angles in 64 bits."""
    d = x.shape[-1]
    w = theta ** (-2.0 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    a = pos.double()[:, None] * w
    c, s = a.cos().to(x.dtype)[:, None], a.sin().to(x.dtype)[:, None]
    re, im = (x[..., 0::2], x[..., 1::2]) if il else (x[..., :d // 2], x[..., d // 2:])
    re, im = re * c - im * s, re * s + im * c
    return torch.stack((re, im), -1).flatten(-2) if il else torch.cat((re, im), -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + case["lens_seed"])
    dev, d, hq, h, bs, S = "cuda", case["d"], case["hq"], case["h"], case["bs"], case["seqs"]
    new, old = _lens(case)
    T, N = sum(new), [n + o for n, o in zip(new, old)]
    randn = lambda *n: torch.randn(*n, generator=g, device=dev)  # noqa: E731
    st = {"case": case, "T": T + case["pad"]}
    # rows (sequence, KV head) end to end; in the paged layout they only give the lengths
    lens = torch.tensor([0] + [n for n in N for _ in range(h)], dtype=torch.int64, device=dev)
    st["row_off"] = lens.cumsum(0)
    st["keys"] = sum(N) * h
    st["tok_off"] = torch.tensor([0] + new, dtype=torch.int64, device=dev).cumsum(0)
    seq = torch.repeat_interleave(torch.arange(S, device=dev), torch.tensor(new, device=dev))
    st["seq"] = seq
    st["new"], st["len"] = torch.tensor(new, device=dev), torch.tensor(N, device=dev)
    first = st["len"] - st["new"]
    place = torch.arange(T, device=dev) - st["tok_off"][seq]
    st["slot"] = first[seq] + place
    st["positions"] = torch.zeros(st["T"], dtype=torch.int32, device=dev)
    st["positions"][:T] = (case["far"] + st["slot"]).int()  # compacted caches hold fewer slots than positions
    shape = (sum(N) * h, d)
    if case["layout"] == "paged":
        need = [(n + bs - 1) // bs for n in N]
        perm = torch.randperm(sum(need), generator=g, device=dev).int()
        st["table"] = torch.full((S, max(need)), -1, dtype=torch.int32, device=dev)
        at = 0
        for s, n in enumerate(need):
            st["table"][s, :n] = perm[at:at + n]
            at += n
        st["blocks"] = sum(need)
        shape = (1, sum(need), bs, h, d)
    # every head's keys (and queries) lie around a centre of its own, as pre-RoPE keys and
    # queries do: noise of 0.3 of the centre's magnitude per pair
    mag = 0.6 * torch.exp(0.5 * randn(hq + h, d // 2)).repeat_interleave(2, -1)
    centre = mag * torch.randn(hq + h, d, generator=g, device=dev) / 2 ** 0.5
    if not case["il"]:
        mag, centre = (torch.cat((x[:, 0::2], x[:, 1::2]), -1) for x in (mag, centre))
    if case["op"] == "append":
        # one row of the query-key-value projection per token
        qkv = torch.cat(((centre + 0.3 * mag * randn(st["T"], hq + h, d)), randn(st["T"], h, d)), 1).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        st["q_out"] = torch.zeros(st["T"], hq, d, dtype=torch.bfloat16, device=dev)
        st["K"], st["V"] = (_to_elem(randn(*shape), case["elem"]) for _ in range(2))
        st["pos"] = torch.zeros(shape[:-1], dtype=torch.int32, device=dev)
        return st
    st["q"] = torch.zeros(st["T"], hq, d, dtype=torch.bfloat16, device=dev)
    q = centre[:hq] + 0.3 * mag[:hq] * randn(T, hq, d)
    st["q"][:T] = _turned(q, st["positions"][:T], case["il"], case["theta"]).to(torch.bfloat16)
    st["K"], st["V"] = (torch.empty(shape, dtype=torch.bfloat16 if case["elem"] == "bf16" else torch.float8_e4m3fn,
                                    device=dev) for _ in range(2))
    st["V"].copy_(_to_elem(randn(*shape), case["elem"]))
    for s, n in enumerate(N):
        j = torch.arange(n, device=dev)
        k = _turned(centre[hq:] + 0.3 * mag[hq:] * randn(n, h, d), case["far"] + j, case["il"], case["theta"])
        _rows(st["K"])[_records(st, torch.full_like(j, s), j)] = _bits(_to_elem(k, case["elem"]))
    st["scale"] = d ** -0.5
    st["out"] = torch.zeros(st["T"], hq, d, dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.zeros(st["T"], hq, device=dev)
    return st


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _rows(x):
    """A cache's records as rows [records, d], fp8 as its bytes."""
    return _bits(x).view(-1, x.shape[-1])


def _records(st, s, j):
    """Record numbers [..., h] of slot j of sequence s."""
    c = st["case"]
    head = torch.arange(c["h"], device=j.device)
    if c["layout"] == "paged":
        blk = st["table"][s, j // c["bs"]].long()
        return (blk * c["bs"] + j % c["bs"])[..., None] * c["h"] + head
    return st["row_off"][s[..., None] * c["h"] + head] + j[..., None]


def run(state):
    if own:
        return _run_own(state)
    return _append(state) if state["case"]["op"] == "append" else _attend(state)


def _append(st):
    c, T = st["case"], st["seq"].shape[0]
    pos = st["positions"][:T]
    turn = lambda x: _turned(x[:T].float(), pos, c["il"], c["theta"])  # noqa: E731
    st["q_out"][:T] = turn(st["q"]).to(torch.bfloat16)
    rec = _records(st, st["seq"], st["slot"])
    _rows(st["K"])[rec] = _bits(_to_elem(turn(st["k"]), c["elem"]))
    _rows(st["V"])[rec] = _bits(_to_elem(st["v"][:T].float(), c["elem"]))
    st["pos"].view(-1)[rec] = pos[:, None].expand_as(rec)
    return {"q": st["q_out"], "K": st["K"], "V": st["V"], "pos": st["pos"]}


def _attend(st):
    """Sequences as a padded batch, as many query tokens at a time as 2 GiB of scores allow."""
    c, T, dev = st["case"], st["seq"].shape[0], st["K"].device
    S, h, hq, d = c["seqs"], c["h"], c["hq"], c["d"]
    new, length = _lens(c)[0], [n + o for n, o in zip(*_lens(c))]
    most, deep = max(new), max(length)
    s, j = torch.arange(S, device=dev)[:, None], torch.arange(deep, device=dev)
    there = j < st["len"][:, None]
    rec = _records(st, s.expand(S, deep), torch.where(there, j, 0)).transpose(1, 2)  # [S, h, deep]
    k, v = (_rows(st[x])[rec].view(st[x].dtype).float() for x in ("K", "V"))
    step = max(1, (1 << 29) // (S * hq * deep))
    for a in range(0, most, step):
        i = torch.arange(a, min(a + step, most), device=dev)
        real = i < st["new"][:, None]  # [S, chunk]
        token = torch.where(real, st["tok_off"][:-1, None] + i, 0)
        seen = (j <= (st["len"] - st["new"])[:, None, None] + i[:, None]) & there[:, None]  # [S, chunk, deep]
        q = st["q"][token].float().view(S, len(i), h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(S, h, -1, d)
        x = (q @ k.transpose(-1, -2)).view(S, h, hq // h, len(i), deep).mul_(st["scale"])
        x.masked_fill_(~seen[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x.sub_(top.clamp_min(torch.finfo(x.dtype).min)).exp_()
        total = x.sum(-1, keepdim=True)
        o = (x.view(S, h, -1, deep) @ v).view(S, h, hq // h, len(i), d) / total.clamp_min(1e-30)
        o = o.permute(0, 3, 1, 2, 4).reshape(S, len(i), hq, d)
        lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(S, len(i), hq)
        st["out"][token[real]] = o[real].to(torch.bfloat16)
        st["lse"][token[real]] = lse[real]
    return {"out": st["out"], "lse": st["lse"]}


def _run_own(st):
    import kv_cache_compression_calib_b200 as tri

    c = st["case"]
    if "kv" not in st:  # what a serving program makes once per batch and keeps
        style = tri.TRI_ROPE_INTERLEAVED if c["il"] else tri.TRI_ROPE_HALF
        st["model"] = tri.model(1, c["hq"], c["h"], c["theta"], c["d"], style)
        elem = tri.elem_type_of(st["K"])
        if c["layout"] == "paged":
            st["kv"] = tri.kv_paged(c["seqs"], st["row_off"], st["keys"], st["table"], c["bs"], st["blocks"], elem)
        else:
            st["kv"] = tri.kv_contig(c["seqs"], st["row_off"], st["keys"], elem)
        if c["op"] == "append":
            st["ws"] = tri.alloc_append_workspace()
            st["tokens"] = tri.tokens(st["k"], st["v"], st["tok_off"], st["positions"], q=st["q"])
        else:
            st["ws"] = tri.alloc_prefill_attention_workspace(st["model"], c["seqs"], st["T"])
    if c["op"] == "append":
        tri.tri_append(st["model"], st["kv"], st["tokens"], tri.TRI_KEYS_POST_ROPE, st["q_out"], st["K"], st["V"], st["pos"],
                       st["ws"])
        return {"q": st["q_out"], "K": st["K"], "V": st["V"], "pos": st["pos"]}
    tri.tri_prefill_attention(st["model"], st["kv"], st["K"], st["V"], st["q"], st["tok_off"], st["scale"], st["out"],
                              st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def exact(case, seed):
    """The definitions in 64 bits, a sequence (and a KV head) at a time."""
    st = prepare(case, seed)
    new, old = _lens(case)
    h, hq, d, G = case["h"], case["hq"], case["d"], case["hq"] // case["h"]
    dev = st["K"].device
    if case["op"] == "append":
        f = torch.arange(d // 2, device=dev, dtype=torch.float64)
        wave = torch.exp(-2.0 / d * math.log(case["theta"]) * f)

        def turn(x, p):  # multiplication of the pairs by e^{i w p}, as complex numbers
            z = x.double().unflatten(-1, (d // 2, 2) if case["il"] else (2, d // 2))
            z = z if case["il"] else z.transpose(-1, -2)
            z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(wave), p.double() * wave)[:, None]
            z = torch.view_as_real(z)
            return (z if case["il"] else z.transpose(-1, -2)).flatten(-2)

        q = st["q_out"].double()
        K, V, P = _rows_double(st["K"]), _rows_double(st["V"]), st["pos"].clone().view(-1)
        held = (lambda x: x) if case["elem"] == "bf16" else (lambda x: x.clamp(-448.0, 448.0))
        t = 0
        for s, (n, o) in enumerate(zip(new, old)):
            p = st["positions"][t:t + n, None]
            q[t:t + n] = turn(st["q"][t:t + n], p)
            for x in range(h):
                slots = torch.arange(o, o + n, device=dev)
                if case["layout"] == "paged":
                    r = (st["table"][s][slots // case["bs"]].long() * case["bs"] + slots % case["bs"]) * h + x
                else:
                    r = sum(a + b for a, b in zip(new[:s], old[:s])) * h + x * (n + o) + slots
                K[r] = held(turn(st["k"][t:t + n, x:x + 1], p)[:, 0])
                V[r] = held(st["v"][t:t + n, x].double())
                P[r] = p[:, 0]
            t += n
        return {"q": q, "K": K.view(st["K"].shape), "V": V.view(st["V"].shape), "pos": P.view(st["pos"].shape)}
    out, lse = st["out"].double(), st["lse"].double()
    t = 0
    for s, (n, o) in enumerate(zip(new, old)):
        slots = torch.arange(n + o, device=dev)
        step = max(1, (1 << 27) // (n + o) // G)
        for x in range(h):
            if case["layout"] == "paged":
                r = (st["table"][s][slots // case["bs"]].long() * case["bs"] + slots % case["bs"]) * h + x
            else:
                r = sum(a + b for a, b in zip(new[:s], old[:s])) * h + x * (n + o) + slots
            k, v = (_rows(st[y])[r].view(st[y].dtype).double() for y in ("K", "V"))
            for a in range(0, n, step):
                b = min(n, a + step)
                qs = st["q"][t + a:t + b, x * G:(x + 1) * G].double()
                seen = o + b  # no later slot is seen by any of these tokens
                w = torch.einsum("igd,jd->igj", qs, k[:seen]) * st["scale"]
                w = torch.where(slots[:seen] > o + torch.arange(a, b, device=dev)[:, None, None], -math.inf, w)
                z = torch.logsumexp(w, -1)
                out[t + a:t + b, x * G:(x + 1) * G] = torch.einsum("igj,jd->igd", torch.exp(w - z[..., None]), v[:seen])
                lse[t + a:t + b, x * G:(x + 1) * G] = z
        t += n
    return {"out": out, "lse": lse}


def _rows_double(x):
    return x.double().view(-1, x.shape[-1]).clone()
