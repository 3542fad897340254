"""Operators around the dual-pool KV cache, as they are measured.

Three families, each reached through the package's public calls:

  rope      rotary positions over several axes (time, height, width) for queries and keys, alone
            (`rope_fwd`) and together with the commit into the pool (`kv_pool_append_rope`)
  i4        the 4-bit KV cache: commit (`kv_pool_append`), decode (`hybrid_decode_fwd`) and chunked
            prefill (`full_prefill_fwd`) over a pool of HSWA_KV_INT4
  mod       attention with capped scores, a distance bias and per-row key ranges (document and prefix
            masks): `swa_prefill_mod_fwd`, `full_prefill_mod_fwd`, `hybrid_decode_mod_fwd`

`own` is set from outside: False computes plain 32-bit forms from elementary torch operations, True
calls the package.
"""
import math

import torch

own = False

DEV = "cuda"
PAGE = 64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token of one request: pure latency
        dict(name="rope_one_token", kind="rope", tokens=1, hq=32, hkv=8, d=128, far=4096, style="half"),
        # one decode step of a 256-request batch, one token and three drafts each, positions up to 1M
        dict(name="rope_step_256x4", kind="rope", tokens=1024, hq=64, hkv=8, d=128, far=1 << 20, style="half"),
        # a 16K-token prompt chunk with images and video, committed to the pages of a full layer
        dict(name="rope_append_16k", kind="rope_append", tokens=16384, hq=32, hkv=8, d=128, far=40000,
             style="half"),
        # a chat request with a short history: latency of a single decode call
        dict(name="i4_decode_short", kind="i4_decode", n=1, lo=613, hi=613, nq=1, hq=32, hkv=8, d=128, window=0),
        # the sliding-window layers of a 256-request step with three drafts per token
        dict(name="i4_decode_ring_256", kind="i4_decode", n=256, lo=1024, hi=262144, nq=4, hq=64, hkv=8, d=128,
             window=128),
        # one long-document request: the split over the keys is all the parallelism there is
        dict(name="i4_decode_256k", kind="i4_decode", n=1, lo=262141, hi=262141, nq=1, hq=64, hkv=8, d=128, window=0),
        # a batch of mixed lengths on a full layer, with drafts
        dict(name="i4_decode_batch", kind="i4_decode", n=64, lo=1024, hi=65536, nq=4, hq=64, hkv=8, d=128,
             window=0),
        # the next 2048-token chunk of a long prompt: commit in 4 bits, then attend over the pages
        dict(name="i4_prefill_chunk", kind="i4_prefill", B=1, prefix=30000, tokens=2048, hq=32, hkv=8, d=128),
        # the 16K sliding-window chunk with capped scores
        dict(name="cap_swa_16k", kind="mod_swa", B=2, tokens=16384, prefix=0, window=4096, hq=32, hkv=8, d=128,
             cap=50.0, bias=False, mask="none"),
        # packed documents of uneven lengths in one row, padded tail
        dict(name="docs_full_8k", kind="mod_full", B=2, tokens=8192, prefix=0, hq=32, hkv=8, d=128, cap=0.0,
             bias=False, mask="docs"),
        # small requests with a bidirectional prefix and a distance bias, odd sizes, resumed mid-prompt
        dict(name="prefix_bias_odd", kind="mod_full", B=3, tokens=999, prefix=333, hq=12, hkv=4, d=64, cap=0.0,
             bias=True, mask="prefix"),
        # a decode step over packed contexts with capped scores (bf16 entries)
        dict(name="cap_decode_48", kind="mod_decode", n=48, lo=512, hi=32768, nq=1, hq=32, hkv=8, d=128, cap=30.0,
             bias=False, mask="docs"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_append", "i4_decode", "i4_decode", "i4_prefill", "mod_swa", "mod_full",
                       "mod_decode"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(kind=kind, hq=hkv * g, hkv=hkv, d=d)
    if kind in ("rope", "rope_append"):
        c.update(tokens=_log(rng, 1, 16384), far=_log(rng, 1000, 1 << 20), style=rng.choice(["half", "pairs"]))
    elif kind in ("i4_decode", "mod_decode"):
        nq = rng.choice([1, 1, 2, 4])
        n = _log(rng, 1, 48)
        c.update(n=n, lo=rng.randint(1, 700), hi=_log(rng, 800, min(200000, 800000 // n + 1000)), nq=nq)
        if kind == "i4_decode":
            c.update(window=rng.choice([0, 0, 0, 100, 128, 500]))
        else:
            c.update(cap=rng.choice([0.0, 20.0, 50.0]), bias=rng.random() < 0.5,
                     mask=rng.choice(["none", "docs"]))
    else:
        b = rng.choice([1, 1, 2, 3])
        c.update(B=b, tokens=_log(rng, 1, 6144 // b), prefix=rng.choice([0, _log(rng, 1, 5000)]))
        if kind == "mod_swa":
            c.update(window=_log(rng, 2, 4500))
        if kind in ("mod_swa", "mod_full"):
            c.update(cap=rng.choice([0.0, 20.0, 50.0]), bias=rng.random() < 0.5,
                     mask=rng.choice(["none", "docs", "prefix"]))
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, s=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * s).to(torch.bfloat16)


def _keys(g, n, hkv, d):
    """Keys with a per-channel mean, as projections with a bias give them, and zero-mean values."""
    mean = torch.randn(hkv, d, generator=g, device=DEV) * 0.5
    k = (torch.randn(n, hkv, d, generator=g, device=DEV) + mean).to(torch.bfloat16)
    return k, _randn(g, n, hkv, d)


def _context_lens(case, seed):
    if case["lo"] == case["hi"]:
        return [case["lo"]] * case["n"]
    g = torch.Generator()
    g.manual_seed(seed + 17)
    u = torch.rand(case["n"], generator=g, dtype=torch.float64)
    return [int(math.exp(math.log(case["lo"]) + float(x) * (math.log(case["hi"]) - math.log(case["lo"]))))
            for x in u]


def _table(seed, rows, per_row, total):
    g = torch.Generator()
    g.manual_seed(seed + 29)
    perm = torch.randperm(total, generator=g)[: rows * per_row]
    return perm.view(rows, per_row).to(torch.int32).to(DEV)


def _rope_plan(case):
    """Frequencies of base 10000 over the whole head, the first half of the pairs split 1:1 between
    height and width, the rest reading time (a text token has the same position on every axis)."""
    half = case["d"] // 2
    inv = [10000.0 ** (-2.0 * i / case["d"]) for i in range(half)]
    axis = [1 + (i % 2) if i < half // 2 else 0 for i in range(half)]
    return inv, axis


def _rope_positions(case, g):
    """Runs of text interleaved with frames of a 24 x 40 patch grid; positions run up to `far`."""
    n = case["tokens"]
    i = torch.arange(n, device=DEV)
    patch = (i // 700) % 2 == 1
    base = int(torch.randint(0, max(1, case["far"]), (1,), generator=g, device=DEV))
    t = torch.where(patch, base + i - (i % 960), base + i)
    h = torch.where(patch, t + (i % 960) // 40, t)
    w = torch.where(patch, t + i % 40, t)
    return torch.stack([t, h, w]).to(torch.int64).contiguous()


def _documents(n, seed, mean):
    """Start of the document of each of n positions: documents of uneven lengths."""
    g = torch.Generator()
    g.manual_seed(seed + 41)
    start = torch.zeros(n, dtype=torch.int64)
    at = 0
    while at < n:
        size = max(1, int(-mean * math.log(1.0 - float(torch.rand(1, generator=g, dtype=torch.float64)))))
        start[at: at + size] = at
        at += size
    return start


def _ranges(case, seed):
    """key_begin and key_end (each [B][tokens] or None) of a prefill case."""
    b, n, p = case["B"], case["tokens"], case["prefix"]
    if case["mask"] == "none":
        return None, None
    pos = torch.arange(p, p + n)
    begins, ends = [], []
    for r in range(b):
        if case["mask"] == "docs":
            begin = _documents(p + n, seed + r, max(2.0, (p + n) / 6))[p:]
            end = pos + 1
            if n > 20:  # padding behind the last token of a row: nothing to attend
                pad = n // 16 + r
                end[n - pad:] = 0
        else:
            begin = torch.zeros(n, dtype=torch.int64)
            end = torch.maximum(pos + 1, torch.full_like(pos, p + (n * (r + 1)) // (b + 2)))
        begins.append(begin)
        ends.append(end)
    begin, end = torch.stack(begins).to(DEV), torch.stack(ends).to(DEV)
    return (begin, end) if case["mask"] == "docs" else (None, end)


def _slopes(case):
    if not case.get("bias"):
        return None
    h = case["hq"]
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], dtype=torch.float32, device=DEV)


def _inputs(case, seed):
    """The tensors a user's program has in hand, the same for both forms."""
    g = _gen(seed)
    kind, hq, hkv, d = case["kind"], case["hq"], case["hkv"], case["d"]
    s = {}
    if kind in ("rope", "rope_append"):
        n = case["tokens"]
        s["pos"] = _rope_positions(case, g)
        s["q"] = _randn(g, 1, n, hq, d)
        s["k"], s["v"] = _randn(g, 1, n, hkv, d), _randn(g, 1, n, hkv, d)
        if kind == "rope_append":
            pages = -(-n // PAGE)
            s["table"] = _table(seed, 1, pages, pages)
        return s
    if kind in ("i4_decode", "mod_decode"):
        lens = _context_lens(case, seed)
        n, nq, w = len(lens), case["nq"], case.get("window", 0)
        s["lens"] = lens
        s["first"] = [max(0, length - w) if w else 0 for length in lens]
        s["kv"] = [_keys(g, length - f, hkv, d) for length, f in zip(lens, s["first"])]
        s["q"] = _randn(g, n, nq, hq, d, s=1.5)
        s["k_new"], s["v_new"] = _randn(g, n, nq, hkv, d), _randn(g, n, nq, hkv, d)
        s["ctx"] = torch.tensor(lens, dtype=torch.int64, device=DEV)
        if not w:
            per = -(-max(lens) // PAGE) if max(lens) else 1
            used = [-(-length // PAGE) for length in lens]
            g2 = torch.Generator()
            g2.manual_seed(seed + 29)
            perm = torch.randperm(max(1, sum(used)), generator=g2).to(torch.int32)
            table = torch.zeros(n, per, dtype=torch.int32)
            at = 0
            for b, u in enumerate(used):
                table[b, :u] = perm[at: at + u]
                at += u
            s["table"], s["pages"] = table.to(DEV), max(1, sum(used))
        if kind == "mod_decode" and case["mask"] == "docs":
            begin = torch.stack([_documents(length + nq, seed + b, max(2.0, length * 1.5))[length:]
                                 for b, length in enumerate(lens)])
            s["begin"] = begin.to(DEV).contiguous()
        return s
    b, n, p = case["B"], case["tokens"], case["prefix"]
    kv = [_keys(g, p + n, hkv, d) for _ in range(b)]
    s["k"], s["v"] = torch.stack([x[0] for x in kv]), torch.stack([x[1] for x in kv])  # [B][p + n]
    s["q"] = _randn(g, b, n, hq, d, s=1.5)
    s["k_chunk"], s["v_chunk"] = s["k"][:, p:].contiguous(), s["v"][:, p:].contiguous()
    s["start"] = torch.full((b,), p, dtype=torch.int64, device=DEV)
    if kind != "mod_swa":
        per = -(-(p + n) // PAGE)
        s["table"], s["pages"] = _table(seed, b, per, b * per), b * per
    if kind != "i4_prefill":
        s["begin"], s["end"] = _ranges(case, seed)
    return s


# ------------------------------------------------------------------ the package's calls

def _own_state(case, s):
    import hybrid_sliding_window_swa_b200 as hs
    kind, hkv, d = case["kind"], case["hkv"], case["d"]
    if kind in ("rope", "rope_append"):
        inv, axis = _rope_plan(case)
        s["rope"] = hs.RopeDesc(inv_freq=inv, axis=axis, n_axes=3, interleaved=case["style"] == "pairs")
        if kind == "rope_append":
            s["pool"] = hs.kv_pool_create(hs.PoolDesc(
                n_swa_layers=0, n_full_layers=1, window=1, n_kv_heads=hkv, head_dim=d, max_seqs=1,
                pages_per_full_layer=s["table"].shape[1]))
            s["pool"].data.zero_()
            s["start"] = torch.zeros(1, dtype=torch.int64, device=DEV)
        return s
    window = case.get("window", 0)
    seqs = len(s["lens"]) if "lens" in s else case["B"]
    swa = kind == "mod_swa" or window > 0
    s["pool"] = pool = hs.kv_pool_create(hs.PoolDesc(
        n_swa_layers=1 if swa else 0, n_full_layers=0 if swa else 1, window=window if swa else 1, n_kv_heads=hkv,
        head_dim=d, max_seqs=seqs, pages_per_full_layer=0 if swa else s["pages"],
        kv_format=hs.HSWA_KV_INT4 if kind.startswith("i4") else hs.HSWA_KV_BF16))
    s["ids"] = torch.arange(seqs, dtype=torch.int32, device=DEV)

    def commit(b, k, v, first):
        if k.shape[0] == 0:
            return
        hs.kv_pool_append(pool, 0, k[None].contiguous(), v[None].contiguous(),
                          torch.tensor([first], dtype=torch.int64, device=DEV),
                          seq_ids=s["ids"][b:b + 1] if swa else None,
                          page_table=None if swa else s["table"][b:b + 1].contiguous())

    if "kv" in s:
        for b, (k, v) in enumerate(s["kv"]):
            commit(b, k, v, s["first"][b])
        s["longest"] = max(s["lens"])
        s["ws"] = torch.empty(hs.hybrid_decode_workspace_size(pool, seqs, case["nq"], case["hq"], s["longest"]),
                              dtype=torch.uint8, device=DEV)
    else:
        p = case["prefix"]
        lo = max(0, p - window) if swa else 0
        hi = p if (swa or kind == "i4_prefill") else p + case["tokens"]
        for b in range(seqs):
            commit(b, s["k"][b, lo:hi], s["v"][b, lo:hi], lo)
    if kind.startswith("mod"):
        s["mod"] = hs.ScoreMod(softcap=case["cap"], dist_slope=_slopes(case), key_begin=s.get("begin"),
                               key_end=s.get("end"))
        if kind != "mod_decode":
            s["ws"] = torch.empty(hs.prefill_mod_workspace_size(pool, seqs, case["tokens"]), dtype=torch.uint8,
                                  device=DEV)
    for name in ("kv", "k", "v"):  # the pool holds them now
        s.pop(name, None)
    return s


def _own_run(case, s):
    import hybrid_sliding_window_swa_b200 as hs
    kind = case["kind"]
    if kind == "rope":
        return hs.rope_fwd(s["rope"], s["q"], s["k"], s["pos"])
    if kind == "rope_append":
        q, k = hs.kv_pool_append_rope(s["pool"], 0, s["rope"], s["q"], s["k"], s["v"], s["pos"], s["start"],
                                      page_table=s["table"])
        pages = s["pool"].pages
        return q, k, pages[0, 0], pages[1, 0]
    if kind == "i4_decode":
        ring = case["window"] > 0
        return hs.hybrid_decode_fwd(s["pool"], 0, s["q"], s["k_new"], s["v_new"], s["ctx"], s["longest"], s["ws"],
                                    seq_ids=s["ids"] if ring else None, page_table=None if ring else s["table"])
    if kind == "mod_decode":
        return hs.hybrid_decode_mod_fwd(s["pool"], 0, s["q"], s["k_new"], s["v_new"], s["ctx"], s["longest"],
                                        s["mod"], s["ws"], page_table=s["table"])
    if kind == "i4_prefill":
        hs.kv_pool_append(s["pool"], 0, s["k_chunk"], s["v_chunk"], s["start"], page_table=s["table"])
        return hs.full_prefill_fwd(s["pool"], 0, s["q"], s["table"], start_pos=s["start"])
    if kind == "mod_full":
        return hs.full_prefill_mod_fwd(s["pool"], 0, s["q"], s["table"], s["mod"], s["ws"], start_pos=s["start"])
    return hs.swa_prefill_mod_fwd(s["pool"], 0, s["q"], s["k_chunk"], s["v_chunk"], s["mod"], s["ws"],
                                  start_pos=s["start"], seq_ids=s["ids"])


# ------------------------------------------------------------------ the plain forms

def _quantize(x):
    """Codes 0 .. 15 (uint8), step and minimum (bf16) of each row of x [..., d] bf16."""
    f = x.float()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    step = ((hi - lo) * (1.0 / 15.0)).to(torch.bfloat16)
    inv = torch.where(step > 0, 1.0 / step.float(), torch.zeros_like(lo))
    codes = torch.round((f - lo) * inv).clamp_(0, 15)
    return codes.to(torch.uint8), step, lo.to(torch.bfloat16)


def _value(codes, step, low):
    return codes.float() * step.float() + low.float()


def _attend(q, k, v, lo, hi, q_pos, k_pos0, cap=0.0, slope=None):
    """q [n, Hq, d], k and v [m, Hkv, d] at positions k_pos0 .. ; row i sees positions [lo[i], hi[i])."""
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    g = hq // hkv
    out = torch.zeros(n, hq, d, dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(d)
    kt, vt = k.float().permute(1, 2, 0).contiguous(), v.float().permute(1, 0, 2).contiguous()
    rows = max(1, min(512, 200_000_000 // (hq * max(1, m))))
    los = torch.clamp(lo - k_pos0, min=0)
    his = torch.clamp(hi - k_pos0, max=m)
    n_blocks = -(-n // rows)
    pad = n_blocks * rows - n
    firsts = torch.nn.functional.pad(los, (0, pad), value=m).view(n_blocks, rows).amin(1).tolist()
    lasts = torch.nn.functional.pad(his, (0, pad), value=0).view(n_blocks, rows).amax(1).tolist()
    for blk in range(n_blocks):
        r0, r1 = blk * rows, min(n, (blk + 1) * rows)
        a, b = firsts[blk], lasts[blk]
        if b <= a:
            continue
        qb = (q[r0:r1].float() * scale).view(r1 - r0, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
        x = torch.bmm(qb, kt[:, :, a:b]).view(hq, r1 - r0, b - a)
        if cap:
            x = cap * torch.tanh(x / cap)
        at = torch.arange(a, b, device=q.device)
        if slope is not None:
            x = x - slope.view(-1, 1, 1) * (q_pos[r0:r1, None] - (at + k_pos0)[None]).abs().float()
        see = (at[None] >= los[r0:r1, None]) & (at[None] < his[r0:r1, None])
        x = x.masked_fill(~see, float("-inf"))
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
        total = e.sum(-1, keepdim=True)
        y = torch.bmm(e.view(hkv, -1, b - a), vt[:, a:b]).view(hq, r1 - r0, d)
        y = torch.where(total > 0, y / total, torch.zeros_like(y))
        out[r0:r1] = y.permute(1, 0, 2)
    return out


def _plain_state(case, s):
    if case["kind"] in ("rope", "rope_append"):
        inv, axis = _rope_plan(case)
        s["inv"] = torch.tensor(inv, dtype=torch.float64, device=DEV)
        s["axis"] = torch.tensor(axis, device=DEV)
        if case["kind"] == "rope_append":
            shape = (s["table"].shape[1], case["hkv"], PAGE, case["d"])
            s["pages_k"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
            s["pages_v"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    elif case["kind"] == "i4_decode":  # the cache already holds codes
        s["cache"] = [(_quantize(k), _quantize(v)) for k, v in s.pop("kv")]
    elif case["kind"] == "i4_prefill":
        p = case["prefix"]
        s["cache"] = [(_quantize(s["k"][b, :p]), _quantize(s["v"][b, :p])) for b in range(case["B"])]
        s.pop("k"), s.pop("v")
    return s


def _rotate(x, cos, sin, style):
    """x [1, n, heads, d]; cos and sin [n, d / 2]."""
    f = x.float()
    c, s = cos[None, :, None], sin[None, :, None]
    if style == "half":
        a, b = f.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16)
    a, b = f[..., 0::2], f[..., 1::2]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2).to(torch.bfloat16)


def _plain_run(case, s):
    kind = case["kind"]
    if kind in ("rope", "rope_append"):
        angle = s["pos"][s["axis"]].t().double() * s["inv"]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q, k = _rotate(s["q"], cos, sin, case["style"]), _rotate(s["k"], cos, sin, case["style"])
        if kind == "rope":
            return q, k
        at = torch.arange(case["tokens"], device=DEV)
        page = s["table"][0].long()[at // PAGE]
        s["pages_k"][page, :, at % PAGE] = k[0]
        s["pages_v"][page, :, at % PAGE] = s["v"][0]
        return q, k, s["pages_k"], s["pages_v"]
    if kind in ("i4_decode", "mod_decode"):
        outs = []
        w, nq = case.get("window", 0), case["nq"]
        slope = _slopes(case)
        for b, length in enumerate(s["lens"]):
            first = s["first"][b]
            if kind == "i4_decode":
                (ck, cv), nk, nv = s["cache"][b], _quantize(s["k_new"][b]), _quantize(s["v_new"][b])
                k = torch.cat([_value(*ck), _value(*nk)])
                v = torch.cat([_value(*cv), _value(*nv)])
            else:
                k = torch.cat([s["kv"][b][0], s["k_new"][b]]).float()
                v = torch.cat([s["kv"][b][1], s["v_new"][b]]).float()
            q_pos = torch.arange(length, length + nq, device=DEV)
            lo = torch.clamp(q_pos - w + 1, min=0) if w else torch.zeros_like(q_pos)
            if s.get("begin") is not None:
                lo = torch.maximum(lo, s["begin"][b])
            outs.append(_attend(s["q"][b], k, v, lo, q_pos + 1, q_pos, first, case.get("cap", 0.0), slope))
        return torch.stack(outs).to(torch.bfloat16)
    p, n, outs = case["prefix"], case["tokens"], []
    slope = _slopes(case)
    q_pos = torch.arange(p, p + n, device=DEV)
    for b in range(case["B"]):
        lo, hi = torch.zeros_like(q_pos), q_pos + 1
        if kind == "i4_prefill":
            # entries are read as bf16 values by the prefill
            nk, nv = _quantize(s["k_chunk"][b]), _quantize(s["v_chunk"][b])
            ck, cv = s["cache"][b]
            k = torch.cat([_value(*ck), _value(*nk)]).to(torch.bfloat16)
            v = torch.cat([_value(*cv), _value(*nv)]).to(torch.bfloat16)
        else:
            k, v = s["k"][b], s["v"][b]
            if s["end"] is not None:
                hi = torch.clamp(s["end"][b], max=p + n)
            if s["begin"] is not None:
                lo = torch.maximum(lo, s["begin"][b])
            if kind == "mod_swa":
                lo = torch.maximum(lo, q_pos - case["window"] + 1)
                hi = torch.minimum(hi, q_pos + case["window"])
        outs.append(_attend(s["q"][b], k, v, lo, hi, q_pos, 0, case.get("cap", 0.0), slope))
    return torch.stack(outs).to(torch.bfloat16)


# ------------------------------------------------------------------ interface

def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    return _own_state(case, s) if own else _plain_state(case, s)


def run(state):
    return _own_run(state["case"], state) if own else _plain_run(state["case"], state)


def _pairs(case, seed=0):
    """Visible (query, key) pairs of one query head."""
    if case["kind"] in ("i4_decode", "mod_decode"):
        nq, total = case["nq"], 0
        for b, length in enumerate(_context_lens(case, seed)):
            w = case.get("window", 0)
            begin = [0] * nq
            if case.get("mask") == "docs":
                begin = _documents(length + nq, seed + b, max(2.0, length * 1.5))[length:].tolist()
            for t in range(nq):
                lo = max(length + t - w + 1 if w else 0, begin[t], 0)
                total += length + t + 1 - lo
        return total
    p, n = case["prefix"], case["tokens"]
    pos = torch.arange(p, p + n, device=DEV)
    total = 0
    begin, end = _ranges(case, seed) if case["kind"] != "i4_prefill" else (None, None)
    for b in range(case["B"]):
        lo, hi = torch.zeros_like(pos), pos + 1
        if end is not None:
            hi = torch.clamp(end[b], max=p + n)
        if begin is not None:
            lo = torch.maximum(lo, begin[b])
        if case["kind"] == "mod_swa":
            lo, hi = torch.maximum(lo, pos - case["window"] + 1), torch.minimum(hi, pos + case["window"])
        total += int(torch.clamp(hi - lo, min=0).sum())
    return total


def work(case):
    kind, hq, hkv, d = case["kind"], case["hq"], case["hkv"], case["d"]
    if kind in ("rope", "rope_append"):
        n = case["tokens"]
        if kind == "rope":
            return {"bytes": 2 * n * (hq + hkv) * d * 2 + 24 * n, "flops": 3 * n * (hq + hkv) * d}
        # q, k, v read; q, k and both pages written
        return {"bytes": (2 * hq + 5 * hkv) * n * d * 2 + 24 * n, "flops": 3 * n * (hq + hkv) * d}
    flops = 4 * d * hq * _pairs(case)
    i4 = d // 2 + 4
    if kind in ("i4_decode", "mod_decode"):
        lens = _context_lens(case, 0)
        nq, w = case["nq"], case.get("window", 0)
        entry = i4 if kind == "i4_decode" else 2 * d
        seen = 0
        for b, length in enumerate(lens):
            lo = max(0, length - w + 1) if w else 0
            if case.get("mask") == "docs":
                lo = int(_documents(length + nq, b, max(2.0, length * 1.5))[length:].min())
            seen += max(0, length - lo)
        return {"bytes": 2 * seen * hkv * entry + len(lens) * nq * (2 * hq + 2 * hkv) * d * 2, "flops": flops}
    n, p, b = case["tokens"], case["prefix"], case["B"]
    q_o = 2 * b * n * hq * d * 2
    if kind == "i4_prefill":  # the chunk in, its codes out, every entry read once
        kv = 2 * b * n * hkv * (2 * d + i4) + 2 * b * (p + n) * hkv * i4
    elif kind == "mod_swa":
        kv = 2 * b * (n + min(p, case["window"])) * hkv * d * 2
    else:
        kv = 2 * b * (p + n) * hkv * d * 2
    return {"bytes": q_o + kv, "flops": flops}


# ------------------------------------------------------------------ 64-bit values

def _exact_entry(x):
    """What a 4-bit row stands for, in 64 bits: the row's step is its range over 15 as a bf16."""
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    step = ((high.float() - low.float()) * torch.tensor(1.0 / 15.0, device=x.device)).to(torch.bfloat16)
    inv = torch.zeros_like(step, dtype=torch.float32)
    inv[step > 0] = torch.reciprocal(step.float()[step > 0])
    code = torch.clamp(torch.round((x.float() - low.float()) * inv), 0.0, 15.0)
    return code.double() * step.double() + low.double()


def _exact_attention(q, k, v, visible, bias, cap):
    """q [n, Hq, d]; k, v [m, Hkv, d] double; visible(rows) -> [rows, m] bool; one head at a time."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    res = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    step = max(1, 60_000_000 // max(1, k.shape[0]))
    for r0 in range(0, n, step):
        rows = torch.arange(r0, min(n, r0 + step), device=q.device)
        see = visible(rows)
        cols = torch.nonzero(see.any(0)).flatten()
        if cols.numel() == 0:
            continue
        c0, c1 = int(cols[0]), int(cols[-1]) + 1
        see = see[:, c0:c1]
        for h in range(hq):
            z = q[rows, h].double() @ k[c0:c1, h // group].double().T / math.sqrt(d)
            if cap:
                z = torch.tanh(z / cap) * cap
            if bias is not None:
                z = z + bias(h, rows, c0, c1)
            z = torch.where(see, z, -math.inf)
            w = torch.softmax(z, -1)
            w = torch.where(see.any(-1, keepdim=True), w, 0.0)
            res[rows, h] = w @ v[c0:c1, h // group].double()
    return res


def exact(case, seed):
    kind, hq, d = case["kind"], case["hq"], case["d"]
    if kind not in ("rope", "rope_append") and work(case)["flops"] > 2.5e12:
        return None
    s = _inputs(case, seed)
    if kind in ("rope", "rope_append"):
        inv, axis = _rope_plan(case)
        turn = torch.stack([s["pos"][a].double() * f for f, a in zip(inv, axis)], -1)  # [n, d / 2]
        rot = torch.polar(torch.ones_like(turn), turn)[None, :, None]

        def turned(x):
            y = x.double()
            if case["style"] == "pairs":
                z = torch.view_as_complex(y.reshape(*y.shape[:-1], d // 2, 2)) * rot
                return torch.view_as_real(z).reshape(y.shape)
            z = torch.complex(y[..., : d // 2], y[..., d // 2:]) * rot
            return torch.cat([z.real, z.imag], -1)

        q, k = turned(s["q"]), turned(s["k"])
        if kind == "rope":
            return q, k
        n, hkv = case["tokens"], case["hkv"]
        pages = s["table"].shape[1]
        filled = []
        for x in (k[0], s["v"][0].double()):
            flat = torch.zeros(pages * PAGE, hkv, d, dtype=torch.float64, device=DEV)
            flat[:n] = x
            by_page = torch.empty(pages, hkv, PAGE, d, dtype=torch.float64, device=DEV)
            by_page[s["table"][0].long()] = flat.view(pages, PAGE, hkv, d).transpose(1, 2)
            filled.append(by_page)
        return q, k, filled[0], filled[1]
    cap = case.get("cap", 0.0)
    heads = [-(2.0 ** (-8.0 * (i + 1) / hq)) for i in range(hq)] if case.get("bias") else None
    if heads is not None:
        heads = [float(torch.tensor(x, dtype=torch.float32)) for x in heads]
    res = []
    batch = len(s["lens"]) if "lens" in s else case["B"]
    for b in range(batch):
        if "lens" in s:
            first, p, n = s["first"][b], s["lens"][b], case["nq"]
            k = torch.cat([s["kv"][b][0], s["k_new"][b]])
            v = torch.cat([s["kv"][b][1], s["v_new"][b]])
        else:
            first, p, n = 0, case["prefix"], case["tokens"]
            k, v = s["k"][b], s["v"][b]
        if kind.startswith("i4"):
            k, v = _exact_entry(k), _exact_entry(v)
            if kind == "i4_prefill":  # read as bf16 values
                k, v = k.float().to(torch.bfloat16), v.float().to(torch.bfloat16)
        begin = None if s.get("begin") is None else s["begin"][b]
        end = None if s.get("end") is None else s["end"][b]
        w = case.get("window", 0)
        at = torch.arange(first, first + k.shape[0], device=DEV)[None]

        def visible(rows):
            i = (rows + p)[:, None]
            see = at <= i if end is None else at < end[rows][:, None]
            if begin is not None:
                see = see & (at >= begin[rows][:, None])
            if w:
                see = see & ((at - i).abs() < w)
            return see

        def bias(h, rows, c0, c1):
            return heads[h] * (at[:, c0:c1] - (rows + p)[:, None]).abs().double()

        res.append(_exact_attention(s["q"][b], k, v, visible, bias if heads else None, cap))
    return torch.stack(res)
