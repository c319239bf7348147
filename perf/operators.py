"""The 8-bit compressed cache and the shared-prefix decode: cases, plain forms and exact values.

Operators (keys "op" of a case):
  write   pooling raw K / V into 8-bit entries (``compress_quant``): every block of a prompt
  append  one serving step's cache update with 8-bit entries (``append_quant``)
  read    8-bit entries of a batch, contiguous or paged, back to bf16 (``read_quant``)
  decode  one query per sequence over its 8-bit entries and raw window (``decode_quant``)
  shared  one query per sequence, the batch's common prefix of entries held once (``decode_shared``)

An 8-bit entry is d e4m3 codes of its key, dv of its value, and two e8m0 scales (powers of two): the
smallest 2^e, -64 <= e <= 120, with max|x| <= 448 * 2^e.  Sizes come from this repository's workloads
(64 heads on one KV head, 512 channels, blocks of 128, 128K and 1M contexts) and its tests.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -64, 120
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # two short prompts entering the cache, the last block of each incomplete: launch-bound
        dict(name="write 2 x 1000", op="write", B=2, T=1000, Hkv=1, d=512, dv=512, blk=128, w=False),
        # the 128K-token prompt of the prefill workload, pooling weights given: a stream over K and V
        dict(name="write 1 x 128K", op="write", B=1, T=131072, Hkv=1, d=512, dv=512, blk=128, w=True),
        # a single user's next token
        dict(name="append 1", op="append", B=1, Hkv=1, d=512, dv=512, blk=128, W=128, paged=False, full=0.0),
        # the serving batch's next token, half of the sequences completing a block, paged
        dict(name="append 64 paged", op="append", B=64, Hkv=1, d=512, dv=512, blk=128, W=128, paged=True, full=0.5),
        # two short sequences' entries back in bf16 (to go on with a prefill)
        dict(name="read 2 x 61", op="read", B=2, n=61, Hkv=1, d=512, dv=512, paged=False),
        # the whole cache of the 64 x 128K workload out of its pages
        dict(name="read 64 x 1023 paged", op="read", B=64, n=1023, Hkv=1, d=512, dv=512, paged=True),
        # one user at a short context: latency
        dict(name="decode 1 x 4K", op="decode", B=1, Hq=64, Hkv=1, lo=4096, hi=4096, blk=128, W=128, paged=False,
             norm=False, gate=False, ring=True, vha=0),
        # the 64 x 128K decode workload
        dict(name="decode 64 x 128K", op="decode", B=64, Hq=64, Hkv=1, lo=131072, hi=131072, blk=128, W=128, paged=False,
             norm=False, gate=False, ring=False, vha=0),
        # the ragged workload: 128 sequences of 4K to 1M tokens, shuffled pages, QK norm and gate
        dict(name="decode 128 x 4K-1M ragged", op="decode", B=128, Hq=64, Hkv=1, lo=4096, hi=1048576, blk=128, W=256,
             paged=True, norm=True, gate=True, ring=False, vha=0),
        # a few users on a short common prompt
        dict(name="shared 4 on 32 entries", op="shared", B=4, Hq=64, Hkv=1, prefix=32, lo=100, hi=700, blk=128, W=128,
             paged=False, norm=False, gate=False, ring=False),
        # the 64-sequence batch on one 128K-token document, each with its own turn of up to 4K tokens
        dict(name="shared 64 on 1023 entries", op="shared", B=64, Hq=64, Hkv=1, prefix=1023, lo=1, hi=4096, blk=128,
             W=128, paged=True, norm=False, gate=True, ring=True),
        # the same batch on a 1M-token document, with QK norm
        dict(name="shared 64 on 8191 entries", op="shared", B=64, Hq=64, Hkv=1, prefix=8191, lo=128, hi=2048, blk=128,
             W=128, paged=False, norm=True, gate=False, ring=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "append", "read", "decode", "decode", "shared", "shared"])
    dims = (64, 128, 256, 512)
    if op == "write":
        B, Hkv = rng.choice([1, 1, 2, 3, 5]), rng.choice([1, 1, 2])
        blk = rng.choice([128, 128, 64, rng.randint(3, 128)])
        return dict(op=op, B=B, T=_log(rng, 2 * blk, 131072 // (B * Hkv)), Hkv=Hkv, d=rng.choice(dims), dv=rng.choice(dims),
                    blk=blk, w=rng.random() < 0.5)
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 256), Hkv=rng.choice([1, 1, 2, 3]), d=rng.choice(dims), dv=rng.choice(dims),
                    blk=rng.choice([128, 128, rng.randint(1, 127)]), W=_log(rng, 1, 512), paged=rng.random() < 0.5,
                    full=rng.choice([0.0, 0.1, 1.0]))
    if op == "read":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, n=_log(rng, 1, 65000 // B), Hkv=rng.choice([1, 1, 2]) if B < 32 else 1, d=rng.choice(dims),
                    dv=rng.choice(dims), paged=rng.random() < 0.5)
    Hq, Hkv = rng.choice([(64, 1), (64, 1), (32, 1), (16, 2), (64, 4)])
    if op == "decode":
        if rng.random() < 0.25:
            Hq, Hkv = rng.choice([(40, 1), (12, 1), (9, 3)])       # groups of any size up to 64
        B = _log(rng, 1, 160)
        hi = _log(rng, 200, min(1 << 20, (1 << 25) // (B * Hkv)))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi,
                    blk=rng.choice([128, 128, 64, 100]), W=rng.choice([128, 128, 256, rng.randint(1, 300)]),
                    paged=rng.random() < 0.5, norm=rng.random() < 0.4, gate=rng.random() < 0.4, ring=rng.random() < 0.5,
                    vha=rng.choice([0, 4]) if Hkv == 1 else 0)
    B = _log(rng, 2, 64)
    hi = _log(rng, 2, 4000)
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, prefix=_log(rng, 8, 8191 // Hkv), lo=max(1, rng.choice([1, hi // 2, hi])), hi=hi,
                blk=rng.choice([128, 128, 64]), W=rng.choice([128, 128, 256, rng.randint(1, 300)]), paged=rng.random() < 0.5,
                norm=rng.random() < 0.4, gate=rng.random() < 0.4, ring=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _scale_exp(amax):
    """The exponent e of an entry's scale: the smallest with amax <= 448 * 2^e, in [-64, 120]."""
    f, x = torch.frexp(amax)                                  # amax = f * 2^x, f in [0.5, 1) (0 for 0)
    e = torch.where(f <= 0.875, x - 9, x - 8)                 # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)


def _quantise(x):
    """(e4m3 codes, e8m0 scales of the last axis) of fp32 or fp64 entries."""
    e = _scale_exp(x.abs().amax(-1))
    codes = torch.ldexp(x, -e[..., None]).to(torch.float32).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _exact_e4m3(x):
    """fp64 values rounded to e4m3 (nearest, ties to even) without leaving fp64; |x| <= 448."""
    _, p = torch.frexp(x)                                     # |x| in [2^(p-1), 2^p)
    ulp = torch.clamp(p - 1, min=-6) - 3                      # 3 mantissa bits, smallest normal 2^-6
    return torch.ldexp(torch.round(torch.ldexp(x, -ulp)), ulp)


def _values(codes, sc):
    return codes.float() * sc.float()[..., None]


def _rows(g, dev, *shape):
    """Entries as a pooled cache holds them: channels of spread about 0.5, one row in a hundred 8 times
    larger."""
    x = torch.randn(shape, generator=g, device=dev) * 0.5
    big = torch.rand(shape[:-1] + (1,), generator=g, device=dev) < 0.01
    return torch.where(big, x * 8, x)


def _lengths(case, seed):
    gen = torch.Generator().manual_seed(seed)
    L = torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=gen)
    L[0] = case["hi"]
    return L


def _pages(g, dev, need, page=64):
    """A page table of shuffled pages for sequences that hold `need` (list) entries, and the pool's page count."""
    counts = [max(1, -(-n // page)) for n in need]
    total = sum(counts)
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    cnt = torch.tensor(counts, device=dev)
    first = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(max(counts), device=dev)
    at = first[:, None] + torch.minimum(col[None], cnt[:, None] - 1)
    return order[at].contiguous(), total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    s = dict(case)
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    if op == "write":
        s["k"] = randn(B, case["T"], Hkv, case["d"]).to(torch.bfloat16)
        s["v"] = randn(B, case["T"], Hkv, case["dv"]).to(torch.bfloat16)
        s["pw"] = randn(B, case["T"]) * 0.5 if case["w"] else None
        return s
    if op == "append":
        d, dv, blk, W = case["d"], case["dv"], case["blk"], case["W"]
        Nmax = 128
        gen = torch.Generator().manual_seed(seed)
        L = torch.randint(1, Nmax * blk, (B,), generator=gen)
        done = torch.rand(B, generator=gen) < case["full"]
        L = torch.where(done, (L // blk + 1) * blk, L)
        s["seqlens"] = L.to(torch.int32).to(dev)
        s["k_new"], s["v_new"] = randn(B, Hkv, d).to(torch.bfloat16), randn(B, Hkv, dv).to(torch.bfloat16)
        s["w_new"] = randn(B) * 0.5
        s["kw"], s["vw"] = randn(B, W, Hkv, d).to(torch.bfloat16), randn(B, W, Hkv, dv).to(torch.bfloat16)
        s["table"], shape = None, (B, Nmax)
        if case["paged"]:
            s["table"], total = _pages(g, dev, [Nmax] * B)
            shape = (total, 64)
        s["kc"], ks = _quantise(randn(*shape, Hkv, d))
        s["vc"], vs = _quantise(randn(*shape, Hkv, dv))
        s["sc"] = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)], -1).view(torch.float8_e8m0fnu)
        # the pooling state of the block's earlier tokens: largest weight, sum, accumulators
        n = ((L - 1) % blk).to(dev).float()[:, None].expand(B, Hkv)
        st = torch.zeros(B, Hkv, 4 + d + dv, device=dev)
        st[..., 0] = torch.where(n > 0, torch.rand(B, Hkv, generator=g, device=dev), torch.zeros_like(n))
        st[..., 1] = n * 0.7
        st[..., 4:] = randn(B, Hkv, d + dv) * n.sqrt()[..., None] * 0.7
        s["state"] = st
        return s
    if op == "read":
        d, dv, n = case["d"], case["dv"], case["n"]
        gen = torch.Generator().manual_seed(seed)
        cnt = torch.randint(max(1, n // 2), n + 1, (B,), generator=gen)
        cnt[0] = n
        s["counts"] = cnt.to(torch.int32).to(dev)
        s["table"], shape = None, (B, n)
        if case["paged"]:
            s["table"], total = _pages(g, dev, [n] * B)
            shape = (total, 64)
        s["kc"], ks = _quantise(_rows(g, dev, *shape, Hkv, d))
        s["vc"], vs = _quantise(_rows(g, dev, *shape, Hkv, dv))
        s["sc"] = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)], -1).view(torch.float8_e8m0fnu)
        s["k_out"] = torch.zeros(B, n, Hkv, d, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros(B, n, Hkv, dv, dtype=torch.bfloat16, device=dev)
        return s
    d, Hq, W, blk = 512, case["Hq"], case["W"], case["blk"]
    skip = case["prefix"] if op == "shared" else 0
    L = _lengths(case, seed) + skip * blk
    nc = torch.clamp((L - W) // blk, min=0)
    need = torch.clamp(nc - skip, min=0).tolist()
    s["scale"] = d ** -0.5
    s["seqlens"] = L.to(torch.int32).to(dev)
    s["q"] = randn(B, Hq, d).to(torch.bfloat16)
    s["kw"], s["vw"] = randn(B, W, Hkv, d).to(torch.bfloat16), randn(B, W, Hkv, d).to(torch.bfloat16)
    s["table"], shape = None, (B, max(1, max(need)))
    if case["paged"]:
        s["table"], total = _pages(g, dev, need)
        shape = (total, 64)
    kc, vc = _rows(g, dev, *shape, Hkv, d), _rows(g, dev, *shape, Hkv, d)
    if op == "decode":
        s["kc"], ks = _quantise(kc)
        s["vc"], vs = _quantise(vc)
        s["sc"] = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)], -1).view(torch.float8_e8m0fnu)
    else:
        s["kc"], s["vc"] = kc.to(torch.bfloat16), vc.to(torch.bfloat16)
        s["kp"] = _rows(g, dev, skip, Hkv, d).to(torch.bfloat16)
        s["vp"] = _rows(g, dev, skip, Hkv, d).to(torch.bfloat16)
    del kc, vc
    s["gq"] = torch.rand(d, generator=g, device=dev) + 0.5 if case["norm"] else None
    s["gk"] = torch.rand(d, generator=g, device=dev) + 0.5 if case["norm"] else None
    s["gates"] = randn(B, Hq, d).to(torch.bfloat16) if case["gate"] else None
    r = case.get("vha", 0)
    s["U"], s["V"] = (randn(Hq, r) * 0.1, randn(Hq, r) * 0.1) if r else (None, None)
    return s


# ---------------------------------------------------------------- plain forms

def _pool(s):
    B, T, Hkv, blk = s["B"], s["T"], s["Hkv"], s["blk"]
    n = T // blk
    w = s["pw"][:, :n * blk].view(B, n, blk) if s["pw"] is not None else torch.zeros(B, n, blk, device=s["k"].device)
    a = torch.exp(w - w.amax(-1, keepdim=True))
    a = (a / a.sum(-1, keepdim=True))[..., None, None]
    mean = lambda x: (x[:, :n * blk].float().view(B, n, blk, Hkv, -1) * a).sum(2)  # noqa: E731
    return mean(s["k"]), mean(s["v"])


def _write(s):
    k, v = _pool(s)
    kc, ks = _quantise(k)
    vc, vs = _quantise(v)
    sc = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)], -1).view(torch.float8_e8m0fnu)
    return kc, vc, sc


def _append(s):
    d, blk, W, B, Hkv = s["d"], s["blk"], s["W"], s["B"], s["Hkv"]
    pos = s["seqlens"].long() - 1
    row = torch.arange(B, device=pos.device)
    s["kw"][row, pos % W] = s["k_new"]
    s["vw"][row, pos % W] = s["v_new"]
    st = s["state"].clone()
    m0, n0 = st[..., 0], st[..., 1]
    w = s["w_new"][:, None].expand(B, Hkv)
    m1 = torch.where(n0 > 0, torch.maximum(m0, w), w)
    a, e = torch.where(n0 > 0, torch.exp(m0 - m1), torch.zeros_like(w)), torch.exp(w - m1)
    n1 = n0 * a + e
    x = torch.cat([s["k_new"], s["v_new"]], -1).float()
    acc = st[..., 4:] * a[..., None] + x * e[..., None]
    done = (pos + 1) % blk == 0
    mean = acc / n1[..., None]
    kc, ks = _quantise(mean[..., :d])
    vc, vs = _quantise(mean[..., d:])
    sc = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)], -1)
    j = pos // blk
    if s["table"] is not None:
        at = (s["table"].long()[row, torch.clamp(j // 64, max=s["table"].shape[1] - 1)], j % 64)
    else:
        at = (row, torch.clamp(j, max=s["kc"].shape[1] - 1))
    for name, new in (("kc", kc.view(torch.uint8)), ("vc", vc.view(torch.uint8)), ("sc", sc)):
        old = s[name].view(torch.uint8)
        old[at] = torch.where(done.view(-1, 1, 1), new, old[at])
    keep = ~done.view(-1, 1)
    st[..., 0], st[..., 1] = m1 * keep, n1 * keep
    st[..., 4:] = acc * keep[..., None]
    return s["kw"], s["vw"], s["kc"], s["vc"], s["sc"], st


def _gather(x, table, n):
    """[B, n, ...] rows of a contiguous cache or of a page pool."""
    return x[:, :n] if table is None else x.view(torch.uint8)[table.long()].view(x.dtype).flatten(1, 2)[:, :n]


def _read(s):
    n = s["n"]
    live = torch.arange(n, device=s["kc"].device)[None] < s["counts"][:, None]
    sc = _gather(s["sc"], s["table"], n).float()
    for i, (src, dst) in enumerate((("kc", "k_out"), ("vc", "v_out"))):
        x = _gather(s[src], s["table"], n).float() * sc[..., i:i + 1]
        s[dst].copy_(torch.where(live[..., None, None], x.to(torch.bfloat16), s[dst]))
    return s["k_out"], s["v_out"]


def _unit(x, gain, on):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain if on else x


def _attend(s):
    """The decode of either kind in fp32: logits over [prefix entries, own entries, window], one softmax."""
    B, Hq, Hkv, W, blk = s["B"], s["Hq"], s["Hkv"], s["W"], s["blk"]
    dev, on = s["q"].device, s["norm"]
    L = s["seqlens"].long()
    nc = torch.clamp(torch.div(L - W, blk, rounding_mode="floor"), min=0)[:, None]
    q = _unit(s["q"].float(), s["gq"], on).view(B, Hkv, Hq // Hkv, 512) * s["scale"]
    skip = s["kp"].shape[0] if "kp" in s else 0
    n = s["kc"].shape[1] if s["table"] is None else s["table"].shape[1] * 64
    if s["op"] == "decode":
        sc = _gather(s["sc"], s["table"], n).float()
        k = _gather(s["kc"], s["table"], n).float() * sc[..., :1]
        v = _gather(s["vc"], s["table"], n).float() * sc[..., 1:]
    else:
        k, v = (s[x][s["table"].long()].flatten(1, 2) if s["table"] is not None else s[x] for x in ("kc", "vc"))
        k, v = k.float(), v.float()
    z = [torch.einsum("bghd,bngd->bghn", q, _unit(k, s["gk"], on)),
         torch.einsum("bghd,bngd->bghn", q, _unit(s["kw"].float(), s["gk"], on))]
    slot = torch.arange(W, device=dev)[None]
    live = [skip + torch.arange(n, device=dev)[None] < nc,
            slot < torch.clamp(L, max=W)[:, None] if s["ring"] else slot >= W - torch.clamp(L, max=W)[:, None]]
    if skip:
        z.insert(0, torch.einsum("bghd,ngd->bghn", q, _unit(s["kp"].float(), s["gk"], on)))
        live.insert(0, torch.arange(skip, device=dev)[None] < nc)
    z = torch.cat(z, -1).masked_fill(~torch.cat(live, -1)[:, None, None], float("-inf"))
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = torch.einsum("bghn,bngd->bghd", p[..., skip:skip + n], v)
    out = out + torch.einsum("bghn,bngd->bghd", p[..., skip + n:], s["vw"].float())
    if skip:
        out = out + torch.einsum("bghn,ngd->bghd", p[..., :skip], s["vp"].float())
    out = out.reshape(B, Hq, 512)
    if s["gates"] is not None:
        out = out / (1 + torch.exp(-s["gates"].float()))
    if s.get("U") is not None:
        out = out + torch.einsum("hr,brd->bhd", s["U"], torch.einsum("hr,bhd->brd", s["V"], out))
    return out.to(torch.bfloat16)


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return (_write if op == "write" else _append if op == "append" else _read if op == "read" else _attend)(s)
    import compressed_long_context_b200 as hca
    if op == "write":
        return hca.compress_quant(s["k"], s["v"], s["pw"], blk=s["blk"])
    if op == "append":
        st = s["state"].clone()                # a pass starts from the same pool each time
        hca.append_quant(s["k_new"], s["v_new"], s["w_new"], s["seqlens"], s["kw"], s["vw"], s["kc"], s["vc"], s["sc"], st,
                      blk=s["blk"], page_table=s["table"])
        return s["kw"], s["vw"], s["kc"], s["vc"], s["sc"], st
    if op == "read":
        return hca.read_quant(s["kc"], s["vc"], s["sc"], s["counts"], s["n"], page_table=s["table"], k_out=s["k_out"],
                              v_out=s["v_out"])
    if op == "decode":
        return hca.decode_quant(s["q"], s["kc"], s["vc"], s["sc"], s["kw"], s["vw"], s["seqlens"], s["blk"], s["W"], s["scale"],
                             page_table=s["table"], gq=s["gq"], gk=s["gk"], eps=EPS, gate=s["gates"],
                             window_ring=s["ring"], vha_u=s["U"], vha_v=s["V"])
    return hca.decode_shared(s["q"], s["kp"], s["vp"], s["kc"], s["vc"], s["kw"], s["vw"], s["seqlens"], s["blk"], s["W"],
                             s["scale"], page_table=s["table"], gq=s["gq"], gk=s["gk"], eps=EPS, gate=s["gates"],
                             window_ring=s["ring"])


# ---------------------------------------------------------------- work

def work(case):
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    if op == "write":
        d, n = case["d"] + case["dv"], B * (case["T"] // case["blk"])
        tok = n * case["blk"]
        return {"bytes": tok * Hkv * d * 2 + (tok * 4 if case["w"] else 0) + n * Hkv * (d + 2), "flops": 2 * tok * Hkv * d}
    if op == "append":
        d = case["d"] + case["dv"]
        per = d * 2 + d * 2 + 2 * (4 + d) * 4 + case["full"] * (d + 2)      # token, ring slot, state in and out, entry
        return {"bytes": B * (Hkv * per + 8), "flops": 2 * B * Hkv * d}
    if op == "read":
        d, n = case["d"] + case["dv"], B * case["n"] * 0.75
        return {"bytes": n * Hkv * (d + 2 + 2 * d) + 4 * B, "flops": n * Hkv * d}
    Hq, W, blk = case["Hq"], case["W"], case["blk"]
    L = (case["lo"] + case["hi"]) / 2
    nw = min(W, L)
    io = B * Hq * 512 * (4 + (2 if case["gate"] else 0))
    if op == "decode":
        nc = max(0.0, (L - W) / blk)
        return {"bytes": B * Hkv * (nc * 1026 + nw * 2048) + io, "flops": 2 * 1024 * Hq * B * (nc + nw)}
    nc = case["prefix"] + max(0.0, (L - W) / blk)
    suffix = max(0.0, (L - W) / blk)
    nw = min(W, case["prefix"] * blk + L)
    return {"bytes": Hkv * 2048 * (case["prefix"] + B * (suffix + nw)) + io, "flops": 2 * 1024 * Hq * B * (nc + nw)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda x: x.to(torch.float64)  # noqa: E731
    op, B, Hkv = case["op"], case["B"], case["Hkv"]

    def code(x):
        e = _scale_exp(x.abs().amax(-1))
        return _exact_e4m3(torch.ldexp(x, -e[..., None])), torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)

    if op == "write":
        n, blk = case["T"] // case["blk"], case["blk"]
        if s["pw"] is None:
            a = torch.full((B, n, blk), 1.0 / blk, dtype=torch.float64, device=s["k"].device)
        else:
            a = torch.softmax(f(s["pw"][:, :n * blk]).view(B, n, blk), -1)
        outs = [code(torch.einsum("bni,bnigd->bngd", a, f(x[:, :n * blk]).view(B, n, blk, Hkv, -1))) for x in (s["k"], s["v"])]
        return outs[0][0], outs[1][0], torch.stack([outs[0][1], outs[1][1]], -1)
    if op == "append":
        kw, vw, st, d = s["kw"], s["vw"], f(s["state"]), case["d"]
        kc, vc, sc = f(s["kc"].float()), f(s["vc"].float()), f(s["sc"].float())
        for b in range(B):
            p = int(s["seqlens"][b]) - 1
            kw[b, p % case["W"]], vw[b, p % case["W"]] = s["k_new"][b], s["v_new"][b]
            for h in range(Hkv):
                w, (m, t) = float(s["w_new"][b]), st[b, h, :2].tolist()
                ref = max(m, w) if t > 0 else w
                a, e = (math.exp(m - ref) if t > 0 else 0.0), math.exp(w - ref)
                acc = st[b, h, 4:] * a + f(torch.cat([s["k_new"][b, h], s["v_new"][b, h]])) * e
                st[b, h, 0], st[b, h, 1], st[b, h, 4:] = ref, t * a + e, acc
                if (p + 1) % case["blk"] == 0:
                    j = p // case["blk"]
                    at = (b, j, h) if s["table"] is None else (int(s["table"][b, j // 64]), j % 64, h)
                    mean = acc / (t * a + e)
                    kc[at], sc[at + (0,)] = code(mean[:d])
                    vc[at], sc[at + (1,)] = code(mean[d:])
                    st[b, h] = 0
        return kw, vw, kc, vc, sc, st
    n_of = lambda b, n: (b, slice(0, n))  # noqa: E731

    def rows(x, b, n):
        """The first n rows of sequence b in 64 bits (e4m3 and e8m0 as the values they stand for)."""
        if s["table"] is None:
            y = x[n_of(b, n)]
        else:
            y = x.view(torch.uint8)[s["table"][b].long()].view(x.dtype).flatten(0, 1)[:n] if x.element_size() == 1 else \
                x[s["table"][b].long()].flatten(0, 1)[:n]
        return f(y.float())

    if op == "read":
        k, v = f(s["k_out"]), f(s["v_out"])
        for b in range(B):
            n = int(s["counts"][b])
            sc = rows(s["sc"], b, n)
            k[b, :n], v[b, :n] = rows(s["kc"], b, n) * sc[..., :1], rows(s["vc"], b, n) * sc[..., 1:]
        return k, v
    Hq, W, blk = case["Hq"], case["W"], case["blk"]
    skip = case.get("prefix", 0)
    norm = lambda x, gain: x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * f(gain) if case["norm"] else x  # noqa: E731
    kp, vp = (norm(f(s["kp"]), s["gk"]), f(s["vp"])) if skip else (None, None)
    out = torch.empty(B, Hq, 512, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        L = int(s["seqlens"][b])
        nc = max(0, (L - W) // blk)
        mine, nw = max(0, nc - skip), min(W, L)
        k, v = rows(s["kc"], b, mine), rows(s["vc"], b, mine)
        if op == "decode":
            sc = rows(s["sc"], b, mine)
            k, v = k * sc[..., :1], v * sc[..., 1:]
        win = slice(0, nw) if case["ring"] else slice(W - nw, W)
        k = norm(torch.cat([k, f(s["kw"][b, win])]), s["gk"])
        v = torch.cat([v, f(s["vw"][b, win])])
        if skip:
            k, v = torch.cat([kp[:min(nc, skip)], k]), torch.cat([vp[:min(nc, skip)], v])
        q = norm(f(s["q"][b]), s["gq"]).view(Hkv, Hq // Hkv, 512)
        p = torch.softmax(torch.einsum("ghd,ngd->ghn", q, k) * s["scale"], -1)
        out[b] = torch.einsum("ghn,ngd->ghd", p, v).reshape(Hq, 512)
    if s["gates"] is not None:
        out = out * torch.sigmoid(f(s["gates"]))
    if s.get("U") is not None:
        out = out + torch.einsum("hr,kr,bkd->bhd", f(s["U"]), f(s["V"]), out)
    return out
