"""The 8-bit compressed cache (compress_quant, append_quant, read_quant, decode_quant): refusals on the
CPU, and on the GPU every output against the formulas in 64 bits.

Bounds, from the formats.  e4m3 rounds by at most 2^-4 of the value (2^-10 * 2^e below its normal range).
decode_quant multiplies probabilities held as e4m3 + e5m2 terms, at most 2^-4 * 2^-3 = 2^-7 off (2^-8 over
the bf16 window), and bf16 outputs add 2^-8 of themselves: |err| <= 2^-7 sum p|v| + 2^-8 |out|, plus
2 delta sum p|v| where delta is how far a logit may be off (fp32 sums and exponentials, 2^-18 of
sum |q||k| scale; with QK normalisation the query is rounded to 8 significant bits, 2^-8 of it).
The 2^-7 holds where the e4m3 term is normal.  In the kernel's units (reference 2^-m, the row's largest
p * 2^e, e the value's scale, held at 2^4 or more) that is p * 2^e >= 2^-6; below, the e4m3 term is off by at most
half its last step, 2^-10, and the e5m2 term holds that to 2^-3 (or to 2^-17, half its last step): 2^-13 in all,
which is 2^-13 / 2^4 = 2^-17 of max(p * 2^e) for
each code of an entry that is multiplied with it."""
import ctypes

import pytest
import torch

import compressed_long_context_b200 as hca
from compressed_long_context_b200 import _lib
from test_binding_host import stub  # noqa: F401

bf, f8, e8 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=torch.uint8).view(dtype) if dtype in (f8, e8) else torch.zeros(shape, dtype=dtype)


# ------------------------------------------------------------------ refusals (CPU)

def test_footprints(stub):  # noqa: F811
    B, T, d, dv = 2, 300, 64, 128
    k, v = z(B, T, 1, d), z(B, T, 1, dv)
    kc, vc, sc = hca.compress_quant(k, v, blk=128)
    assert kc.dtype == f8 and sc.dtype == e8 and kc.shape == (B, 2, 1, d) and sc.shape == (B, 2, 1, 2)
    for kw in (dict(kc=z(B, 1, 1, d, dtype=f8)), dict(vc=z(B, 2, 1, d, dtype=f8)), dict(sc=z(B, 2, 1, 1, dtype=e8)),
               dict(w=z(B, T - 1, dtype=torch.float32))):
        with pytest.raises(ValueError):
            hca.compress_quant(k, v, blk=128, **kw)
    with pytest.raises(TypeError):
        hca.compress_quant(k, v, kc=z(B, 2, 1, d))
    with pytest.raises(TypeError):
        hca.compress_quant(k, v, sc=z(B, 2, 1, 2))
    cnt, table = z(B, dtype=torch.int32), z(B, 3, dtype=torch.int32)
    hca.read_quant(kc, vc, sc, cnt, 2)
    pool = dict(kc=z(5, 64, 1, d, dtype=f8), vc=z(5, 64, 1, dv, dtype=f8), sc=z(5, 64, 1, 2, dtype=e8))
    hca.read_quant(**pool, counts=cnt, n=100, page_table=table)
    n = len(stub.calls)
    for bad in (dict(vc=z(4, 64, 1, dv, dtype=f8)), dict(sc=z(5, 64, 1, 1, dtype=e8)), dict(k_out=z(B, 99, 1, d)),
                dict(page_table=z(1, 3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            hca.read_quant(**{**pool, **dict(counts=cnt, n=100, page_table=table), **bad})
    assert len(stub.calls) == n
    st = torch.zeros(hca.append_state_size(B, 1, d, dv) // 4)
    a = dict(k_new=z(B, 1, d), v_new=z(B, 1, dv), w_new=None, seqlens=cnt, kw=z(B, 9, 1, d), vw=z(B, 9, 1, dv), kc=kc, vc=vc,
             sc=sc, state=st, blk=16)
    hca.append_quant(**a)
    for bad in (dict(kw=z(1, 9, 1, d)), dict(vc=z(1, 2, 1, dv, dtype=f8)), dict(sc=z(1, 2, 1, 2, dtype=e8)), dict(state=st[1:]),
                dict(seqlens=z(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            hca.append_quant(**{**a, **bad})
    q = z(B, 64, 512)
    c = dict(q=q, kc=z(B, 7, 1, 512, dtype=f8), vc=z(B, 7, 1, 512, dtype=f8), sc=z(B, 7, 1, 2, dtype=e8), kw=z(B, 9, 1, 512),
             vw=z(B, 9, 1, 512), seqlens=cnt, blk=16, W=9, scale=0.1, workspace=z(64, dtype=torch.uint8))
    assert hca.decode_quant(**c).dtype == bf and hca.decode_quant(**c, out_f32=True).dtype == torch.float32
    for bad in (dict(W=10), dict(vc=z(1, 7, 1, 512, dtype=f8)), dict(sc=z(B, 7, 1, 1, dtype=e8)), dict(gate=z(B, 63, 512)),
                dict(out=z(B, 63, 512)), dict(vha_u=z(64, 2, dtype=torch.float32), vha_v=z(63, 2, dtype=torch.float32))):
        with pytest.raises(ValueError):
            hca.decode_quant(**{**c, **bad})


def test_rejects_before_launch(libhca):
    p, odd = ctypes.c_void_p(16), ctypes.c_void_p(17)
    U, I, OK = _lib.HCA_ERR_UNSUPPORTED, _lib.HCA_ERR_INVALID_ARG, _lib.HCA_OK

    def write(k=p, sc=p, B=1, T=256, Hkv=1, d=64, dv=64, blk=128):
        return libhca.hca_compress_quant(k, p, None, p, p, sc, B, T, Hkv, d, dv, blk, None)
    assert [write(d=96), write(blk=129), write(k=None), write(sc=odd), write(B=-1), write(Hkv=0), write(blk=0)] == \
        [U, U, I, I, I, I, I]
    assert write(T=100, k=None) == OK

    def append(seq=p, sc=p, table=None, ps=0, mp=0, npg=0, B=1, d=64, blk=16, W=4, Nmax=4, flags=0):
        return libhca.hca_append_quant(p, p, None, seq, p, p, p, p, sc, table, ps, mp, npg, p, B, 1, d, 64, blk, W, Nmax,
                                       flags, None)
    assert [append(d=32), append(blk=129), append(flags=_lib.HCA_QK_NORM), append(seq=None), append(sc=odd), append(W=0),
            append(Nmax=0), append(flags=_lib.HCA_PAGED), append(flags=_lib.HCA_PAGED, table=p, ps=65, mp=1, npg=1)] == \
        [U, U, U, I, I, I, I, I, I]
    assert append(B=0, seq=None) == OK

    def read(cnt=p, B=1, n=4, d=64, Nmax=4, flags=0, table=None):
        return libhca.hca_read_quant(p, p, p, table, 64, 1, 1, cnt, p, p, B, n, 1, d, 64, Nmax, flags, None)
    assert [read(d=8), read(flags=2), read(cnt=None), read(cnt=odd), read(n=-1), read(Nmax=0), read(flags=_lib.HCA_PAGED)] == \
        [U, U, I, I, I, I, I]
    assert read(n=0, cnt=None) == OK

    def decode(q=p, sc=p, ws=p, wsb=1 << 20, B=1, Hq=64, Hkv=1, d=512, blk=128, W=128, Nmax=8, scale=0.05, eps=1e-6, flags=0,
               gate=None, vu=None, vv=None, r=0):
        return libhca.hca_decode_quant(q, p, p, sc, None, 0, 0, 0, p, p, p, None, None, eps, gate, vu, vv, r, p, ws, wsb, B,
                                       Hq, Hkv, d, 512, blk, W, Nmax, scale, flags, None)
    assert [decode(d=256), decode(Hq=65), decode(Hq=3, Hkv=2), decode(blk=129), decode(flags=1 << 9),
            decode(vu=p, vv=p, r=4, Hkv=2)] == [U] * 6
    assert [decode(q=None), decode(sc=odd), decode(ws=None), decode(W=0), decode(Nmax=0), decode(scale=float("nan")),
            decode(eps=-1.0), decode(flags=_lib.HCA_QK_NORM), decode(flags=_lib.HCA_OUT_GATE), decode(vu=p, r=4),
            decode(flags=_lib.HCA_PAGED)] == [I] * 11
    assert decode(B=0, q=None) == OK


# ------------------------------------------------------------------ formulas in 64 bits

def exponent(amax):
    """Smallest e in [-64, 120] with amax <= 448 * 2^e."""
    e = torch.full(amax.shape, -64, dtype=torch.int64, device=amax.device)
    for _ in range(184):
        e = torch.where(amax > 448.0 * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=e.device), e.double()), e + 1, e)
    return e.clamp(max=120)


def rand_cache(g, dev, shape, boost=True):
    """Codes, scale bytes and the values they stand for, of random entries [.., Hkv, D]."""
    x = torch.randn(shape, generator=g, device=dev) * 0.5
    if boost:
        x = torch.where(torch.rand(shape[:-1] + (1,), generator=g, device=dev) < 0.05, x * 8, x)
    e = exponent(x.double().abs().amax(-1))
    codes = torch.ldexp(x, -e[..., None]).to(f8)
    return codes, (e + 127).to(torch.uint8), codes.float().double() * torch.pow(2.0, e.double())[..., None]


def pair(a, b):
    return torch.stack([a, b], -1).contiguous().view(e8)


def table_for(g, dev, B, pages, spare=3):
    perm = torch.randperm(B * pages + spare, generator=torch.Generator().manual_seed(g))[:B * pages]
    return perm.view(B, pages).to(torch.int32).to(dev), B * pages + spare


def paged(x, table, total, ps):
    """[B, N, ...] into a pool of pages of ps rows (rows behind the end and unused pages: garbage bytes)."""
    B, N = x.shape[:2]
    pool = torch.full((total, ps) + x.shape[2:], 0x7f, dtype=torch.uint8, device=x.device)
    xb = x.view(torch.uint8)
    for b in range(B):
        for i in range(-(-N // ps)):
            part = xb[b, i * ps:(i + 1) * ps]
            pool[int(table[b, i]), :part.shape[0]] = part
    return pool.view(x.dtype)


def done():
    torch.cuda.synchronize()
    hca.get_device_error()


# ------------------------------------------------------------------ write

@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hkv,d,dv,blk,w", [(1, 256, 1, 512, 512, 128, True), (2, 1000, 1, 512, 512, 128, False),
                                                (3, 300, 2, 64, 128, 37, True), (1, 9, 3, 256, 64, 1, True),
                                                (2, 513, 1, 128, 256, 128, True)])
def test_write(cuda_device, libhca, B, T, Hkv, d, dv, blk, w):
    dev, g = cuda_device, torch.Generator(device=cuda_device).manual_seed(T)
    k, v = (torch.randn(B, T, Hkv, x, generator=g, device=dev).to(bf) for x in (d, dv))
    k[0, :blk] = 0                                       # a zero vector: the smallest scale, zero codes
    v[0, blk:2 * blk] *= 2.0 ** 100
    pw = torch.randn(B, T, generator=g, device=dev) if w else None
    if w and blk > 2:
        pw[0, 1] = float("-inf")                         # a token pooled with no weight
    kc, vc, sc = hca.compress_quant(k, v, pw, blk=blk)
    done()
    n = T // blk
    a = torch.softmax((pw if w else torch.zeros(B, T, device=dev)).double()[:, :n * blk].view(B, n, blk), -1)
    for x, codes, s in ((k, kc, sc[..., 0]), (v, vc, sc[..., 1])):
        ref = torch.einsum("bni,bnigd->bngd", a, x.double()[:, :n * blk].view(B, n, blk, Hkv, -1))
        amax = ref.abs().amax(-1)
        e = s.contiguous().view(torch.uint8).long() - 127
        # a maximum within fp32 rounding of a border may fall on either side of it
        near = (exponent(amax * (1 - 2.0 ** -18)) == e) | (exponent(amax * (1 + 2.0 ** -18)) == e)
        assert bool(near.all())
        two_e = torch.pow(2.0, e.double())[..., None]
        err = (codes.float().double() * two_e - ref).abs()
        # half a step of e4m3, and the fp32 sum over the block (at most 128 terms, 2^-17 of sum a|x|)
        mass = torch.einsum("bni,bnigd->bngd", a, x.double().abs()[:, :n * blk].view(B, n, blk, Hkv, -1))
        assert bool((err <= torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * two_e) + 2.0 ** -16 * mass).all())


@pytest.mark.gpu
def test_write_not_finite(cuda_device, libhca):
    """A value that is not finite becomes NaN and leaves the rest of its entry alone."""
    dev = cuda_device
    k = torch.ones(1, 4, 1, 64, dtype=bf, device=dev)
    k[0, 1, 0, 5], k[0, 1, 0, 6], k[0, 2, 0, 7] = float("inf"), float("nan"), float("-inf")
    kc, vc, sc = hca.compress_quant(k, torch.ones_like(k), blk=4)
    done()
    x = kc[0, 0, 0].float() * sc[0, 0, 0, 0].float()
    bad = torch.zeros(64, dtype=torch.bool, device=dev)
    bad[5:8] = True
    assert torch.equal(x.isnan(), bad) and bool((x[~bad] == 1).all())


# ------------------------------------------------------------------ append, then read back

@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,d,dv,blk,W,ps", [(3, 1, 512, 512, 128, 128, 0), (2, 2, 64, 128, 16, 7, 64),
                                                 (4, 1, 256, 64, 5, 1, 128)])
def test_append_equals_write(cuda_device, libhca, B, Hkv, d, dv, blk, W, ps):
    """Token after token: the ring bit for bit, and entries equal to those of the whole prompt up to a step
    (two orders of one fp32 sum may fall on either side of a code's border)."""
    dev, g = cuda_device, torch.Generator(device=cuda_device).manual_seed(7)
    T = 3 * blk + 2
    k, v = (torch.randn(B, T, Hkv, x, generator=g, device=dev).to(bf) for x in (d, dv))
    w = torch.randn(B, T, generator=g, device=dev) * 0.5
    w[0, 0], w[0, blk + 1] = float("-inf"), float("-inf")
    kc, vc, sc = hca.compress_quant(k, v, w, blk=blk)
    table, total, N = None, 0, 4
    if ps:
        table, total = table_for(3, dev, B, 1)
    shape = (total, ps) if ps else (B, N)
    kw, vw = torch.zeros(B, W, Hkv, d, dtype=bf, device=dev), torch.zeros(B, W, Hkv, dv, dtype=bf, device=dev)
    ak, av = (torch.full(shape + (Hkv, x), 9, dtype=torch.uint8, device=dev).view(f8) for x in (d, dv))
    asc = torch.full(shape + (Hkv, 2), 9, dtype=torch.uint8, device=dev).view(e8)
    st = torch.zeros(hca.append_state_size(B, Hkv, d, dv), dtype=torch.uint8, device=dev)
    for t in range(T):
        seq = torch.full((B,), t + 1, dtype=torch.int32, device=dev)
        hca.append_quant(k[:, t].contiguous(), v[:, t].contiguous(), w[:, t].contiguous(), seq, kw, vw, ak, av, asc, st, blk,
                         page_table=table)
    hca.append_quant(k[:, 0].contiguous(), v[:, 0].contiguous(), None, torch.zeros_like(seq), kw, vw, ak, av, asc, st, blk,
                     page_table=table)                    # padding rows: nothing changes
    cnt = torch.full((B,), 3, dtype=torch.int32, device=dev)
    rk, rv = hca.read_quant(ak, av, asc, cnt, 5, page_table=table) if ps else hca.read_quant(ak, av, asc, cnt, 4)
    done()
    for p in range(max(0, T - W), T):
        assert torch.equal(kw[:, p % W], k[:, p]) and torch.equal(vw[:, p % W], v[:, p])
    for got, codes, s in ((rk, kc, sc[..., 0]), (rv, vc, sc[..., 1])):
        ref = codes.float() * s.float()[..., None]
        step = torch.maximum(2.0 ** -3 * ref.abs(), 2.0 ** -9 * s.float()[..., None])
        assert bool(((got[:, :3].float() - ref).abs() <= step).all())
        assert float((got[:, :3].float() != ref).float().mean()) < 0.01
        assert bool((got[:, 3:] == 0).all())
    for t in (ak, av, asc):                                # rows past the last entry: as they were
        b = t.view(torch.uint8)
        rows = b[table.long()].flatten(1, 2) if ps else b
        assert bool((rows[:, 3:] == 9).all())


@pytest.mark.gpu
def test_device_input_errors(cuda_device, libhca):
    dev = cuda_device
    kn = torch.ones((1, 1, 64), dtype=bf, device=dev)
    kw, kc = torch.zeros((1, 8, 1, 64), dtype=bf, device=dev), torch.zeros((1, 1, 1, 64), device=dev).to(f8)
    sc = torch.zeros((1, 1, 1, 2), dtype=torch.uint8, device=dev)
    st = torch.zeros(hca.append_state_size(1, 1, 64, 64), dtype=torch.uint8, device=dev)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731

    def reported():
        with pytest.raises(hca.HCAError) as e:
            hca.get_device_error()
        assert e.value.code == 5
        hca.get_device_error()
    hca.append_quant(kn, kn, None, i32(8), kw, kw.clone(), kc, kc.clone(), sc, st, 4)      # entry 1 of a cache of 1
    reported()
    hca.append_quant(kn, kn, None, i32(-1), kw, kw.clone(), kc, kc.clone(), sc, st, 4)
    reported()
    pool, psc = torch.zeros((2, 64, 1, 64), device=dev).to(f8), torch.zeros((2, 64, 1, 2), dtype=torch.uint8, device=dev)
    for cnt, tab in ((65, 0), (-1, 0), (3, 2), (3, -1)):
        k, v = hca.read_quant(pool, pool, psc, i32(cnt), 64, page_table=i32(tab).view(1, 1))
        reported()
        assert bool((k[:, 64 if cnt == 65 else 0:] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,Hkv,d,dv,ps", [(1, 1, 1, 512, 512, 0), (3, 70, 2, 64, 128, 64), (2, 300, 1, 256, 512, 128),
                                             (5, 33, 3, 128, 64, 0)])
def test_read(cuda_device, libhca, B, n, Hkv, d, dv, ps):
    """Exact, every code among the values; rows behind the counts stay."""
    dev, g = cuda_device, torch.Generator(device=cuda_device).manual_seed(n)
    kc, vc = (torch.randint(0, 256, (B, n, Hkv, x), generator=g, device=dev, dtype=torch.uint8).view(f8) for x in (d, dv))
    sc = torch.randint(63, 248, (B, n, Hkv, 2), generator=g, device=dev, dtype=torch.uint8).view(e8)
    cnt = torch.randint(0, n + 1, (B,), generator=g, device=dev).to(torch.int32)
    cnt[0] = n
    ko, vo = torch.full((B, n, Hkv, d), 3.0, dtype=bf, device=dev), torch.full((B, n, Hkv, dv), 3.0, dtype=bf, device=dev)
    table = None
    a = (kc, vc, sc)
    if ps:
        table, total = table_for(1, dev, B, -(-n // ps))
        a = tuple(paged(x, table, total, ps) for x in a)
    hca.read_quant(*a, cnt, n, page_table=table, k_out=ko, v_out=vo)
    done()
    live = (torch.arange(n, device=dev)[None] < cnt[:, None])[..., None, None]
    for got, c, s in ((ko, kc, sc[..., :1]), (vo, vc, sc[..., 1:])):
        want = torch.where(live, (c.float() * s.float()).to(bf), torch.full_like(got, 3.0))
        assert torch.equal(torch.nan_to_num(got, 77.0), torch.nan_to_num(want, 77.0))


# ------------------------------------------------------------------ decode

def decode_case(dev, seed, lengths, Hq, Hkv, blk, W, ps=0, norm=False, gate=False, ring=False, vha=0, onehot=False):
    """Arguments of decode_quant, and the reference with its bound."""
    g = torch.Generator(device=dev).manual_seed(seed)
    B, G = len(lengths), Hq // Hkv
    nc = [max(0, (L - W) // blk) for L in lengths]
    N = max(1, max(nc))
    kc, ks, kval = rand_cache(g, dev, (B, N, Hkv, 512))
    vc, vs, vval = rand_cache(g, dev, (B, N, Hkv, 512))
    rb = lambda *s: torch.randn(s, generator=g, device=dev).to(bf)  # noqa: E731
    kw, vw = rb(B, W, Hkv, 512), rb(B, W, Hkv, 512)
    if onehot:
        # entry j lights channel j, window slot i channel 511 - i, entries of different magnitudes: the
        # outputs are the probabilities themselves
        assert N + W <= 512
        vc, vw = torch.zeros((B, N, Hkv, 512), device=dev), torch.zeros_like(vw)
        for j in range(N):
            vc[:, j, :, j] = 1
        for i in range(W):
            vw[:, i, :, 511 - i] = 1
        vs = (127 + (torch.arange(N, device=dev) % 7) * 5 - 15).to(torch.uint8)[None, :, None].expand(B, N, Hkv).contiguous()
        vval = vc.double() * torch.pow(2.0, vs.double() - 127)[..., None]
        vc = vc.to(f8)
    sc = pair(ks, vs)
    for b, n in enumerate(nc):                        # what lies behind the entries is garbage
        kc.view(torch.uint8)[b, n:], vc.view(torch.uint8)[b, n:], sc.view(torch.uint8)[b, n:] = 0x7f, 0x7f, 0xff
    q = rb(B, Hq, 512)
    gq, gk = ((torch.rand(512, generator=g, device=dev) + 0.5) for _ in range(2)) if norm else (None, None)
    gates = rb(B, Hq, 512) if gate else None
    u, v = ((torch.randn(Hq, vha, generator=g, device=dev) * 0.1) for _ in range(2)) if vha else (None, None)
    scale = 512 ** -0.5
    table = None
    a = (kc, vc, sc)
    if ps:
        table, total = table_for(seed, dev, B, -(-N // ps))
        a = tuple(paged(x, table, total, ps) for x in a)
    args = dict(q=q, kc=a[0], vc=a[1], sc=a[2], kw=kw, vw=vw, seqlens=torch.tensor(lengths, dtype=torch.int32, device=dev),
                blk=blk, W=W, scale=scale, page_table=table, gq=gq, gk=gk, gate=gates, window_ring=ring, vha_u=u, vha_v=v)
    out = torch.zeros(B, Hq, 512, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    unit = lambda x: x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) if norm else x  # noqa: E731
    for b, L in enumerate(lengths):
        if L == 0:
            continue
        nw = min(L, W)
        win = slice(0, nw) if ring else slice(W - nw, W)
        K = unit(torch.cat([kval[b, :nc[b]], kw[b, win].double()]))
        V = torch.cat([vval[b, :nc[b]], vw[b, win].double()])
        Q = unit(q[b].double()).view(Hkv, G, 512)
        if norm:
            Q, K = Q * gq.double(), K * gk.double()
        p = torch.softmax(torch.einsum("ghd,ngd->ghn", Q, K) * scale, -1)
        o = torch.einsum("ghn,ngd->ghd", p, V).reshape(Hq, 512)
        mass = torch.einsum("ghn,ngd->ghd", p, V.abs()).reshape(Hq, 512)
        d = (torch.einsum("ghd,ngd->ghn", Q.abs(), K.abs()).amax(-1) * scale).reshape(Hq, 1)
        s = torch.cat([torch.pow(2.0, vs[b, :nc[b]].double() - 127), torch.ones(nw, Hkv, dtype=torch.float64, device=dev)])
        lost = (p * s.T[:, None]).amax(-1)[..., None] * (vval[b, :nc[b]].abs() / s[:nc[b], :, None]).sum(0)[:, None]
        out[b] = o
        tol[b] = 2.0 ** -17 * lost.reshape(Hq, 512) + mass * (2.0 ** -7 + 2 * d * (2.0 ** -8 if norm else 2.0 ** -18) + 2.0 ** -16)
    if gate:
        s = torch.sigmoid(gates.double())
        out, tol = out * s, tol * s
    if vha:
        m = torch.eye(Hq, dtype=torch.float64, device=dev) + u.double() @ v.double().T
        out, tol = torch.einsum("hk,bkd->bhd", m, out), torch.einsum("hk,bkd->bhd", m.abs(), tol)
    return args, out, tol


def check(got, out, tol, extra=2.0 ** -8):
    err = (got.double() - out).abs()
    lim = tol + extra * (out.abs() + tol) + 1e-30
    assert bool((err <= lim).all()), float((err / lim).max())


LENGTHS = {"one": [1], "short": [1, 0, 127, 128, 129, 255, 256, 257], "ragged": [128 * 300 + 5, 1, 0, 16000, 128 * 129, 128 * 130],
           "long": [1 << 20], "many": list(range(1, 6000, 37))}


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,Hq,Hkv,blk,W,kw", [
    ("one", 64, 1, 128, 128, {}), ("short", 64, 1, 128, 128, dict(ring=True)), ("ragged", 64, 1, 128, 128, {}),
    ("ragged", 64, 1, 128, 256, dict(ps=64, norm=True, gate=True)), ("ragged", 40, 1, 100, 3, dict(ps=128, vha=4)),
    ("ragged", 9, 3, 64, 300, dict(norm=True, ring=True)), ("long", 64, 1, 128, 128, dict(vha=4, gate=True)),
    ("many", 16, 2, 128, 130, dict(gate=True)), ("many", 64, 1, 64, 1, dict(ps=64, ring=True, norm=True))])
def test_decode(cuda_device, libhca, lengths, Hq, Hkv, blk, W, kw):
    args, out, tol = decode_case(cuda_device, 5, LENGTHS[lengths], Hq, Hkv, blk, W, **kw)
    got = hca.decode_quant(**args)
    got32 = hca.decode_quant(**args, out_f32=True)
    done()
    check(got, out, tol)
    check(got32, out, tol, 2.0 ** -16)
    for b, L in enumerate(LENGTHS[lengths]):
        assert L or bool((got[b] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,Hq,Hkv,W,kw", [([16 * 300 + 9, 16 * 128 + 40, 55, 3], 64, 1, 40, {}),
                                                 ([16 * 200 + 9, 500], 4, 2, 200, dict(ps=64, ring=True)),
                                                 ([16 * 400 + 9], 64, 1, 60, dict(norm=True))])
def test_decode_probabilities(cuda_device, libhca, lengths, Hq, Hkv, W, kw):
    """One-hot values: each output channel is one key's probability, so the bound holds key by key."""
    args, out, tol = decode_case(cuda_device, 9, lengths, Hq, Hkv, 16, W, onehot=True, **kw)
    got = hca.decode_quant(**args, out_f32=True)
    done()
    check(got, out, tol, 2.0 ** -16)


@pytest.mark.gpu
def test_decode_growing_logits(cuda_device, libhca):
    """Keys that grow along the cache: the reference moves again and again; and huge logits."""
    args, _, _ = decode_case(cuda_device, 3, [16 * 1000 + 50], 64, 1, 16, 40)
    n = 1000
    grow = torch.arange(n, device=cuda_device) // 100
    sc = args["sc"].view(torch.uint8)
    sc[0, :n, 0, 0] += grow.to(torch.uint8)
    got = hca.decode_quant(**args, out_f32=True)
    done()
    k = args["kc"][0, :n, 0].float().double() * torch.pow(2.0, sc[0, :n, 0, :1].double() - 127)
    v = args["vc"][0, :n, 0].float().double() * torch.pow(2.0, sc[0, :n, 0, 1:].double() - 127)
    k, v = torch.cat([k, args["kw"][0, :, 0].double()]), torch.cat([v, args["vw"][0, :, 0].double()])
    q = args["q"][0].double()
    p = torch.softmax(q @ k.T * args["scale"], -1)
    d = (q.abs() @ k.abs().T * args["scale"]).amax(-1, keepdim=True)
    check(got[0], p @ v, (p @ v.abs()) * (2.0 ** -7 + 2 * d * 2.0 ** -18 + 2.0 ** -16), 2.0 ** -16)


@pytest.mark.gpu
def test_pipeline_streams_graph(cuda_device, libhca):
    """Prompt written, tokens appended, decoded and read back: on a side stream, captured and replayed."""
    dev, g = cuda_device, torch.Generator(device=cuda_device).manual_seed(11)
    B, T, W, blk = 2, 700, 64, 32
    k, v = (torch.randn(B, T + 40, 1, 512, generator=g, device=dev).to(bf) for _ in range(2))
    q = torch.randn(B, 64, 512, generator=g, device=dev).to(bf)
    n0 = T // blk

    def start():
        kc, vc, sc = hca.compress_quant(k[:, :n0 * blk].contiguous(), v[:, :n0 * blk].contiguous(), blk=blk)
        pad = lambda x: torch.cat([x.view(torch.uint8), torch.zeros_like(x.view(torch.uint8))], 1).view(x.dtype)  # noqa: E731
        kw, vw = (x[:, n0 * blk - W:n0 * blk].roll((n0 * blk) % W, 1).contiguous() for x in (k, v))
        st = torch.zeros(hca.append_state_size(B, 1, 512, 512), dtype=torch.uint8, device=dev)
        return [pad(kc), pad(vc), pad(sc), kw, vw, st, torch.full((B,), n0 * blk, dtype=torch.int32, device=dev)]

    def step(s, kn, vn, out):
        kc, vc, sc, kw, vw, st, seq = s
        seq += 1
        hca.append_quant(kn, vn, None, seq, kw, vw, kc, vc, sc, st, blk)
        hca.decode_quant(q, kc, vc, sc, kw, vw, seq, blk, W, 512 ** -0.5, window_ring=True, out=out)

    tok = [(k[:, n0 * blk + i].contiguous(), v[:, n0 * blk + i].contiguous()) for i in range(40)]
    a, want = start(), []
    for kn, vn in tok:
        out = torch.empty(B, 64, 512, dtype=bf, device=dev)
        step(a, kn, vn, out)
        want.append(out)
    done()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = start()
        kn, vn, out = torch.empty_like(tok[0][0]), torch.empty_like(tok[0][1]), torch.empty(B, 64, 512, dtype=bf, device=dev)
        saved = [t.clone() for t in b]
        step(b, *tok[0], out)                              # warm-up
        for t, o in zip(b, saved):
            t.view(torch.uint8).copy_(o.view(torch.uint8))
        torch.cuda.current_stream().synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            step(b, kn, vn, out)
        for (x, y), w in zip(tok, want):
            kn.copy_(x)
            vn.copy_(y)
            gr.replay()
            assert torch.equal(out, w)
    done()
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.gpu
def test_decode_device_input_errors(cuda_device, libhca):
    """A length past the cache, a negative one and a page outside the pool are reported, not followed."""
    args, _, _ = decode_case(cuda_device, 3, [16 * 300 + 50, 900], 64, 1, 16, 40, ps=64)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    for bad in (dict(seqlens=i32(1 << 30, 900)), dict(seqlens=i32(-5, 900)),
                dict(page_table=torch.full_like(args["page_table"], 1 << 20)),
                dict(page_table=torch.full_like(args["page_table"], -1))):
        hca.decode_quant(**{**args, **bad})
        with pytest.raises(hca.HCAError) as e:
            hca.get_device_error()
        assert e.value.code == 5
        hca.get_device_error()


@pytest.mark.gpu
def test_decode_large_batch(cuda_device, libhca):
    """More units than CTAs, and than tile counts are kept on chip: every row equals its own small batch's."""
    dev, g = cuda_device, torch.Generator(device=cuda_device).manual_seed(2)
    B, N, W = 2500, 9, 5
    kc, ks, _ = rand_cache(g, dev, (B, N, 1, 512))
    vc, vs, _ = rand_cache(g, dev, (B, N, 1, 512))
    sc = pair(ks, vs)
    q, kw, vw = (torch.randn(s, generator=g, device=dev).to(bf) for s in ((B, 4, 512), (B, W, 1, 512), (B, W, 1, 512)))
    seq = torch.randint(0, 16 * N + W + 16, (B,), generator=g, device=dev).to(torch.int32)
    a = lambda s: (q[s], kc[s], vc[s], sc[s], kw[s], vw[s], seq[s])  # noqa: E731
    big = hca.decode_quant(*a(slice(None)), 16, W, 0.05, out_f32=True)
    for b in (0, 1, 1023, 2047, 2048, 2300, 2499):
        one = hca.decode_quant(*a(slice(b, b + 1)), 16, W, 0.05, out_f32=True)
        done()
        assert torch.allclose(big[b], one[0], rtol=2e-6, atol=1e-6)     # (fp32 merge in another order)


@pytest.mark.gpu
def test_decode_two_streams(cuda_device, libhca):
    """Two calls at once, each with its own workspace."""
    cases = [decode_case(cuda_device, s, [16 * 700 + 50, 16 * 90], 64, 1, 16, 40, norm=s == 1) for s in range(2)]
    want = [hca.decode_quant(**c[0]) for c in cases]
    done()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(hca.decode_quant(**cases[i][0]))
    done()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)


@pytest.mark.gpu
def test_decode_unwinds_after_a_missing_slab(cuda_device, libhca):
    """A wait that runs out (shortened, on a key slab that is never requested) is reported and marks the output."""
    stream = torch.cuda.current_stream().cuda_stream
    args, out, tol = decode_case(cuda_device, 3, [16 * 300 + 50, 900], 64, 1, 16, 40)
    hca.get_device_error()
    try:
        assert libhca.hca_debug_set_wait_limit(2_000_000, stream) == _lib.HCA_OK      # 2 ms
        assert libhca.hca_debug_set_drop_slab(1, stream) == _lib.HCA_OK
        bad = hca.decode_quant(**args)
        torch.cuda.synchronize()
        assert libhca.hca_get_device_error(stream) == _lib.HCA_ERR_TIMEOUT
        assert torch.isnan(bad).all()
    finally:
        libhca.hca_debug_set_drop_slab(0, stream)
        libhca.hca_debug_set_wait_limit(0, stream)
    hca.get_device_error()
    good = hca.decode_quant(**args)
    done()
    check(good, out, tol)


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_device, libhca):
    """A pool of more than 2^32 code bytes, used at its end: the same bits as from a small pool."""
    dev = cuda_device
    args, _, _ = decode_case(dev, 6, [16 * 200 + 45], 64, 1, 16, 40, ps=64)
    P = (1 << 32) // (64 * 512) + 100
    move = lambda t: t + (P - 1 - int(args["page_table"].max()))  # noqa: E731
    pools = {}
    for name in ("kc", "vc", "sc"):
        small = args[name]
        big = torch.empty((P,) + small.shape[1:], dtype=torch.uint8, device=dev).view(small.dtype)
        big.view(torch.uint8)[P - small.shape[0]:] = 0
        for i in args["page_table"].flatten().tolist():
            big.view(torch.uint8)[int(move(i))] = small.view(torch.uint8)[i]
        pools[name] = big
    table = move(args["page_table"])
    want, got = hca.decode_quant(**args), hca.decode_quant(**{**args, **pools, "page_table": table})
    cnt = torch.tensor([200], dtype=torch.int32, device=dev)
    rw = hca.read_quant(args["kc"], args["vc"], args["sc"], cnt, 200, page_table=args["page_table"])
    rg = hca.read_quant(pools["kc"], pools["vc"], pools["sc"], cnt, 200, page_table=table)
    # and an entry written there
    g = torch.Generator(device=dev).manual_seed(1)
    kn, vn = (torch.randn(1, 1, 512, generator=g, device=dev).to(bf) for _ in range(2))
    kw = torch.zeros(1, 8, 1, 512, dtype=bf, device=dev)
    outs = []
    for kc, vc, sc, t in ((args["kc"], args["vc"], args["sc"], args["page_table"]), (pools["kc"], pools["vc"], pools["sc"], table)):
        st = torch.zeros(hca.append_state_size(1, 1, 512, 512), dtype=torch.uint8, device=dev)
        hca.append_quant(kn, vn, None, torch.tensor([131], dtype=torch.int32, device=dev), kw, kw.clone(), kc, vc, sc, st, 1,
                         page_table=t)
        pg = int(t[0, 130 // 64])
        outs.append([x.view(torch.uint8)[pg, 130 % 64] for x in (kc, vc, sc)])
    done()
    assert torch.equal(want, got) and all(torch.equal(a, b) for a, b in zip(rw, rg))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and torch.equal(outs[0][0].view(f8)[0].float().nan_to_num().ne(0),
                                                                         outs[1][0].view(f8)[0].float().nan_to_num().ne(0))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3])
def test_write_no_entries(cuda_device, libhca, n):
    """Fewer tokens than a block: nothing to write, empty results."""
    k = torch.ones(2, n, 1, 64, dtype=bf, device=cuda_device)
    kc, vc, sc = hca.compress_quant(k, k, blk=4)
    done()
    assert kc.shape == (2, 0, 1, 64) and sc.shape == (2, 0, 1, 2)


@pytest.mark.gpu
def test_decode_not_finite_query(cuda_device, libhca):
    """NaN or infinity in one head's query stays in that head."""
    args, out, tol = decode_case(cuda_device, 3, [16 * 300 + 50], 64, 1, 16, 40)
    q = args["q"].clone()
    q[0, 5, 100], q[0, 9, 3] = float("nan"), float("inf")
    got = hca.decode_quant(**{**args, "q": q})
    done()
    rest = [h for h in range(64) if h not in (5, 9)]
    assert torch.isnan(got[0, 5]).all() and torch.isnan(got[0, 9]).all()
    check(got[:, rest], out[:, rest], tol[:, rest])


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, 1])
def test_tokens_without_weight(cuda_device, libhca, first):
    """Tokens of weight -inf may hold NaN or infinities: the entry is that of the others, written at once or token by token."""
    dev, g = cuda_device, torch.Generator(device=cuda_device).manual_seed(4)
    blk, d = 8, 64
    k, v = (torch.randn(1, blk, 1, d, generator=g, device=dev).to(bf) for _ in range(2))
    w = torch.randn(1, blk, generator=g, device=dev)
    none = [first, 5]
    w[0, none] = float("-inf")
    clean = [hca.compress_quant(*(torch.where((w == float("-inf"))[..., None, None], 0, x) for x in (k, v)), w, blk=blk)]
    for x in (k, v):
        x[0, none[0]], x[0, none[1]] = float("nan"), float("inf")
    clean.append(hca.compress_quant(k, v, w, blk=blk))
    kw = torch.zeros(1, 4, 1, d, dtype=bf, device=dev)
    kc, vc, sc = (torch.zeros_like(x.view(torch.uint8)).view(x.dtype) for x in clean[0])
    st = torch.zeros(hca.append_state_size(1, 1, d, d), dtype=torch.uint8, device=dev)
    for t in range(blk):
        hca.append_quant(k[:, t].contiguous(), v[:, t].contiguous(), w[:, t].contiguous(),
                         torch.tensor([t + 1], dtype=torch.int32, device=dev), kw, kw.clone(), kc, vc, sc, st, blk)
    done()
    val = lambda c, s, i: c.float() * s.float()[..., i:i + 1]  # noqa: E731
    for i in range(2):
        a, b, c = (val(x[i], x[2], i) for x in (clean[0], clean[1], (kc, vc, sc)))
        step = torch.maximum(2.0 ** -3 * a.abs(), 2.0 ** -9 * clean[0][2].float()[..., i:i + 1])
        assert torch.equal(a, b) and bool(((c - a).abs() <= step).all())


@pytest.mark.gpu
@pytest.mark.parametrize("blk", [128, 37])
def test_write_largest_values(cuda_device, libhca, blk):
    """bf16's largest values pool without leaving fp32's range.  All tokens are equal, so an entry is its token: 2^-4 for the
    code's rounding, and far less than 2^-12 for the pooling's."""
    dev = cuda_device
    top = torch.finfo(bf).max
    x = torch.full((1, 2 * blk, 1, 64), top, dtype=bf, device=dev)
    x[..., ::2] = -top
    for w in (None, torch.linspace(-3, 3, 2 * blk, device=dev)[None].contiguous()):
        kc, vc, sc = hca.compress_quant(x, x, w, blk=blk)
        done()
        for i, c in enumerate((kc, vc)):
            e = c.double() * sc.double()[..., i:i + 1]
            want = x[:, :2].double()
            assert bool(((e - want).abs() <= (2.0 ** -4 + 2.0 ** -12) * want.abs()).all())
