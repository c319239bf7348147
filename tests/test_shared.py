"""decode_shared (a batch over one copy of its common prefix): refusals on the CPU, and on the GPU every
output against softmax attention in 64 bits over [prefix, own entries, window].

Bound: probabilities are rounded to bf16 (2^-8) and the prefix's part is normalised by the sum of the rounded
ones (another 2^-8), bf16 outputs add 2^-8 of themselves: |err| <= 2^-7 sum p|v| + 2^-8 |out|, plus
2 delta sum p|v| for logits off by delta (fp32 sums and exponentials: 2^-18 of sum |q||k| scale; with QK
normalisation the query is rounded to bf16: 2^-8 of it)."""
import ctypes

import pytest
import torch

import compressed_long_context_b200 as hca
from compressed_long_context_b200 import _lib
from test_binding_host import stub  # noqa: F401

bf = torch.bfloat16


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def test_footprints(stub):  # noqa: F811
    B, W = 3, 9
    a = dict(q=z(B, 64, 512), kp=z(5, 1, 512), vp=z(5, 1, 512), kc=z(B, 7, 1, 512), vc=z(B, 7, 1, 512), kw=z(B, W, 1, 512),
             vw=z(B, W, 1, 512), seqlens=z(B, dtype=torch.int32), blk=16, W=W, scale=0.1, workspace=z(64, dtype=torch.uint8))
    assert hca.decode_shared(**a).dtype == bf and hca.decode_shared(**a, out_f32=True).dtype == torch.float32
    hca.decode_shared(**{**a, "kp": z(0, 1, 512), "vp": z(0, 1, 512)})
    n = len(stub.calls)
    for bad in (dict(vp=z(4, 1, 512)), dict(W=10), dict(vc=z(2, 7, 1, 512)), dict(kp=z(5, 1, 256)), dict(gate=z(B, 63, 512)),
                dict(seqlens=z(2, dtype=torch.int32)), dict(out=z(B, 63, 512)),
                dict(vha_u=z(64, 2, dtype=torch.float32), vha_v=z(64, 3, dtype=torch.float32))):
        with pytest.raises(ValueError):
            hca.decode_shared(**{**a, **bad})
    with pytest.raises(TypeError):
        hca.decode_shared(**{**a, "kp": z(5, 1, 512, dtype=torch.float32)})
    assert len(stub.calls) == n


def test_rejects_before_launch(libhca):
    p, odd = ctypes.c_void_p(16), ctypes.c_void_p(20)
    U, I, OK = _lib.HCA_ERR_UNSUPPORTED, _lib.HCA_ERR_INVALID_ARG, _lib.HCA_OK

    def call(q=p, kp=p, ws=p, wsb=1 << 20, gq=None, B=1, Hq=64, Hkv=1, d=512, blk=128, W=128, Np=4, Nmax=8, scale=0.05,
             eps=1e-6, flags=0, gate=None, vu=None, vv=None, r=0):
        return libhca.hca_decode_shared(q, kp, p, p, p, None, 0, 0, 0, p, p, p, gq, gq, eps, gate, vu, vv, r, p, ws, wsb, B, Hq,
                                        Hkv, d, 512, blk, W, Np, Nmax, scale, flags, None)
    assert [call(d=256), call(Hq=65), call(Hq=3, Hkv=2), call(blk=129), call(flags=1 << 9), call(vu=p, vv=p, r=4, Hkv=2)] == \
        [U] * 6
    assert [call(q=None), call(kp=None), call(kp=odd), call(ws=None), call(W=0), call(Np=-1), call(Nmax=0),
            call(scale=float("nan")), call(eps=-1.0), call(flags=_lib.HCA_QK_NORM), call(flags=_lib.HCA_QK_NORM, gq=odd),
            call(flags=_lib.HCA_OUT_GATE), call(vu=p, r=4), call(flags=_lib.HCA_PAGED)] == [I] * 14
    assert call(B=0, q=None) == OK


def make(dev, seed, lengths, Np, Hq, Hkv, blk, W, ps=0, norm=False, gate=False, ring=False, vha=0, onehot=False, grow=0.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    B, G = len(lengths), Hq // Hkv
    nc = [max(0, (L - W) // blk) for L in lengths]
    N = max(1, max(nc) - Np)
    rb = lambda *s: torch.randn(s, generator=g, device=dev).to(bf)  # noqa: E731

    def rows(*s):
        x = torch.randn(s, generator=g, device=dev) * 0.5
        return torch.where(torch.rand(s[:-1] + (1,), generator=g, device=dev) < 0.05, x * 8, x).to(bf)
    q, kp, vp, kc, vc = rb(B, Hq, 512), rows(Np, Hkv, 512), rows(Np, Hkv, 512), rows(B, N, Hkv, 512), rows(B, N, Hkv, 512)
    kw, vw = rb(B, W, Hkv, 512), rb(B, W, Hkv, 512)
    if grow:                                              # logits that grow along the prefix
        kp = (kp.float() * (1 + grow * torch.arange(Np, device=dev)[:, None, None])).to(bf)
    if onehot:                                            # outputs are the probabilities
        assert Np + N + W <= 512
        vp, vc, vw = torch.zeros_like(vp), torch.zeros_like(vc), torch.zeros_like(vw)
        for j in range(Np):
            vp[j, :, j] = 1
        for j in range(N):
            vc[:, j, :, Np + j] = 1
        for j in range(W):
            vw[:, j, :, 511 - j] = 1
    for b, n in enumerate(nc):
        kc[b, max(0, n - Np):], vc[b, max(0, n - Np):] = float("nan"), float("nan")
    gq, gk = ((torch.rand(512, generator=g, device=dev) + 0.5) for _ in range(2)) if norm else (None, None)
    gates = rb(B, Hq, 512) if gate else None
    u, v = ((torch.randn(Hq, vha, generator=g, device=dev) * 0.1) for _ in range(2)) if vha else (None, None)
    table, ck, cv = None, kc, vc
    if ps:
        pages = -(-N // ps)
        total = B * pages + 2
        table = torch.randperm(total, generator=torch.Generator().manual_seed(seed))[:B * pages].view(B, pages)
        ck, cv = (torch.full((total, ps, Hkv, 512), float("nan"), dtype=bf, device=dev) for _ in range(2))
        for b in range(B):
            for i in range(pages):
                n = min(ps, N - i * ps)
                ck[table[b, i], :n], cv[table[b, i], :n] = kc[b, i * ps:i * ps + n], vc[b, i * ps:i * ps + n]
        table = table.to(torch.int32).to(dev)
    args = dict(q=q, kp=kp, vp=vp, kc=ck, vc=cv, kw=kw, vw=vw, seqlens=torch.tensor(lengths, dtype=torch.int32, device=dev),
                blk=blk, W=W, scale=512 ** -0.5, page_table=table, gq=gq, gk=gk, gate=gates, window_ring=ring, vha_u=u, vha_v=v)
    out = torch.zeros(B, Hq, 512, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    unit = lambda x: x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) if norm else x  # noqa: E731
    for b, L in enumerate(lengths):
        if L == 0:
            continue
        nw, own = min(L, W), max(0, nc[b] - Np)
        win = slice(0, nw) if ring else slice(W - nw, W)
        K = unit(torch.cat([kp[:min(nc[b], Np)], kc[b, :own], kw[b, win]]).double())
        V = torch.cat([vp[:min(nc[b], Np)], vc[b, :own], vw[b, win]]).double()
        Q = unit(q[b].double()).view(Hkv, G, 512)
        if norm:
            Q, K = Q * gq.double(), K * gk.double()
        p = torch.softmax(torch.einsum("ghd,ngd->ghn", Q, K) * 512 ** -0.5, -1)
        mass = torch.einsum("ghn,ngd->ghd", p, V.abs()).reshape(Hq, 512)
        d = (torch.einsum("ghd,ngd->ghn", Q.abs(), K.abs()).amax(-1) * 512 ** -0.5).reshape(Hq, 1)
        out[b] = torch.einsum("ghn,ngd->ghd", p, V).reshape(Hq, 512)
        tol[b] = mass * (2.0 ** -7 + 2 * d * (2.0 ** -8 if norm else 2.0 ** -18) + 2.0 ** -16)
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


def done():
    torch.cuda.synchronize()
    hca.get_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,Np,Hq,Hkv,blk,W,kw", [
    ([128 * 40 + 130], 32, 64, 1, 128, 128, {}),
    ([128 * 32 + 150, 128 * 33, 128 * 500, 128 * 34 + 1], 32, 64, 1, 128, 128, dict(gate=True)),
    # lengths inside the prefix, inside the window, padding rows
    ([1, 0, 127, 500, 16 * 255 + 40, 16 * 256 + 40, 16 * 257 + 40, 16 * 700], 300, 64, 1, 16, 40, dict(ring=True)),
    ([16 * 700 + 3, 40, 0, 16 * 300], 513, 40, 1, 16, 33, dict(ps=64, norm=True)),
    ([16 * 700 + 3, 40, 0, 16 * 300, 16 * 512 + 40], 512, 9, 3, 16, 40, dict(ps=128, gate=True, ring=True)),
    ([64 * 90 + i for i in range(0, 900, 50)], 70, 16, 2, 64, 300, dict(norm=True, gate=True)),
    ([16 * 1025 + 60 + 3 * i for i in range(33)], 1000, 32, 1, 16, 50, dict(vha=4, gate=True)),
    ([16 * 3000 + 60 + 7 * i for i in range(64)], 2999, 64, 1, 16, 50, dict(norm=True)),
    ([16 * 5000 + 60 + 7 * i for i in range(9)], 4990, 64, 4, 16, 50, {}),
    ([200, 100, 3], 1, 64, 1, 16, 40, dict(vha=2)), ([200, 100, 0], 0, 64, 1, 16, 40, {}),
    ([16 * 800 + 60, 16 * 800 + 90], 790, 1, 1, 16, 50, dict(grow=0.02))])
def test_shared(cuda_device, libhca, lengths, Np, Hq, Hkv, blk, W, kw):
    args, out, tol = make(cuda_device, 5, lengths, Np, Hq, Hkv, blk, W, **kw)
    got, got32 = hca.decode_shared(**args), hca.decode_shared(**args, out_f32=True)
    done()
    check(got32, out, tol, 2.0 ** -16)
    check(got, out, tol)
    for b, L in enumerate(lengths):
        assert L or bool((got[b] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [{}, dict(norm=True, ps=64)])
def test_probabilities(cuda_device, libhca, kw):
    """One-hot values: each output channel is one key's probability, so the bound holds key by key."""
    args, out, tol = make(cuda_device, 8, [16 * 340 + 45, 16 * 330 + 45, 16 * 257 + 45, 45, 7], 320, 64, 1, 16, 40, onehot=True, **kw)
    got = hca.decode_shared(**args, out_f32=True)
    done()
    check(got, out, tol, 2.0 ** -16)


@pytest.mark.gpu
def test_shared_equals_decode(cuda_device, libhca):
    """The same batch with the prefix copied into every sequence's cache, through decode."""
    dev = cuda_device
    args, out, tol = make(dev, 6, [16 * 400 + 60, 16 * 390 + 70], 380, 64, 1, 16, 50)
    a = dict(args)
    kp, vp = a.pop("kp"), a.pop("vp")
    kc, vc = (torch.cat([p[None].expand(2, -1, -1, -1), c], 1).contiguous() for p, c in ((kp, a["kc"]), (vp, a["vc"])))
    ref = hca.decode(a["q"], kc, vc, a["kw"], a["vw"], a["seqlens"], 16, 50, a["scale"])
    got = hca.decode_shared(**args, out_f32=True)
    done()
    check(got, out, tol, 2.0 ** -16)
    check(ref, out, tol, 2.0 ** -16)


@pytest.mark.gpu
def test_stream_and_graph(cuda_device, libhca):
    args, out, tol = make(cuda_device, 4, [16 * 400 + 60 + i for i in range(7)], 390, 64, 1, 16, 50, norm=True)
    want = hca.decode_shared(**args)
    done()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = hca.decode_shared(**args)
        gr = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(gr, stream=s):
            g1 = hca.decode_shared(**args)
            g2 = hca.decode_shared(**args)
        for _ in range(3):
            gr.replay()
    s.synchronize()
    done()
    assert torch.equal(got, want) and torch.equal(g1, want) and torch.equal(g2, want)


@pytest.mark.gpu
def test_device_input_errors(cuda_device, libhca):
    args, _, _ = make(cuda_device, 4, [16 * 30 + 60], 20, 64, 1, 16, 50, ps=64)
    for bad in (dict(seqlens=torch.tensor([-3], dtype=torch.int32, device=cuda_device)),
                dict(seqlens=torch.tensor([16 * 200], dtype=torch.int32, device=cuda_device)),
                dict(page_table=torch.full_like(args["page_table"], 99))):
        hca.decode_shared(**{**args, **bad})
        with pytest.raises(hca.HCAError) as e:
            hca.get_device_error()
        assert e.value.code == 5
        hca.get_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
def test_large_batch(cuda_device, libhca, norm):
    """Many row tiles and more units than CTAs: rows equal their own small batch's (fp32 sums in another order, and
    bf16 probabilities against another reference: 2^-8 of the mass at most, here against the formula's bound)."""
    L = [16 * 320 + 60 + 5 * i for i in range(300)]
    args, out, tol = make(cuda_device, 3, L, 310, 8, 1, 16, 50, norm=norm)
    got = hca.decode_shared(**args, out_f32=True)
    done()
    check(got, out, tol, 2.0 ** -16)


@pytest.mark.gpu
def test_two_streams(cuda_device, libhca):
    """Two calls at once, each with its own workspace, and one workspace used again."""
    cases = [make(cuda_device, s, [16 * 700 + 50 + i for i in range(5)], 600, 64, 1, 16, 40, norm=s == 1) for s in range(2)]
    want = [hca.decode_shared(**c[0]) for c in cases]
    ws = torch.empty(hca.decode_shared_workspace_size(5, 64, 1, 512, 600), dtype=torch.uint8, device=cuda_device)
    again = [hca.decode_shared(**c[0], workspace=ws) for c in cases]
    done()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(hca.decode_shared(**cases[i][0]))
    done()
    for g, w, a in zip(got, want, again):
        assert torch.equal(a, w) and all(torch.equal(x, w) for x in g)


@pytest.mark.gpu
def test_short_workspace_is_refused(cuda_device, libhca):
    args, _, _ = make(cuda_device, 4, [16 * 30 + 60], 20, 64, 1, 16, 50)
    n = hca.decode_shared_workspace_size(1, 64, 1, 512, 20)
    with pytest.raises(hca.HCAError) as e:
        hca.decode_shared(**args, workspace=torch.empty(n - 256, dtype=torch.uint8, device=cuda_device))
    assert e.value.code == _lib.HCA_ERR_INVALID_ARG
    done()


@pytest.mark.gpu
def test_unwinds_after_a_missing_slab(cuda_device, libhca):
    """A wait that runs out in the own pass is reported and marks the output; the next call is right."""
    stream = torch.cuda.current_stream().cuda_stream
    args, out, tol = make(cuda_device, 4, [16 * 400 + 60 + i for i in range(7)], 390, 64, 1, 16, 50)
    hca.get_device_error()
    try:
        assert libhca.hca_debug_set_wait_limit(2_000_000, stream) == _lib.HCA_OK      # 2 ms
        assert libhca.hca_debug_set_drop_slab(1, stream) == _lib.HCA_OK
        bad = hca.decode_shared(**args)
        torch.cuda.synchronize()
        assert libhca.hca_get_device_error(stream) == _lib.HCA_ERR_TIMEOUT
        assert torch.isnan(bad).all()
    finally:
        libhca.hca_debug_set_drop_slab(0, stream)
        libhca.hca_debug_set_wait_limit(0, stream)
    hca.get_device_error()
    good = hca.decode_shared(**args)
    done()
    check(good, out, tol)
