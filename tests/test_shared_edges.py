"""decode_shared at its edges: references that move, keys that are not finite, refusals, the serving loop, and how far off
QK normalisation may be.

Bound of `reference`: with logits off by at most delta_j for key j, |err| <= sum_j p_j delta_j (|v_j| + sum p|v|) to first order
(1.2 times that while delta <= 0.1), plus 2^-7 sum p|v| for probabilities of one bf16 term and a sum of rounded ones, plus 2^-16
of it for fp32 sums, plus the output's own rounding."""

import ctypes

import pytest
import torch

import compressed_long_context_b200 as hca
from compressed_long_context_b200 import _lib

bf = torch.bfloat16


def done():
    torch.cuda.synchronize()
    hca.get_device_error()


def check(got, out, tol, extra):
    err = (got.double() - out).abs()
    lim = tol + extra * (out.abs() + tol) + 1e-30
    assert bool((err <= lim).all()), float((err / lim).max())


def batch(dev, seed, B, Hq, Np, N, W, L):
    """Arguments of decode_shared on random inputs: one KV head, blocks of 16, sequences of lengths L."""
    g = torch.Generator(device=dev).manual_seed(seed)
    rb = lambda *s: torch.randn(s, generator=g, device=dev).to(bf)  # noqa: E731
    return dict(q=rb(B, Hq, 512), kp=rb(Np, 1, 512), vp=rb(Np, 1, 512), kc=rb(B, N, 1, 512), vc=rb(B, N, 1, 512),
                kw=rb(B, W, 1, 512), vw=rb(B, W, 1, 512), seqlens=torch.tensor(L, dtype=torch.int32, device=dev), blk=16, W=W,
                scale=512 ** -0.5)


def reference(a, dq_prefix=0.0, dq_own=0.0):
    """Softmax attention in 64 bits over [prefix, own entries, window] (linear window, one KV head), and its bound.  dq_*: how far
    (2-norm over the channels) a logit may be off for the rounding of normalised operands."""
    B, Hq, _ = a["q"].shape
    norm = a.get("gq") is not None
    unit = lambda x, g: x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * g.double() if norm else x  # noqa: E731
    out = torch.zeros(B, Hq, 512, dtype=torch.float64, device=a["q"].device)
    tol = torch.zeros_like(out)
    Np = a["kp"].shape[0]
    for b, L in enumerate(a["seqlens"].tolist()):
        nc, nw = max(0, (L - a["W"]) // a["blk"]), min(L, a["W"])
        own, pre = max(0, nc - Np), min(nc, Np)
        K = unit(torch.cat([a["kp"][:pre, 0], a["kc"][b, :own, 0], a["kw"][b, a["W"] - nw:, 0]]).double(), a.get("gk"))
        V = torch.cat([a["vp"][:pre, 0], a["vc"][b, :own, 0], a["vw"][b, a["W"] - nw:, 0]]).double()
        Q = unit(a["q"][b].double(), a.get("gq"))
        p = torch.softmax(Q @ K.T * a["scale"], -1)
        # every product is off by the same share of itself at most, with independent signs: 6 times the 2-norm of the bounds
        # is passed with probability 2 exp(-18)
        rms = torch.sqrt(Q ** 2 @ (K ** 2).T) * abs(a["scale"])
        delta = 2.0 ** -18 * (Q.abs() @ K.abs().T) * abs(a["scale"])
        delta = delta + 6 * torch.cat([rms[:, :pre] * dq_prefix, rms[:, pre:] * dq_own], -1)
        assert float(delta.max()) <= 0.1
        mass = p @ V.abs()
        out[b] = p @ V
        tol[b] = 1.2 * ((p * delta) @ V.abs() + (p * delta).sum(-1, keepdim=True) * mass) + mass * (2.0 ** -7 + 2.0 ** -16)
    return out, tol


@pytest.mark.gpu
@pytest.mark.parametrize("Np,step", [(1100, 3), (1100, 1), (395, 2)])
def test_references_move(cuda_device, libhca, Np, step):
    """Logits of half the heads rise by more than 2^32 every `step` units of 128 entries, the other half's fall: a unit that moves
    a row's reference is followed by units that weigh as much, so P against an older reference would show.  The same bits
    again and again."""
    dev = cuda_device
    a = batch(dev, 3, 5, 64, Np, 8, 40, [16 * (Np + i) + 60 for i in range(5)])
    axis = torch.zeros(512, device=dev)
    axis[:256] = 1.0
    level = (torch.arange(Np, device=dev) // (128 * step)).float()           # 40 log2 units more each
    per = 40 * 0.6931471805599453 / (256 * a["scale"])
    a["kp"] = (a["kp"].float() + axis * (level * per)[:, None, None]).to(bf)
    sign = torch.where(torch.arange(64, device=dev) % 2 == 0, 1.0, -1.0)
    a["q"] = (a["q"].float() * 0.25 + sign[None, :, None] * axis).to(bf)
    out, tol = reference(a)
    got = hca.decode_shared(**a, out_f32=True)
    done()
    check(got, out, tol, 2.0 ** -16)
    again = [hca.decode_shared(**a, out_f32=True) for _ in range(20)]
    done()
    assert all(torch.equal(x, got) for x in again)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-(512 ** -0.5), 0.0])
def test_negative_and_zero_scale(cuda_device, libhca, scale):
    """Any finite logit scale: with a negative one a row's largest logit is its least product.  The third sequence sees a part of the
    prefix's last tile, the fourth none of it."""
    a = batch(cuda_device, 4, 4, 24, 700, 12, 33, [16 * 712 + 33, 16 * 705 + 40, 16 * 650 + 33, 40])
    a["scale"] = scale
    out, tol = reference(a)
    got = hca.decode_shared(**a, out_f32=True)
    done()
    check(got, out, tol, 2.0 ** -16)


def test_too_many_tiles_are_refused(libhca):
    """A batch whose caches hold 2^31 tiles of 128 rows or more is refused before anything is launched."""
    p = ctypes.c_void_p(16)

    def call(B, Nmax=0, mp=0):
        paged = _lib.HCA_PAGED if mp else 0
        a = (p if mp else None, 1 << 20 if mp else 0, mp, mp, p, p, p, None, None, 1e-6, None, None, None, 0, p, p, 1 << 62, B, 64, 1,
             512, 512, 128, 128)
        return (libhca.hca_decode_shared(p, p, p, p, p, *a, 4, Nmax, 0.05, paged, None),
                libhca.hca_decode_quant(p, p, p, p, *a, Nmax, 0.05, paged, None))
    for args in (dict(B=200, Nmax=0x7fffffff), dict(B=300, mp=2047), dict(B=1 << 24, Nmax=1 << 15)):
        assert call(**args) == (_lib.HCA_ERR_INVALID_ARG,) * 2


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
def test_a_refusal_leaves_the_workspace(cuda_device, libhca, norm):
    """... and leaves the caller's workspace alone."""
    dev, B, Np = cuda_device, 200, 40
    a = batch(dev, 5, B, 64, Np, 1, 16, [16 * Np + 20] * B)
    gain = torch.ones(512, device=dev)
    ws = torch.full((hca.decode_shared_workspace_size(B, 64, 1, 512, Np),), 0x5a, dtype=torch.uint8, device=dev)
    out = torch.zeros(B, 64, 512, dtype=bf, device=dev)
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    code = libhca.hca_decode_shared(P(a["q"]), P(a["kp"]), P(a["vp"]), P(a["kc"]), P(a["vc"]), None, 0, 0, 0, P(a["kw"]), P(a["vw"]),
                                    P(a["seqlens"]), P(gain), P(gain), 1e-6, None, None, None, 0, P(out), P(ws), ws.numel(), B, 64, 1,
                                    512, 512, 16, 16, Np, 0x7fffffff, 0.05, _lib.HCA_QK_NORM if norm else 0,
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    done()
    assert code == _lib.HCA_ERR_INVALID_ARG and bool((ws == 0x5a).all())


@pytest.mark.gpu
@pytest.mark.parametrize("W,ps", [(40, 0), (32, 64)])
def test_serving_on_a_shared_prefix(cuda_device, libhca, W, ps):
    """Token after token: append with the lengths behind the prefix, decode_shared with the full ones.  Every step against 64
    bits, and the same sequences through append and decode on caches of their own."""
    dev, blk, P, B, steps = cuda_device, 16, 20, 3, 130
    g = torch.Generator(device=dev).manual_seed(2)
    n0 = P * blk
    rb = lambda *s: torch.randn(s, generator=g, device=dev).to(bf)  # noqa: E731
    k, v, q = (torch.cat([rb(1, n0, 1, 512).expand(B, -1, -1, -1), rb(B, steps, 1, 512)], 1).contiguous() for _ in range(3))
    kp, vp = (t[0] for t in hca.compress(k[:1, :n0].contiguous(), v[:1, :n0].contiguous(), blk=blk))
    N = steps // blk + 1
    zeros = lambda *s: torch.zeros(s, dtype=bf, device=dev)  # noqa: E731
    state = lambda: torch.zeros(hca.append_state_size(B, 1, 512, 512), dtype=torch.uint8, device=dev)  # noqa: E731
    # on the shared prefix: position p in slot (p - n0) % W
    table = torch.randperm(B, generator=torch.Generator().manual_seed(1)).view(B, 1).to(torch.int32).to(dev) if ps else None
    kc, vc = (zeros(B, ps or N, 1, 512) for _ in range(2))
    kw, vw = (x[:, n0 - W:n0].contiguous() for x in (k, v))       # position n0 - W + i is in slot i
    st = state()
    # on caches of their own: position p in slot p % W
    full = [torch.cat([p[None].expand(B, -1, -1, -1), zeros(B, N, 1, 512)], 1).contiguous() for p in (kp, vp)]
    ring = [x[:, n0 - W:n0].roll(n0 % W, 1).contiguous() for x in (k, v)]
    st2 = state()
    seq = torch.full((B,), n0, dtype=torch.int32, device=dev)
    one = [torch.cat([p[None].expand(B, -1, -1, -1), hca.compress(*(x[:, n0:].contiguous() for x in (k, v)), blk=blk)[i]], 1)[:, :, 0]
           for i, p in enumerate((kp, vp))]
    for t in range(n0, n0 + steps):
        seq += 1
        kn, vn, qn = k[:, t].contiguous(), v[:, t].contiguous(), rb(B, 64, 512)
        hca.append(kn, vn, None, seq - n0, kw, vw, kc, vc, st, blk, page_table=table)
        hca.append(kn, vn, None, seq, ring[0], ring[1], full[0], full[1], st2, blk)
        if t % 7 and t < n0 + steps - 3:
            continue
        got = hca.decode_shared(qn, kp, vp, kc, vc, kw, vw, seq, blk, W, 512 ** -0.5, page_table=table, window_ring=True, out_f32=True)
        ref = hca.decode(qn, full[0], full[1], ring[0], ring[1], seq, blk, W, 512 ** -0.5, window_ring=True)
        done()
        nc = (t + 1 - W) // blk
        for b in range(B):
            # entries appended differ from the prompt's by a bf16 step at most: 2^-7 of them, in keys and values
            K = torch.cat([one[0][b, :nc], k[b, t + 1 - W:t + 1, 0]]).double()
            V = torch.cat([one[1][b, :nc], v[b, t + 1 - W:t + 1, 0]]).double()
            Q = qn[b].double()
            p = torch.softmax(Q @ K.T * 512 ** -0.5, -1)
            mass, d = p @ V.abs(), (Q.abs() @ K.abs().T * 512 ** -0.5).amax(-1, keepdim=True)
            own = p[:, P:max(P, nc)]
            step = 2.0 ** -7 * (own @ V[P:max(P, nc)].abs())
            moved = 2.0 ** -7 * torch.einsum("hn,hn->h", own, Q.abs() @ K[P:max(P, nc)].abs().T * 512 ** -0.5)[:, None] * 2 * mass
            for x in (got[b], ref[b]):
                check(x, p @ V, mass * (2.0 ** -7 + 2 * d * 2.0 ** -18 + 2.0 ** -16) + step + 1.2 * moved, 2.0 ** -16)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
def test_lengths_change_between_replays(cuda_device, libhca, norm):
    """A captured call follows the lengths on the device (both grids plan from them): short, long, mixed, padding rows."""
    dev, B, Np = cuda_device, 9, 300
    a = batch(dev, 6, B, 64, Np, 200, 40, [40] * B)
    if norm:
        a["gq"] = a["gk"] = torch.ones(512, device=dev)
    lens = [[40] * B, [16 * 500 + 40] * B, [16 * (Np + 25 * i) + 41 + i for i in range(B)], [0, 3, 16 * 301 + 40, 0, 16 * 499 + 40, 39, 40, 5000, 1]]
    want = []
    for n in lens:
        a["seqlens"].copy_(torch.tensor(n, dtype=torch.int32))
        want.append(hca.decode_shared(**a))
    done()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            got = hca.decode_shared(**a)
        for n, w in list(zip(lens, want)) * 2:
            a["seqlens"].copy_(torch.tensor(n, dtype=torch.int32))
            gr.replay()
            assert torch.equal(got, w)
    done()


@pytest.mark.gpu
def test_shared_beside_other_work(cuda_device, libhca):
    """Calls on three streams at once, one of them a prefill that fills the GPU: each has its own result."""
    dev = cuda_device
    a = [batch(dev, s, 6, 64, 500, 30, 40, [16 * (500 + 4 * i) + 50 for i in range(6)]) for s in range(2)]
    a[1]["gq"] = a[1]["gk"] = torch.ones(512, device=dev)
    g = torch.Generator(device=dev).manual_seed(9)
    q, k, v = (torch.randn(1, 2000, h, 512, generator=g, device=dev).to(bf) for h in (64, 1, 1))
    kc, vc = hca.compress(k, v, blk=16)
    calls = [lambda: hca.decode_shared(**a[0]), lambda: hca.decode_shared(**a[1]), lambda: hca.prefill(q, k, v, kc, vc, 16, 128, 512 ** -0.5)]
    want = [f() for f in calls]
    done()
    streams, got = [torch.cuda.Stream() for _ in calls], [[], [], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i]())
    done()
    for w, x in zip(want, got):
        assert all(torch.equal(y, w) for y in x)
