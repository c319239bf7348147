"""The 8-bit cache at its edges: errors that meet, keys that are not finite, the largest values, and how far off QK normalisation
may be."""
import pytest
import torch

import compressed_long_context_b200 as hca
from compressed_long_context_b200 import _lib
from test_binding_host import stub  # noqa: F401
from test_quant import check, decode_case, done, z
from test_shared import make

bf, f8, e8 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["decode", "decode_quant", "decode_shared"])
def test_missing_slab_beside_a_bad_length(cuda_device, libhca, op):
    """A negative length is reported before any wait; a wait that runs out in the same call still marks every output."""
    dev, stream = cuda_device, torch.cuda.current_stream().cuda_stream
    if op == "decode_shared":
        a, out, tol = make(dev, 4, [16 * 400 + 60 + i for i in range(7)], 390, 64, 1, 16, 50)
    else:
        a, out, tol = decode_case(dev, 3, [16 * 300 + 50, 900, 16 * 200], 64, 1, 16, 40)
    if op == "decode":
        g = torch.Generator(device=dev).manual_seed(1)
        for n in ("kc", "vc"):
            a[n] = torch.randn(a[n].shape, generator=g, device=dev).to(bf)
        del a["sc"], a["vha_u"], a["vha_v"]
    call = getattr(hca, op)
    bad = a["seqlens"].clone()
    bad[1] = -5
    hca.get_device_error()
    try:
        assert libhca.hca_debug_set_wait_limit(2_000_000, stream) == _lib.HCA_OK      # 2 ms
        assert libhca.hca_debug_set_drop_slab(1, stream) == _lib.HCA_OK
        got = call(**{**a, "seqlens": bad})
        torch.cuda.synchronize()
        assert libhca.hca_get_device_error(stream) == _lib.HCA_ERR_TIMEOUT
        assert torch.isnan(got).all()
    finally:
        libhca.hca_debug_set_drop_slab(0, stream)
        libhca.hca_debug_set_wait_limit(0, stream)
    hca.get_device_error()
    call(**{**a, "seqlens": bad})
    torch.cuda.synchronize()
    assert libhca.hca_get_device_error(stream) == _lib.HCA_ERR_DEVICE_INPUT
    good = call(**a)
    done()
    if op != "decode":
        check(good, out, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,ps", [([16 * 257 + 40], 0), ([16 * 257 + 40] + [16 * 128 + 40] * 400, 0), ([16 * 129 + 40, 16 * 300], 64)])
def test_nan_key(cuda_device, libhca, lengths, ps):
    """The last entry of a sequence is the only one of its tile of 128, and its key is NaN (a pooled value that was not finite): the
    sequence's outputs are NaN, as the softmax is, whichever CTA holds the tile; the others' are right."""
    args, out, tol = decode_case(cuda_device, 3, lengths, 64, 1, 16, 40, ps=ps)
    n = (lengths[0] - 40) // 16
    at = (int(args["page_table"][0, (n - 1) // ps]), (n - 1) % ps) if ps else (0, n - 1)
    args["kc"].view(torch.uint8)[at[0], at[1], 0, 77] = 0x7f
    got = hca.decode_quant(**args)
    done()
    assert torch.isnan(got[0]).all()
    check(got[1:], out[1:], tol[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 400])
def test_shared_key_of_minus_infinity(cuda_device, libhca, B):
    """The only own entry's key has an infinite channel: heads whose logit becomes -inf leave it out, the others are NaN."""
    dev = cuda_device
    args, _, _ = make(dev, 3, [16 * 21 + 50] * B, 20, 8, 1, 16, 50)
    kc = args["kc"].clone()
    kc[:, 0, 0, 9] = float("-inf")
    args["q"][:, ::2, 9], args["q"][:, 1::2, 9] = 1.0, -1.0
    got = hca.decode_shared(**{**args, "kc": kc}, out_f32=True)
    done()
    K, V = (torch.cat([p[None, :, 0].expand(B, -1, -1), w[:, :, 0]], 1).double() for p, w in ((args["kp"], args["kw"]), (args["vp"], args["vw"])))
    Q = args["q"][:, ::2].double()
    p = torch.softmax(Q @ K.mT * args["scale"], -1)
    mass, d = p @ V.abs(), (Q.abs() @ K.abs().mT * args["scale"]).amax(-1, keepdim=True)
    assert torch.isnan(got[:, 1::2]).all()
    check(got[:, ::2], p @ V, mass * (2.0 ** -7 + 2 * d * 2.0 ** -18 + 2.0 ** -16), 2.0 ** -16)


def appended(k, w, blk):
    """(kc, sc) of the single sequence k [T, d], appended token by token as keys and values."""
    T, d = k.shape
    dev = k.device
    kw = torch.zeros(1, 4, 1, d, dtype=bf, device=dev)
    vw, vc = torch.zeros_like(kw), torch.zeros(1, T // blk, 1, d, dtype=torch.uint8, device=dev).view(f8)
    kc, sc = torch.zeros_like(vc.view(torch.uint8)).view(f8), torch.zeros(1, T // blk, 1, 2, dtype=torch.uint8, device=dev).view(e8)
    st = torch.zeros(hca.append_state_size(1, 1, d, d), dtype=torch.uint8, device=dev)
    for t in range(T):
        x = k[t].view(1, 1, d)
        hca.append_quant(x, x.clone(), None if w is None else w[t:t + 1], torch.tensor([t + 1], dtype=torch.int32, device=dev), kw, vw,
                         kc, vc, sc, st, blk)
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))
    return kc, sc


@pytest.mark.gpu
def test_largest_values_read_back(cuda_device, libhca):
    """Values up to bf16's largest, written at once or appended: entries read back finite, and 2^-4 of themselves off at most
    (the pooling: far less than 2^-12)."""
    dev = cuda_device
    top = torch.finfo(bf).max
    # each row's own largest value: below and above 248 * 2^120, where a code would round to 256
    mags = torch.tensor([top, 254 * 2.0 ** 120, 248 * 2.0 ** 120, 247 * 2.0 ** 120, 232 * 2.0 ** 120, 2.0 ** 127, 448 * 2.0 ** 119,
                         2.0 ** 100], device=dev)
    x = mags[:, None].expand(8, 64).clone()
    x[:, 1::2] *= -1
    x[:, 2::4] *= 0.37
    x = x.to(bf)
    for blk in (1, 5):
        rows = x.repeat_interleave(blk, 0)
        k = rows.view(1, -1, 1, 64)
        cases = [hca.compress_quant(k, k, blk=blk)]
        if blk == 1:
            kc, sc = appended(rows, None, blk)
            cases.append((kc, kc, sc))
        for kc, vc, sc in cases:
            back = hca.read_quant(kc, vc, sc, torch.tensor([8], dtype=torch.int32, device=dev), 8)
            done()
            for b in back:
                got, want = b[0, :, 0].double(), x.double()
                assert bool(torch.isfinite(got).all())
                assert bool(((got - want).abs() <= (2.0 ** -4 + 2.0 ** -12) * want.abs()).all())


@pytest.mark.gpu
def test_append_of_large_values(cuda_device, libhca):
    """128 tokens of 2^120 with equal weights are within the pool's range: the entry of the whole prompt."""
    dev, blk = cuda_device, 128
    x = torch.full((blk, 64), 2.0 ** 120, device=dev).to(bf)
    x[:, ::3] = -1.5 * 2.0 ** 119
    a = hca.compress_quant(x.view(1, blk, 1, 64), x.view(1, blk, 1, 64), blk=blk)
    kc, sc = appended(x, torch.full((blk,), 0.25, device=dev), blk)
    done()
    assert torch.equal(kc.view(torch.uint8), a[0].view(torch.uint8)) and torch.equal(sc.view(torch.uint8), a[2].view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("order", [0, 1])
def test_value_scales_far_apart(cuda_device, libhca, order):
    """Value scales 2^100 apart, in tiles of their own: every key keeps its weight in the others' sums."""
    dev = cuda_device
    args, _, _ = decode_case(dev, 7, [16 * 512 + 40] * 160, 64, 1, 16, 40)
    sc = args["sc"].view(torch.uint8)
    small = (torch.arange(512, device=dev) // 128) % 2 == order
    sc[:, :, 0, 1] = torch.where(small, 127 - 40, 127 + 60).to(torch.uint8)
    got = hca.decode_quant(**args, out_f32=True)
    done()
    for b in (0, 77, 159):
        val = lambda c, i: c[b, :, 0].float().double() * torch.pow(2.0, sc[b, :, 0, i:i + 1].double() - 127)  # noqa: E731
        K, V = (torch.cat([val(args[n], i), args[w][b, :, 0].double()]) for i, (n, w) in enumerate((("kc", "kw"), ("vc", "vw"))))
        Q = args["q"][b].double()
        p = torch.softmax(Q @ K.T * args["scale"], -1)
        d = (Q.abs() @ K.abs().T * args["scale"]).amax(-1, keepdim=True)
        check(got[b], p @ V, (p @ V.abs()) * (2.0 ** -7 + 2 * d * 2.0 ** -18 + 2.0 ** -16), 2.0 ** -16)


# ------------------------------------------------------------------ QK normalisation, as exactly as it is held
#
# One-hot values, so that an output is a key's probability.  A logit is a sum of 512 products, each off by a share of itself with
# its own sign: 6 times the 2-norm of the bounds is passed with probability 2 exp(-18), and the root mean square of a rounding is
# at most its bound / sqrt(3).  One probability is off by p_j (delta_j + sum p delta) to first order (1.2 times while delta <=
# 0.1); over all keys the root mean square counts delta_j and the row's mean as if they were independent, at most: twice the square.

def heads_and_keys(args, b, keys):
    """q / rms(q) * gq * gk of the heads and k / rms(k) of the keys, in 64 bits."""
    unit = lambda x: x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    return unit(args["q"][b].double()) * (args["gq"] * args["gk"]).double(), unit(keys.double())


def rounded(Q, K, scale, rel, low=0.0):
    """(2-norm, 1-norm) bounds of the logits for products off by `rel` of themselves, and queries off by `low` of their largest."""
    two = rel ** 2 * (Q ** 2 @ (K ** 2).T)
    if low:
        two = two + (low * Q.abs().amax(-1, keepdim=True)) ** 2 * (K ** 2).sum(-1)
    return torch.sqrt(two) * scale, 2.0 ** -18 * (Q.abs() @ K.abs().T) * scale


def two_terms(Q, lo=True):
    """The query as two e4m3 terms, scaled so that its largest value lies in (224, 448]."""
    e = torch.ceil(torch.log2(Q.abs().amax(-1, keepdim=True) / 448))
    x = Q * torch.pow(2.0, -e)
    hi = x.float().to(f8).double()
    return (hi + ((x - hi).float().to(f8).double() if lo else 0)) * torch.pow(2.0, e)


QUANT_REL, QUANT_LOW = 2.0 ** -8 + 2.0 ** -11, 2.0 ** -10 / 224      # e4m3 of e4m3's rest, from fp16; below its normal range


def quant_norm_case(dev):
    """A sequence of 400 8-bit entries and a window of 60, QK normalisation: (args, keys, probabilities, bounds)."""
    args, out, _ = decode_case(dev, 9, [16 * 400 + 60], 64, 1, 16, 60, norm=True, onehot=True)
    sc = args["sc"].view(torch.uint8)[0, :, 0].double() - 127
    K = torch.cat([args["kc"][0, :, 0].float().double() * torch.pow(2.0, sc[:, :1]), args["kw"][0, :, 0].double()])
    Q, K = heads_and_keys(args, 0, K)
    p = torch.softmax(Q @ K.T * args["scale"], -1)
    v = torch.cat([torch.pow(2.0, sc[:, 1]), torch.ones(60, dtype=torch.float64, device=sc.device)])      # the one-hot values
    two, one = rounded(Q, K, args["scale"], QUANT_REL, QUANT_LOW)
    return args, Q, K, p, v, two, one


def quant_norm_check(got, p, v, two, one):
    """got [heads, keys]: probabilities times values."""
    delta = 6 * two + one
    assert float(delta.max()) <= 0.1
    lost = 2.0 ** -17 * (p * v).amax(-1, keepdim=True)                    # p held in two 8-bit terms (a code of 1 per key)
    tol = 1.2 * (p * delta + (p * delta).sum(-1, keepdim=True) * p) * v + p * v * (2.0 ** -7 + 2.0 ** -16) + lost
    err = (got - p * v).abs()
    # 2-norm: 2^-7 / sqrt(3) for the two terms of p, and what keys lose whose value lies far below the row's largest (a key 2^30
    # below, as here, has p v below 2^-17 of the row's largest altogether and may be lost whole: 2^-17 max(p v) >= p v)
    limit = torch.sqrt(((p * v) ** 2 * (2 * two ** 2 / 3 + 2.0 ** -14 / 3) + lost ** 2).sum())
    rms = torch.sqrt((err ** 2).sum())
    return float((err / tol).max()), float(rms / limit)


def of_channels(got, n, w):
    """[heads, keys] of one-hot outputs: entry j in channel j, window slot i in channel 511 - i."""
    return torch.cat([got[:, :n], got[:, 512 - w:].flip(-1)], -1).double()


def test_norm_bound_sees_the_low_term():
    """The bound holds for the query as the kernel keeps it, and not without its low term."""
    args, Q, K, p, v, two, one = quant_norm_case(torch.device("cpu"))
    both, high = (quant_norm_check(torch.softmax(two_terms(Q, lo) @ K.T * args["scale"], -1) * v, p, v, two, one) for lo in (True, False))
    assert both[0] <= 1 and both[1] <= 1
    assert high[0] > 1 and high[1] > 2


@pytest.mark.gpu
def test_norm_query_is_held_in_eight_bits(cuda_device, libhca):
    args, Q, K, p, v, two, one = quant_norm_case(cuda_device)
    got = hca.decode_quant(**args, out_f32=True)
    done()
    worst, rms = quant_norm_check(of_channels(got[0], 400, 60), p, v, two, one)
    assert worst <= 1 and rms <= 1, (worst, rms)


SHARED_REL = 2.0 ** -10.5                                             # fp16 queries and keys: 2^-11 each


def shared_norm_case(dev):
    """Two sequences wholly behind a prefix of 400 entries, QK normalisation: (args, [Q, K, p, 2-norm, 1-norm] of each)."""
    args, _, _ = make(dev, 8, [16 * 402 + 40, 16 * 401 + 40], 400, 64, 1, 16, 40, norm=True, onehot=True)
    rows = []
    for b in range(2):
        Q, K = heads_and_keys(args, b, torch.cat([args["kp"][:, 0], args["kc"][b, :2 - b, 0], args["kw"][b, :, 0]]))
        rows.append((Q, K, torch.softmax(Q @ K.T * args["scale"], -1)) + rounded(Q, K, args["scale"], SHARED_REL))
    return args, rows


def shared_norm_check(got, p, two):
    """got [heads, prefix keys]: their probabilities, each rounded to bf16 (2^-8 / sqrt(3)); the part of the others in the sum is off
    by their own 2^-8, which all of a row share."""
    n = got.shape[-1]
    err = ((got - p[:, :n]) ** 2).sum()
    limit = (p[:, :n] ** 2 * (2 * two[:, :n] ** 2 / 3 + 2.0 ** -16 / 3 + (2.0 ** -8 * p[:, n:].sum(-1, keepdim=True)) ** 2)).sum()
    return float(torch.sqrt(err / limit))


def test_norm_bound_sees_sixteen_bit_operands():
    """The bound holds for fp16 queries and keys and P in bf16, and not for bf16 queries and keys."""
    args, rows = shared_norm_case(torch.device("cpu"))
    for Q, K, p, two, _ in rows:
        def sim(t):
            z = (Q.to(t).double() @ K.to(t).double().T) * args["scale"]
            e = torch.exp(z - z.amax(-1, keepdim=True)).to(bf).double()
            return (e / e.sum(-1, keepdim=True))[:, :400]
        assert shared_norm_check(sim(torch.float16), p, two) <= 1 < shared_norm_check(sim(bf), p, two)


@pytest.mark.gpu
def test_norm_prefix_is_held_in_eleven_bits(cuda_device, libhca):
    args, rows = shared_norm_case(cuda_device)
    got = hca.decode_shared(**args, out_f32=True)
    done()
    for b, (_, _, p, two, _) in enumerate(rows):
        rel = shared_norm_check(got[b, :, :400].double(), p, two)
        assert rel <= 1, rel


def test_arguments_of_the_wrong_kind(stub):  # noqa: F811
    """What is not a tensor is a TypeError and a wrong number of dimensions a ValueError, before anything reaches the library; a
    prefix that still has its batch dimension would have been read as one entry."""
    B, W, i32 = 2, 9, torch.int32
    cache = dict(kc=z(B, 7, 1, 512, dtype=f8), vc=z(B, 7, 1, 512, dtype=f8), sc=z(B, 7, 1, 2, dtype=e8))
    window = dict(kw=z(B, W, 1, 512), vw=z(B, W, 1, 512), seqlens=z(B, dtype=i32))
    step = dict(q=z(B, 64, 512), blk=16, W=W, scale=0.1, workspace=z(64, dtype=torch.uint8), **window)
    own = dict(kc=z(B, 7, 1, 512), vc=z(B, 7, 1, 512))
    calls = {
        "compress_quant": (dict(k=z(B, 32, 1, 64), v=z(B, 32, 1, 64), blk=16), [("k", z(B, 32, 64)), ("v", z(B, 32, 64))]),
        "append_quant": (dict(k_new=z(B, 1, 512), v_new=z(B, 1, 512), w_new=None, state=torch.zeros(1028 * B), blk=16, **cache, **window),
                         [("k_new", z(B, 512)), ("v_new", z(512)), ("kw", z(9)), ("kc", z(9, dtype=f8)), ("page_table", z(4, dtype=i32))]),
        "read_quant": (dict(counts=z(B, dtype=i32), n=3, **cache), [("kc", z(7, 512, dtype=f8)), ("vc", z(7, dtype=f8)),
                                                                    ("page_table", z(4, dtype=i32))]),
        "decode_quant": (dict(**step, **cache), [("q", z(B, 512)), ("kc", z(7, 512, dtype=f8)), ("vc", z(7, 512, dtype=f8)),
                                                 ("kw", z(B * W * 512)), ("page_table", z(4, dtype=i32))]),
        "decode_shared": (dict(kp=z(5, 1, 512), vp=z(5, 1, 512), **step, **own),
                          [("q", z(B, 512)), ("kp", z(1, 5, 1, 512)), ("vp", z(1, 5, 1, 512)), ("kp", z(5, 512)), ("kc", z(7, 512)),
                           ("vw", z(B * W * 512)), ("page_table", z(4, dtype=i32))]),
    }
    for name, (good, bad) in calls.items():
        call = getattr(hca, name)
        call(**good)
        n = len(stub.calls)
        for arg, t in bad:
            with pytest.raises(ValueError):
                call(**{**good, arg: t})
            with pytest.raises(TypeError):
                call(**{**good, arg: t.tolist() if t.dtype in (bf, i32) else "codes"})
        assert len(stub.calls) == n
    a = {**calls["decode_shared"][0], "kp": z(1, 5, 1, 512), "vp": z(1, 5, 1, 512)}      # both with the batch dimension
    with pytest.raises(ValueError, match="kp"):
        hca.decode_shared(**a)
