"""The 8-bit cache at its edges: errors that meet, keys that are not finite, the largest values, and how far off QK normalisation
may be."""
import pytest
import torch

import compressed_long_context_b200 as hca
from compressed_long_context_b200 import _lib
from test_quant import check, decode_case, done
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
