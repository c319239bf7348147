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
