"""prefill where the rows' reference maxima move: logits that rise along the cache, so that unit after unit of 128 keys exceeds
every earlier one, against softmax attention in 64 bits."""
import pytest
import torch

import compressed_long_context_b200 as hca

bf = torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("step,rise", [(1, 12.0), (1, 36.0), (2, 20.0), (3, 40.0)])
def test_references_move(cuda_device, libhca, step, rise):
    """Half of the heads' logits rise by 2^rise every `step` units of entries, the other half's fall.  A unit that moves a
    reference is followed by units that weigh as much, so probabilities against an older reference would show; and the same
    bits again and again."""
    dev, T, Hq, blk, W = cuda_device, 4000, 16, 4, 64
    g = torch.Generator(device=dev).manual_seed(step)
    rb = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    axis = torch.zeros(512, device=dev)
    axis[:256] = 1.0
    scale = 512 ** -0.5
    level = (torch.arange(T, device=dev) // (128 * blk * step)).float() * rise * 0.6931471805599453 / (256 * scale)
    sign = torch.where(torch.arange(Hq, device=dev) % 2 == 0, 1.0, -1.0)
    q = (rb(1, T, Hq, 512) * 0.25 + sign[:, None] * axis).to(bf)
    k, v = (rb(1, T, 1, 512) + axis * level[:, None, None]).to(bf), rb(1, T, 1, 512).to(bf)
    kc, vc = hca.compress(k, v, blk=blk)
    got, lse = hca.prefill(q, k, v, kc, vc, blk, W, scale, want_lse=True, out_f32=True)
    for _ in range(10):
        again, lse2 = hca.prefill(q, k, v, kc, vc, blk, W, scale, want_lse=True, out_f32=True)
        assert torch.equal(again, got) and torch.equal(lse2, lse)
    torch.cuda.synchronize()
    hca.get_device_error()
    t = torch.arange(T, device=dev)[:, None]
    seen = torch.cat([torch.arange(kc.shape[1], device=dev)[None] < (t - W + 1).clamp(min=0) // blk,
                      (torch.arange(T, device=dev)[None] <= t) & (torch.arange(T, device=dev)[None] > t - W)], 1)
    K, V = torch.cat([kc[0, :, 0], k[0, :, 0]]).double(), torch.cat([vc[0, :, 0], v[0, :, 0]]).double()
    for h in range(Hq):
        Q = q[0, :, h].double()
        z = (Q @ K.T * scale).masked_fill(~seen, float("-inf"))
        p = torch.softmax(z, -1)
        # P and its sum are of bf16 terms (2^-8 each), logits fp32 sums (2^-18 of sum |q||k|)
        d = (Q.abs() @ K.abs().T * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
        mass = p @ V.abs()
        tol = mass * (2.0 ** -7 + 2 * d * 2.0 ** -18 + 2.0 ** -16) * (1 + 2.0 ** -16) + 1e-30
        assert bool(((got[0, :, h].double() - p @ V).abs() <= tol).all())
        want = torch.logsumexp(z, -1)
        # lse: a sum of fp32 exponentials and logits, and its own rounding
        assert bool(((lse[0, h].double() - want).abs() <= d[:, 0] * 2.0 ** -18 + 2.0 ** -16 + want.abs() * 2.0 ** -22).all())
