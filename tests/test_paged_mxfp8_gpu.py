"""Attention over MXFP8 pages where codes, scales and weights are far apart, on each of its kernels
(few rows in tiles of 8 and of 16, many rows, CUDA cores), against the definition in 64 bits.  GPU only."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_gb300 as jfa
import serve_ref as ref
from test_paged_gpu import Batch, check_attention, f64, ragged

pytestmark = pytest.mark.gpu

# what serves it, batch, dtype, hq, hk, dqk, dv
KERNELS = [("rows8", "step", "bf16", 8, 2, 128, 128), ("rows8", "step", "bf16", 3, 1, 64, 128),
           ("rows16", "step", "bf16", 16, 1, 128, 64), ("rows16", "step", "bf16", 32, 2, 128, 128),
           ("tcgen05", "chunk", "bf16", 8, 2, 128, 128), ("tcgen05", "chunk", "bf16", 3, 1, 64, 64),
           ("CUDA cores", "step", "bf16", 4, 2, 96, 32), ("CUDA cores", "chunk", "f32", 4, 2, 64, 128)]
kernels = pytest.mark.parametrize("kernel", KERNELS, ids=["%s-%s-%s-%d-%d-D%d-%d" % k for k in KERNELS])


def batch(kernel, seed=0):
    _, kind, dtype, hq, hk, dqk, dv = kernel
    return Batch(*ragged(kind), hk, dqk, dv, 32, "mxfp8", dtype, seed=seed), hq


def decode(codes, scales):
    """Values of codes whose scale byte 0 makes them zeros."""
    zero = np.repeat(scales.cpu().numpy() == 0, 32, axis=-1)
    return np.where(zero, 0.0, ref.decode(codes.cpu().numpy(), scales.cpu().numpy()))


def set_scales(b, which, s):
    """Scale bytes of the owned rows of the keys or the values."""
    c, t = (b.cache.k, b.cache.k_scale) if which == "k" else (b.cache.v, b.cache.v_scale)
    t.copy_(torch.where(b.owned, s, 255).to(torch.uint8))
    setattr(b, which + "_h", decode(c, t))


@kernels
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("zeros", ["all", "blocks", "keys", "first keys", "some"])
def test_scales_of_zero_read_as_zeros(kernel, which, zeros):
    """Codes that are not zero behind scale bytes of 0: everywhere, in whole blocks of columns, in
    whole keys, in the first keys of a sequence (other scales come later), and here and there."""
    b, hq = batch(kernel)
    scale = b.cache.k_scale if which == "k" else b.cache.v_scale
    g = torch.Generator(device="cuda").manual_seed(2)
    low, high = ((1, 10) if zeros == "some" else (117, 122))
    s = torch.randint(low, high, scale.shape, generator=g, device="cuda", dtype=torch.int32)
    if zeros == "some":  # beside scales of about as little
        gone = torch.rand(s.shape, generator=g, device="cuda") < 0.5
    elif zeros == "all":
        gone = torch.ones_like(s, dtype=torch.bool)
    elif zeros == "blocks":
        gone = torch.zeros_like(s, dtype=torch.bool)
        gone[..., ::2] = True
    elif zeros == "keys":
        gone = torch.rand(s.shape[:-1] + (1,), generator=g, device="cuda").expand(s.shape) < 0.5
    else:
        gone = torch.zeros_like(s, dtype=torch.bool)
        for n, row in zip(b.lens_h, b.table_h):
            for j in range(-(-min(int(n), 70) // b.page)):
                gone[int(row[j]), :, :max(0, 70 - j * b.page)] = True
    set_scales(b, which, torch.where(gone, 0, s))
    check_attention(b, hq)
    # read back as zeros too
    k, v = jfa.jfa_cache_read(*b.args(), b.T, dtype=torch.float32)
    for x, of in ((k, b.k_of), (v, b.v_of)):
        for i in range(b.B):
            n, lo = int(b.lens_h[i]), int(b.offs_h[i])
            new = min(n, int(b.new[i]))
            if new:
                got = f64(x)[lo + int(b.new[i]) - new:lo + int(b.new[i])].transpose(1, 0, 2)
                assert np.array_equal(got, of(i)[:, n - new:].astype(np.float32).astype(np.float64))
