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


def scored(b, scores, g):
    """Keys and queries whose scores (scale 1) are `scores` [pages, hk, page] for all heads, given
    as values that a code of scale 1 holds; the other columns meet zeros."""
    b.cache.k.zero_()
    b.cache.k[..., 0] = scores.to(torch.float8_e4m3fn).view(torch.uint8)
    set_scales(b, "k", torch.full_like(b.cache.k_scale, 127, dtype=torch.int32))
    b.cache.k.copy_(torch.where(b.owned, b.cache.k, 0x7f))
    q = torch.zeros(b.T, b.cache.heads, b.dqk, device="cuda")
    q[..., 0] = 1
    return q


@kernels
@pytest.mark.parametrize("gap", [(10, 18), (0, 12), (18, 40), (60, 84), (10, 84)])
@pytest.mark.parametrize("scales", [(120, 120), (112, 121), (100, 127)])
def test_small_weights_beside_a_key_of_zero_value(kernel, gap, scales):
    """One key with nearly all the weight and a value of zero, the others `gap` nats below it: a
    column is the sum of small weights alone, and keeps its precision relative to that sum."""
    b, hq = batch(kernel, seed=6)
    g = torch.Generator(device="cuda").manual_seed(7)
    # whole and half numbers up to 15 have codes, and multiples of 4 to 60
    step = 0.5 if gap[1] - gap[0] <= 12 else 4.0
    top = 8.0 if gap[1] <= 18 else 48.0
    n = int((gap[1] - gap[0]) / step) + 1
    low = top - gap[0] - step * torch.randint(0, n, b.cache.k.shape[:3], generator=g, device="cuda")
    low = low.to(torch.float8_e4m3fn).float()
    s = torch.randint(scales[0], scales[1] + 1, b.cache.v_scale.shape, generator=g, device="cuda", dtype=torch.int32)
    for n, row in zip(b.lens_h, b.table_h):
        if n:  # the sequence's first key
            low[int(row[0]), :, 0] = top
            b.cache.v[int(row[0]), :, 0] = 0
    q = scored(b, low, g)
    set_scales(b, "v", s)
    b.k_h = decode(b.cache.k, b.cache.k_scale)
    q = q[:, :1].expand(-1, hq, -1).to(torch.bfloat16 if b.dtype == "bf16" else torch.float32).contiguous()
    check_attention(b, hq, q=q, scale=1.0)


@kernels
@pytest.mark.parametrize("low,high,size", [(215, 235, -100), (225, 235, -118), (230, 236, -60), (27, 40, 90)])
def test_keys_of_any_size_against_queries_of_the_other(kernel, low, high, size):
    """Huge keys and tiny queries, and the other way round: only a score itself may leave fp32."""
    b, hq = batch(kernel, seed=8)
    g = torch.Generator(device="cuda").manual_seed(9)
    set_scales(b, "k", torch.randint(low, high + 1, b.cache.k_scale.shape, generator=g, device="cuda", dtype=torch.int32))
    q = torch.randn(b.T, hq, b.dqk, generator=g, device="cuda") * 2.0 ** size
    mid = 2.0 ** -((low + high) // 2 - 127 + size + 10)
    check_attention(b, hq, q=q.to(torch.bfloat16 if b.dtype == "bf16" else torch.float32), scale=mid)
