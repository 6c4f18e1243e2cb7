"""Key bounds of blocks whose elements differ by more than fp32 has exponents: an
element whose quotient by the unit is below every fp32 number is still rounded
outwards, to a code of 1 or -1."""

import numpy as np
import pytest
import torch

import paged_kv_cache_blk_gb300 as pkv

from gpu_util import dev_batch, need_gpu
from test_gpu_sparse import _case, _check_bounds, _layer_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


def _update(dev, w, spec, pool):
    bounds = pkv.BlockBounds.for_pool(pool)
    bounds.codes.fill_(7)
    bounds.scales.fill_(-3.0)
    before = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    pkv.update_block_bounds(pool, w.layer, bounds, bt, ln, offs)
    _check_bounds(bounds, before, w, spec, _layer_values(pool.k_cache, spec, w.layer))
    return bounds


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_elements_far_below_the_unit(dev, dtype, D):
    w, spec, pool = _case(dev, dtype, 1, D, 4, [4] * 6, 151, offsets=False, num_layers=1, layer=0)
    smallest = 2.0 ** (-133 if dtype == "bf16" else -149)
    small = [2.0 ** -100, 2.0 ** -111, 2.0 ** -120, 2.0 ** -126, 2.0 ** -130, smallest]
    k = torch.zeros_like(pool.k_cache)
    for b, top in enumerate([2.0 ** 26, 2.0 ** 40, 2.0 ** 46, 2.0 ** 60, 2.0 ** 120, -2.0 ** 50]):
        blk = int(w.batch.block_tables[b, 0])
        k[blk, 0, 1, 0, 0] = top
        for i, x in enumerate(small):
            k[blk, 0, :, 0, 4 + 2 * i] = x       # a bound from above needs the code 1,
            k[blk, 0, :, 0, 5 + 2 * i] = -x      # one from below the code -1
    pool.k_cache.copy_(k)
    bounds = _update(dev, w, spec, pool)
    codes = bounds.codes[int(w.batch.block_tables[3, 0]), 0, 0].cpu().numpy().astype(int) - 128
    assert np.all(codes[0, 4:16:2] == 1) and np.all(codes[1, 5:16:2] == -1)
    assert not codes[1, 4:16:2].any() and not codes[0, 5:16:2].any()


def test_int8_scales_far_below_the_unit(dev):
    H, D = 2, 64
    w, spec, pool = _case(dev, "i8", H, D, 8, [8, 5], 152, offsets=False)
    k = pool.k_cache
    scales = k[..., H * D:H * D + 4 * H].view(torch.float32)
    blk = int(w.batch.block_tables[0, 0])
    scales[blk, w.layer] = 2.0 ** -118
    k[blk, w.layer, :, :H * D] = 129             # codes 1: every element 2^-118
    k[blk, w.layer, 3, ::2] = 128                # but a row of 0 and 2^60 elements
    scales[blk, w.layer, 3] = 2.0 ** 60
    k[blk, w.layer, 3, 0] = 255
    k[blk, w.layer, 3, D] = 255
    _update(dev, w, spec, pool)
