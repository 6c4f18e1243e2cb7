"""The rotary append of long lists: with 16 tasks an SM (2432 on 152 SMs) or more
tokens a warp takes a whole token, its q, key and value rows one after the other."""

import pytest

import paged_kv_cache_blk_gb300 as pkv

from gpu_util import need_gpu
from test_gpu_rope import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,H,G,D,rd", [
    ("bf16", 2, 4, 128, 128), ("bf16", 3, 3, 64, 32), ("bf16", 1, 1, 256, 200), ("bf16", 1, 1, 32, 32),
    ("f32", 2, 2, 64, 64), ("f32", 1, 7, 128, 96), ("i8", 2, 4, 128, 128), ("i8", 5, 1, 64, 24),
    ("i8", 1, 2, 256, 256),
])
def test_prompts(dev, dtype, H, G, D, rd, inter):
    _run(dev, dtype, H, G, D, rd, inter, bs=64, lens=[2700, 1, 999, 64], seed=141)


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
@pytest.mark.parametrize("n", [1200, 2430, 2435, 4900])
def test_around_one_task_a_token(dev, dtype, n):
    """Token counts on both sides of the one from which a token is one task."""
    _run(dev, dtype, 2, 2, 64, 64, False, bs=64, lens=[n], seed=151)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
def test_in_place(dev, dtype):
    _run(dev, dtype, 2, 3, 128, 64, True, bs=64, lens=[3100, 17], in_place=True, seed=161)
