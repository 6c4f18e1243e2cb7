"""What the binding refuses before it calls the library, without a GPU."""

import pytest
import torch

import paged_kv_cache_blk_gb300 as pkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv.build()
    return pkv.load()


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="base"),
                                dict(scaling="by_parts", factor=4.0, original_len=4096.0),
                                dict(factor=4.0), dict(scaling="other")])
def test_frequencies_and_a_schedule_do_not_go_together(kw):
    with pytest.raises(ValueError):
        pkv.Rope(8, inv_freq=[1.0, 0.5, 0.25, 0.125], **kw)
