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


# ---- queries of another rank ------------------------------------------------------

def _host_args():
    """Arguments of the right shapes in host memory: enough for the shape checks."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    pool = pkv.Pool(torch.zeros(4, 1, 16, 2, 64), torch.zeros(4, 1, 16, 2, 64))
    bounds = pkv.BlockBounds.for_pool(pool)
    return pool, bounds, i


@pytest.mark.parametrize("shape", [(3,), (3, 256), (1, 3, 4, 64), ()])
def test_queries_of_another_rank(shape):
    pool, bounds, i = _host_args()
    q = torch.zeros(shape)
    with pytest.raises(ValueError):
        pkv.select_blocks(pool, 0, bounds, q, i(2, 4), None, i(3), i(3), i(3, 2, 4), i(3, 2))
    with pytest.raises(ValueError):
        pkv.decode_attention_sparse(pool, 0, q, 0.1, i(2, 4), None, i(3), i(3), i(3, 2, 4),
                                    torch.zeros(3, 4, 64))
    k = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        pkv.rope_append(pool, 0, pkv.Rope(64), i(2, 4), None, i(3), i(3), q, k, k,
                        torch.zeros(3, 4, 64))


@pytest.mark.parametrize("bad", ["block_tables", "token_seq"])
def test_index_tensors_of_another_rank(bad):
    pool, bounds, i = _host_args()
    bt = i(8) if bad == "block_tables" else i(2, 4)
    seq = i(3, 1) if bad == "token_seq" else i(3)
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        pkv.select_blocks(pool, 0, bounds, q, bt, None, seq, i(3), i(3, 2, 4), i(3, 2))
    with pytest.raises(ValueError):
        pkv.decode_attention_sparse(pool, 0, q, 0.1, bt, None, seq, i(3), i(3, 2, 4),
                                    torch.zeros(3, 4, 64))
    with pytest.raises(ValueError):
        pkv.rope_append(pool, 0, pkv.Rope(64), bt, None, seq, i(3), q, k, k, torch.zeros(3, 4, 64))
    with pytest.raises(ValueError):
        pkv.update_block_bounds(pool, 0, bounds, bt, i(2, 1) if bad == "token_seq" else i(2), None)


# ---- the current stream ---------------------------------------------------------------

def test_a_pool_in_host_memory_has_no_stream():
    pool, bounds, i = _host_args()
    with pytest.raises(ValueError):
        pkv.update_block_bounds(pool, 0, bounds, i(2, 4), i(2), None)


def test_the_stream_without_torchs_short_cut(monkeypatch):
    """A torch that has no call for the handle alone: the documented one is used."""
    from paged_kv_cache_blk_gb300 import _binding as B

    class Stream:
        cuda_stream = 1234

    seen = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: seen.append(d) or Stream())
    monkeypatch.setattr(B, "_raw_stream", None)
    dev = torch.device("cuda", 0)
    assert B._stream(dev) == 1234 and seen == [dev]


def test_import_without_torchs_short_cut():
    import subprocess
    import sys
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "from paged_kv_cache_blk_gb300 import _binding as B\n"
            "assert B._raw_stream is None\n")
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0
