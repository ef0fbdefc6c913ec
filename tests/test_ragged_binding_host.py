"""Refusals of the ragged-batch binding that need no GPU."""
import pytest
import torch

import speculative_decoding_fc_gb300 as ds


def _tensors():
    q = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16)
    kc = torch.zeros((1, 16, 2, 128), dtype=torch.bfloat16)
    return q, kc, torch.zeros((1, 2, 16)), torch.ones(1, dtype=torch.int32)


@pytest.mark.parametrize("x", [(1 << 32) + 5, 1 << 31, -(1 << 31) - 1, 1 << 62])
def test_sizes_past_32_bits_are_refused_not_cut_off(x):
    q, kc, sc, lens = _tensors()
    for call in (lambda: ds.window_attention(q, kc, kc, lens, x),
                 lambda: ds.window_attention(q, kc, kc, lens, 4, sinks=x),
                 lambda: ds.cache_evict(kc, kc, sc, lens, x),
                 lambda: ds.cache_evict(kc, kc, sc, lens, 8, sinks=x),
                 lambda: ds.cache_evict(kc, kc, sc, lens, 8, recent=x)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ds._on(0, Stream())


def test_outputs_share_no_memory():
    x = torch.zeros(100)
    ds._apart(x[:50], "out", x[50:])
    for a, b in ((x, x), (x[:51], x[50:]), (x[50:], x[:51]), (x[10:20], x)):
        with pytest.raises(ValueError, match="out overlaps"):
            ds._apart(a, "out", b)
