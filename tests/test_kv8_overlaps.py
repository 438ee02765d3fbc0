"""Outputs of tq_kv8_attention whose rows share memory with each other or with the queries are refused: host only."""
import ctypes

import pytest

from test_kv8_refusals import FAKE, INVALID, attention, cache, lib, rows  # noqa: F401 (lib: fixture)

Q = 1 << 20   # an address that is never looked at


def call(lib, q, out, batch=1, heads=4, L=4):
    return attention(lib, c=cache(num_blocks=64), q=rows(data=Q, **q), out=rows(**out), batch=batch, heads=heads, L=L)


@pytest.mark.parametrize("strides", [
    dict(stride_batch=4096, stride_head=0, stride_token=64),       # one row for all heads
    dict(stride_batch=4096, stride_head=256, stride_token=0),
    dict(stride_batch=0, stride_head=256, stride_token=64),
    dict(stride_batch=4096, stride_head=256, stride_token=32),     # rows half over the next one
    dict(stride_batch=4096, stride_head=256, stride_token=-32),
    dict(stride_batch=4096, stride_head=128, stride_token=64),     # a head's third token is the next head's first
    dict(stride_batch=1024 - 256, stride_head=256, stride_token=64),
    dict(stride_batch=4096, stride_head=64, stride_token=64),
    dict(stride_batch=4096, stride_head=64, stride_token=4 * 64 - 8),
])
def test_rows_of_out_over_each_other(lib, strides):  # noqa: F811
    assert call(lib, dict(stride_batch=4096, stride_head=256, stride_token=64), dict(data=Q + (1 << 18), **strides), batch=2) == INVALID


@pytest.mark.parametrize("strides,apart", [
    (dict(stride_batch=4096, stride_head=256, stride_token=64), 0),
    (dict(stride_batch=4096, stride_head=256, stride_token=64), 8),          # 16 bytes on
    (dict(stride_batch=4096, stride_head=256, stride_token=64), -64),        # a token back
    (dict(stride_batch=4096, stride_head=256, stride_token=64), 256),        # a head on
    (dict(stride_batch=4096, stride_head=256, stride_token=64), 4096 + 3 * 256 + 3 * 64 + 56),
    (dict(stride_batch=4096, stride_head=256, stride_token=64), -4096 - 3 * 256 - 3 * 64 - 56),
    (dict(stride_batch=2048, stride_head=64, stride_token=3 * 256), 128),    # two heads on, in a fused projection
    (dict(stride_batch=2048, stride_head=64, stride_token=3 * 256), 3 * 256 - 192),
])
def test_out_over_queries(lib, strides, apart):  # noqa: F811
    assert call(lib, strides, dict(data=Q + 2 * apart, **strides), batch=2) == INVALID
