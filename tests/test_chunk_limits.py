"""CPU: sizes of chunk attention whose line of work could pass 64 bits are refused whatever the
offsets say: offsets that fall may give every second sequence all of the rows."""
import ctypes

import pytest

from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvDims, lib

UNSUPPORTED = -2
P = 1 << 20          # an address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def line(tokens, seqs, heads, group, blocks):
    """Length of the line with offsets 0, tokens, 0, tokens, ... and full contexts."""
    tt = 2 * (128 // group)
    ctx = 16 * blocks
    before, units = max(ctx - tokens, 0), -(-tokens // tt)
    one = (units - 1) * (before + 128) + tt * ((units - 1) * units // 2) + before + tokens + 128
    return (seqs + 1) // 2 * heads * one


@pytest.mark.parametrize("tokens,seqs,heads,group,blocks", [
    (2 ** 31 - 1, 8192, 1, 1, 1), (2 ** 31 - 1, 8192, 1, 1, 1 << 18), (2 ** 28, 8192, 8, 8, 1 << 20), (2 ** 30, 8192, 2, 3, 4)])
def test_refused(tokens, seqs, heads, group, blocks):
    d = PkvDims(seqs, heads * group, heads, 64, 16, 8, blocks, 0)
    assert line(tokens, seqs, heads, group, blocks) > 2 ** 63
    assert lib().paged_chunk_attention(P, P, P, P, P, P, tokens, 1.0, P, P, 1 << 40, ctypes.byref(d), 0) == UNSUPPORTED


def test_every_accepted_size_is_counted_in_64_bits():
    """The host's rule, for sizes on its border."""
    for tokens in (1, 31, 1000, 10 ** 6, 2 ** 31 - 1):
        for seqs in (1, 2, 3, 100, 8192):
            for group in range(1, 9):
                for blocks in (0, 1, 1 << 12, 1 << 26):
                    rule = seqs * (tokens / 32 + 1) * (16 * blocks + tokens + 256)
                    heads = int(4e18 / rule)
                    assert line(tokens, seqs, heads, group, blocks) < 2 ** 63
