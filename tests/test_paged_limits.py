"""Sizes at the documented limits of the paged 4-bit cache, without a device."""
import ctypes

from test_paged_args import handle, lib


def test_workspace_bytes_at_the_limits():
    """Many sequences, long tables and an unknown number of queries: the work's
    bound passes 2^63, and the call still has the whole GPU."""
    for d in (64, 128, 256):
        h = handle(d)
        ws = lambda *a: lib.tq_paged_workspace_bytes(ctypes.byref(h), *a)   # noqa: E731
        full = ws(1024, 1, 65535, 1 << 18, 4096)
        for hq, hkv, batch, pages in [(1024, 1, 65535, 1 << 18), (1024, 1, 65535, (1 << 24) - 1), (1024, 2, 65535, 1 << 22)]:
            for most in (4096, 1 << 30, (1 << 31) - 1):
                assert ws(hq, hkv, batch, pages, most) == full, (d, hq, hkv, batch, pages, most)


def test_sequences_of_up_to_four_rounds_are_not_split():
    """A round is a tile for each of four warps: 64 tokens each, 32 at d = 256."""
    for d, tokens in ((64, 1024), (128, 1024), (256, 512)):
        h = handle(d, 16)
        ws = lambda *a: lib.tq_paged_workspace_bytes(ctypes.byref(h), *a)   # noqa: E731
        for heads, batch in ((1, 1), (8, 40)):
            assert ws(4 * heads, heads, batch, tokens // 16, 1) == 0 < ws(4 * heads, heads, batch, tokens // 16 + 1, 1), d
            assert ws(4 * heads, heads, batch, 512 // 16, 100) == 0 < ws(4 * heads, heads, batch, 512 // 16 + 1, 100), d
