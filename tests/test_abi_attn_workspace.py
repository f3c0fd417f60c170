"""The workspace that attention calls demand, on the CPU: what plain attention needed
by itself, before scored attention and the NVFP4 cache came, is enough for it. (The
calls come back at the check behind the workspace's: their output is on q.)"""
import ctypes

import pytest

import nvfp4_block_scaled_gemv_amd as nv

ERR_WORKSPACE, ERR_ALIAS = 5, 7
BF16, E4M3 = 0, 2
A = [1 << 40 | i << 36 for i in range(1, 12)]


def records(rows, heads, D, tiles, waves):
    """Bytes of two records of every wavefront on the chip: a sum and a maximum, and
    D sums, of the rows of a head that it takes."""
    per_head = -(-rows // (16 * tiles))
    groups = max(1024 * waves // (heads * per_head), 1)
    n = 2 * groups * heads * per_head * min(rows, 16 * tiles)
    at = -(-n * 8 // 256) * 256
    return -(-(at + n * D * 4) // 256) * 256


def plain(rows, heads, D):
    """The largest of the plain caches' needs."""
    most = 0
    for size in (1, 2):
        for whole_runs in (False, True):
            tiles = 1 if rows <= 16 or (D == 256 and not whole_runs) else 2
            waves = 2 if tiles == 1 and D * size < 256 else 1
            most = max(most, records(rows, heads, D, tiles, waves))
    return most


SHAPES = [(G, Q, H, D) for D in (64, 128, 256) for H in (1, 2, 3, 8, 16) for G, Q in
          ((1, 1), (4, 1), (8, 1), (3, 3), (4, 5), (8, 4), (16, 3))]


def call(fn, cache, G, Q, H, D, nbytes, *scores):
    c = nv.KvCache(A[0], A[1], A[2], A[3], 40, 16, H, D, 16 * H * D, H * D, D, cache)
    return fn(A[4], ctypes.byref(c), A[5], A[6], 3, Q, G * H, 12, 0.1, 0, *scores, A[4], A[7],
              nbytes, None)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_plain_attention_takes_what_it_took(cache):
    L = nv.lib()
    for G, Q, H, D in SHAPES:
        need = plain(G * Q, H, D)
        assert call(L.nvfp4_paged_attention, cache, G, Q, H, D, need) == ERR_ALIAS, (G, Q, H, D)
        # without cap and bias it is the same call
        assert call(L.nvfp4_paged_attention_scored, cache, G, Q, H, D, need,
                    None) == ERR_ALIAS, (G, Q, H, D)
        assert call(L.nvfp4_paged_attention, cache, G, Q, H, D, 0) == ERR_WORKSPACE


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_the_query_is_enough_for_every_call(cache):
    L = nv.lib()
    cap = ctypes.byref(nv.AttnScores(30.0, None))
    for G, Q, H, D in SHAPES:
        n = nv.paged_attention_workspace_bytes(3, Q, G * H, H, D)
        assert n >= plain(G * Q, H, D)
        assert call(L.nvfp4_paged_attention, cache, G, Q, H, D, n) == ERR_ALIAS
        assert call(L.nvfp4_paged_attention_scored, cache, G, Q, H, D, n, cap) == ERR_ALIAS
        c = nv.KvCache4(A[0], A[1], A[2], A[3], A[8], A[9], 40, 16, H, D, 16 * H * D // 2,
                        H * D // 2, D // 2, 16 * H * D // 16, H * D // 16, D // 16)
        assert L.nvfp4_paged_attention_nvfp4(A[4], ctypes.byref(c), A[5], A[6], 3, Q, G * H, 12,
                                             0.1, 0, cap, A[4], A[7], n, None) == ERR_ALIAS


def test_two_heads_side_by_side_need_no_more_than_two_apart():
    """One pair of heads: its records are one a run and one a sequence."""
    for D in (64, 128, 256):
        for G in (1, 4, 8):
            n = nv.paged_attention_workspace_bytes(3, 1, 2 * G, 2, D)
            assert n == plain(G, 2, D)
