"""Sizes of the delta rule's and the group norm's workspaces at the edges of what the header admits (CPU only)."""
import os

import pytest

from selective_scan_ssm_amd import _lib

F32, BF16 = 0, 1
BAD = (1 << 64) - 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from selective_scan_ssm_amd import build
        build.build()
    return _lib.load()


def whole(slots, heads):
    """The workspace of sequences that are not cut in time: per chunk and head T and P (12 KB each) and 192 floats."""
    return 2 * 12288 * slots * heads + 768 * slots * heads


# most of the sequences empty, one of millions of steps: the pass over the segments' ends has two or three workgroups of
# 256 (fp32) or 320 lanes to a border between two segments, the walk over the segments one to each and to each sequence
@pytest.mark.parametrize("io,dk,seqlen,nseq", [(BF16, 8, 7_000_000, 7_300_000), (F32, 72, 7_000_000, 7_300_000), (BF16, 72, 7_000_000, 5_000_000),
                                               (BF16, 128, 7_000_000, 7_300_000)])
def test_segments_fit_a_launch(lib, io, dk, seqlen, nseq):
    slots = seqlen // 64 + nseq
    need = lib.ssm_delta_scan_workspace_bytes(1, seqlen, 1, nseq, 1, 1, dk, 8, io)
    assert need != BAD
    groups, lanes, keys = 1 + (1 if dk <= 64 else 2), 256 if io == F32 else 320, 64 if dk <= 64 else 128
    borders = (need - whole(slots, 1)) // (8 * dk * 4 + keys // 32 * (keys // 16) * 2048)
    assert groups * lanes * borders < 1 << 32 and lanes * (nseq + borders) < 1 << 32


def test_fewer_are_cut(lib):
    need = lib.ssm_delta_scan_workspace_bytes(1, 3_800_000, 1, 1000, 1, 1, 8, 8, BF16)
    assert need != BAD and need > whole(3_800_000 // 64 + 1000, 1) + 1000 * 256


@pytest.mark.parametrize("io,dk", [(F32, 64), (F32, 128), (BF16, 64), (BF16, 128)])
def test_sequences_under_twelve_chunks_stay_whole(lib, io, dk):
    """Their results are then the same between others, cut or not."""
    for batch, T in ((1, 64), (1, 705 - 1), (3, 704)):
        need = lib.ssm_delta_scan_workspace_bytes(batch, T, 0, 0, 4, 4, dk, dk, io)
        assert 0 <= need - whole(batch * -(-T // 64), 4) < 3 * 256
    chunks = 16
    need = lib.ssm_delta_scan_workspace_bytes(1, 64 * chunks, 0, 0, 4, 4, dk, dk, F32)
    # fp32: two chunks to a segment, or one; a state and a transition where one ends that is not the last
    ends = (need - whole(chunks, 4)) // (4 * (dk * dk * 4 + (dk // 32) * (dk // 16) * 2048))
    assert ends >= 7


@pytest.mark.parametrize("io", [F32, BF16])
def test_sequences_that_are_not_cut_keep_nothing_at_their_ends(lib, io):
    """A state and a transition are kept between two segments of a sequence, of which eight chunks make one at least."""
    seqlen, nseq = 41000, 300
    slots = seqlen // 64 + nseq
    need = lib.ssm_delta_scan_workspace_bytes(1, seqlen, 1, nseq, 2, 2, 64, 64, io)
    assert whole(slots, 2) < need <= whole(slots, 2) + slots // 8 * 2 * (64 * 64 * 4 + 2 * 4 * 2048) + 5 * 256


# (batch, rows, dim, groups): a layer norm of wide rows, two rows to an entry, a narrow map, head norms
@pytest.mark.parametrize("N,R,C,groups", [(16384, 1, 5120, 1), (65536, 2, 4096, 1), (16384, 1, 2048, 1), (1 << 20, 4, 96, 8), (1 << 20, 1, 1536, 12),
                                          (1 << 16, 64, 256, 2)])
def test_the_gradient_keeps_no_partial_sums_per_entry(lib, N, R, C, groups):
    """What the partial sums take is a part of x, not more than it."""
    need = lib.ssm_group_norm_bwd_workspace_bytes(N, R, C, groups)
    assert need != BAD and need <= N * R * C * 2 // 2
