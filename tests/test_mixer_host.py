"""Sizes of the mixer operators' workspaces, without a GPU."""
import ctypes

import pytest


def _lib():
    import long_sequence_fft_b200 as lsf
    return lsf.library()


def _norm_bytes(N, S, C, G, backward=1):
    return _lib().fftconv_group_norm_workspace_bytes(N, S, C, G, backward)


def _rows_written(N, G, D, V):
    """Rows of partial sums of the token form's backward pass with vectors of
    V elements: row blocks x rows of a block (0: another form)."""
    if D % V:
        return 0
    vecs, lanes, per = D // V, 1, 1
    while lanes < 32 and lanes < vecs:
        lanes *= 2
    while lanes * per < vecs:
        per *= 2
    if per > {8: 2, 4: 4, 1: 8}[V]:
        return 0
    groups = min(G, 256 // lanes)
    rows = min(256 // lanes // groups, N)
    columns = -(-G // groups)
    return min(-(-N // rows), max(1, 148 * 3 // columns)) * rows


@pytest.mark.parametrize("N", [1, 7, 250, 4100, 32768, 131072, 1 << 22])
@pytest.mark.parametrize("C,G", [(8, 1), (8, 8), (35, 7), (64, 64), (96, 4), (760, 8), (768, 12), (2048, 16),
                                 (4096, 32), (8192, 64), (256, 1), (130, 2), (51, 3), (65536, 512)])
def test_norm_workspace_is_what_the_rows_write(N, C, G):
    """Enough for every vector width, and no more than all resident blocks'
    rows: 8 bytes a channel and row, 256 threads x 8 channels a block."""
    rows = max(_rows_written(N, G, C // G, V) for V in (1, 4, 8))
    size = _norm_bytes(N, 1, C, G)
    assert size == -(-rows * 2 * C * 4 // 256) * 256
    assert size <= max(148 * 3, -(-C // 128)) * 256 * 8 * 8 + 256


def test_norm_workspace_of_a_wide_long_call():
    """32768 x 2048 values in 16 groups: a small part of the tensor's 134 MB."""
    assert _norm_bytes(32768, 1, 2048, 16) == 148 * 3 * 2 * 2048 * 4
    assert _norm_bytes(131072, 1, 8192, 64) <= 30 << 20
