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


def _attention_bytes(backward, **kw):
    from long_sequence_fft_b200.linear_attention import _pack_shape
    f = dict(B=1, T=1 << 17, nseq=2048, H=16, K=128, V=128)
    f.update(kw)
    H, K, V, T = f["H"], f["K"], f["V"], f["T"]
    rows = lambda d: (T * H * d, H * d, d)                                   # noqa: E731
    shape = _pack_shape.pack(f["B"], T, f["nseq"], H, H, H, H, K, V, 2, 1.0, 1, *rows(K), *rows(K), *rows(V), *rows(V))
    return _lib().fftconv_linear_attention_workspace_bytes(shape, backward)


@pytest.mark.parametrize("backward,roles", [(0, 1), (1, 3)])
def test_packed_workspace_does_not_grow_with_short_sequences(backward, roles):
    """States are kept for the segments of sequences that may be cut: fewer
    than twice as many as pieces of the length that a cut takes, whatever the
    number of sequences; a sequence more costs its place in the plan."""
    state = 16 * 128 * 128 * 4
    few, many = (_attention_bytes(backward, nseq=n) for n in (64, 1 << 16))
    assert many - few <= ((1 << 16) - 64) * 32 + 256
    # a piece is 5/4 of an SM's share of heads x roles x tokens, in tiles of 128 tokens
    pieces = 148 * 4 // (5 * 16 * roles) + 1
    assert few <= roles * 2 * pieces * state + (1 << 16)
    assert many < 128 << 20


def test_packed_workspace_of_few_long_sequences():
    """No more segments than there are: one sequence of all tokens."""
    state = 2 * 64 * 64 * 4
    size = _attention_bytes(0, nseq=1, T=8192, H=2, K=64, V=64)
    assert 0 < size <= (8192 // 512 + 1) * (state + 64) + 1024


@pytest.mark.parametrize("S,C,G", [(1, 4096, 1), (1, 1032, 2), (1, 520, 1), (2, 1024, 1024), (16, 4096, 4096),
                                   (4, 96, 32), (5, 35, 7), (64, 768, 12), (3, 65536, 8)])
@pytest.mark.parametrize("backward", [0, 1])
def test_norm_workspace_does_not_grow_with_samples(S, C, G, backward):
    """Partial results of some samples at a time."""
    sizes = [_norm_bytes(N, S, C, G, backward) for N in (1, 8, 444, 5000, 1 << 17)]
    assert max(sizes) <= (64 << 20) + 1024
    assert sizes[0] > 0 and sizes[0] < 1 << 23


@pytest.mark.parametrize("D,G", [(17, 600000), (5, 2 << 20), (3, 5 << 20)])
@pytest.mark.parametrize("dtype", [0, 2])
def test_norm_groups_beyond_a_grid(D, G, dtype):
    """Narrow groups that take more blocks of groups than a launch has: refused
    before it, forward and backward."""
    lib, C = _lib(), D * G
    at = [i << 40 for i in range(1, 9)]                      # (never read)
    rc = lib.fftconv_group_norm(at[0], None, None, None, at[1], None, None, 1, 1, C, G, C, 0, dtype, dtype, 1, 1e-5,
                                at[2], 1 << 40, None)
    assert rc == -2 and b"groups" in lib.fftconv_last_error()
    rc = lib.fftconv_group_norm_backward(at[0], None, None, None, at[1], at[2], at[3], at[4], None, None, None, 1, 1,
                                         C, G, C, 0, C, dtype, dtype, 1, at[5], 1 << 40, None)
    assert rc == -2 and b"groups" in lib.fftconv_last_error()
