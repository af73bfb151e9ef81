"""The embedding gradient's workspace: one made for a program's largest batch serves every smaller one."""

import os

import pytest


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from newton_schulz_orthogonalized_gb300 import _build
        _build.build()
    m.lib()
    return m


@pytest.mark.parametrize("vocab", [300, 50257])
@pytest.mark.parametrize("cols", [1, 33, 256, 768, 771, 4096, 16384])
def test_bytes_never_fall_as_rows_grow(nsm, vocab, cols):
    """Every row count up to some past where the sort's tiles grow (65536), and on from there in steps of a piece;
    the pieces' lengths change below, at counts that the width sets."""
    call = nsm.lib().nsm_embedding_workspace_bytes
    last, at = 0, 0
    for rows in list(range(0, 70000)) + list(range(70016, 200000, 32)) + [1 << k for k in range(18, 31)]:
        b = call(rows, vocab, cols)
        assert b >= last, f"{b} bytes for {rows} rows, {last} for {at}"
        last, at = b, rows


@pytest.mark.gpu
def test_a_larger_batch_s_workspace_serves_a_smaller_one(nsm):
    """The same bits, and the workspace is no larger than it was made."""
    import torch
    vocab, cols = 1009, 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    # rows of this width are summed in pieces of 16 up to 19424 of them, of 32 from there on; tiles of 1024 up to 65536
    for small, large in ((19424, 19425), (65536, 65537)):
        ws = torch.full((nsm.embedding_workspace_bytes(large, vocab, cols) + 256,), 0xff, dtype=torch.uint8, device="cuda")
        d = torch.randn(small, cols, generator=g, device="cuda").bfloat16()
        tokens = (vocab * torch.rand(small, generator=g, device="cuda") ** 4).long()
        want, got = torch.empty(vocab, cols, device="cuda"), torch.empty(vocab, cols, device="cuda")
        nsm.embedding_backward(d, tokens, got, ws[:-256])
        assert bool((ws[-256:] == 0xff).all())
        own = torch.empty(nsm.embedding_workspace_bytes(small, vocab, cols), dtype=torch.uint8, device="cuda")
        nsm.embedding_backward(d, tokens, want, own)
        assert torch.equal(got, want)
        # each addition is off by less than 2^-24 of the sizes' sum, and a row goes through 64 of them in its piece, 256
        # in an eighth of a token's 2048 pieces, and 8 over the eighths, at most
        exact = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, tokens, d.double())
        size = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, tokens, d.double().abs())
        assert bool(((got.double() - exact).abs() <= (64 + 256 + 8 + 2) * 2.0 ** -24 * size).all())
    assert nsm.device_status() == nsm.NSM_OK
