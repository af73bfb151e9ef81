"""Clipping a table of which some gradients stay where they are and others go to slots."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_orthogonalized_gb300 as m
    m.lib()
    return m


WORD = {"bfloat16": "int16", "float16": "int16", "float32": "int32"}
# NaNs whose bits a conversion or a product would change
NANS = {"bfloat16": (0x7F81, -1), "float16": (0x7C01, -1), "float32": (0x7F800001, -1)}


@pytest.mark.parametrize("sizes", [(1001, 300), (40000, 900003)])
@pytest.mark.parametrize("kind", sorted(WORD))
def test_in_place_nothing_is_written_where_nothing_is_clipped(nsm, kind, sizes):
    """By a norm that is no number, or no more than the limit, also beside gradients that go elsewhere."""
    import torch
    word = getattr(torch, WORD[kind])
    for no_number in (True, False):
        a = torch.randn(sizes[0], generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(getattr(torch, kind))
        if no_number:
            for i, bits in enumerate(NANS[kind]):
                a.view(word)[7 + 500 * i] = bits
        b = torch.randn(sizes[1], device="cuda")
        slot = torch.empty(sizes[1], dtype=torch.bfloat16, device="cuda")
        kept = a.view(word).clone()
        norm = torch.empty(1, device="cuda")
        table = nsm.GradTable([a, b], [a, slot])
        ws = torch.empty(table.workspace_bytes, dtype=torch.uint8, device="cuda")
        nsm.clip_grads(table, 1e-3 if no_number else 1e9, norm, workspace=ws)
        assert bool(norm.isnan()) == no_number
        assert torch.equal(a.view(word), kept)
        assert torch.equal(slot, b.bfloat16())
    # and clipped: both
    table = nsm.GradTable([a, b], [a, slot])
    before = a.double()
    nsm.clip_grads(table, 0.5, norm, workspace=ws)
    factor = 0.5 / float(torch.cat([before, b.double()]).norm())
    half = torch.finfo(a.dtype).eps / 2
    # a chunk's sum of squares takes 28 additions in fp32 (10 in a running sum, 3 of those, 5 in a warp, 8 of the warps, 2
    # more), of which the root leaves half, and rounds twice; the factor, the product, one rounding, half the least subnormal
    near = (28 / 2 + 2 + 2) * 2.0 ** -24 * 1.0001
    least = {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25, "float32": 2.0 ** -150}[kind]
    assert bool(((a.double() - before * factor).abs() <= (near + half) * (before * factor).abs() + least).all())
    assert bool(((slot.double() - b.double() * factor).abs() <= (near + 2.0 ** -8) * (b.double() * factor).abs() + 2.0 ** -134).all())
    assert nsm.device_status() == nsm.NSM_OK
