"""The most heads that the quantising store takes: refused on the host, before any CUDA call.  No GPU."""
import pytest

from tests.test_tree_checks import P, _cache8, _refused, sd  # noqa: F401  (sd: the fixture)


@pytest.mark.parametrize("dim,most", [(256, 1_048_560), (240, 1_048_560), (128, 2_097_120), (64, 4_194_240), (16, 16_776_960)])
def test_too_many_heads_are_refused(sd, dim, most):  # noqa: F811
    # 256 threads of the store take 256 / (threads of a vector) heads, and a grid 65,535 such lots
    group = 1
    while group * 16 < dim:
        group *= 2
    assert most == 65_535 * (256 // group) and most >= 1_048_560
    f = sd.lib.spec_paged_store8
    c = _cache8(sd, heads=most + 1, head_dim=dim, k_strides=(1 << 32, dim, dim), v_strides=(1 << 32, dim, dim))
    _refused(sd, f(P, P, 4, 2048, 128, 2048, 128, P, c), "heads", str(most))
    # (no tokens: nothing to store)
    assert f(None, None, 0, 2048, 128, 2048, 128, None, c) == sd.SPEC_OK
