"""Which of its two paths bsmm_adapters takes, as its workspace query shows it
without a GPU: sorted by adapter (a workspace is needed) or as they come, the
faster of the two at the sizes measured beside the rule."""

import pytest

import block_scaled_precision_gemm_gb300 as bsmm


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("R,L,as_they_come,by_adapter", [
    (16, 1, (1, 64, 512, 777), (2047, 8192)),
    (16, 8, (1, 16, 128), (384, 1024, 8192)),
    (16, 64, (1, 64, 384, 777), (1024, 2047, 8192)),
    (16, 512, (64, 384, 2047), (8192,)),
    (32, 32, (1, 64, 128), (256, 1024, 8192)),
    (64, 1, (1, 8), (192, 1024)),
    (64, 8, (1, 8), (64, 128, 1024)),
    (128, 4, (1, 8), (32, 128, 1024)),
    (16, 1025, (1, 64, 8192), ()),
])
def test_the_measured_points(R, L, as_they_come, by_adapter):
    assert [T for T in as_they_come if bsmm.adapters_workspace_size(T, R, L)] == []
    assert [T for T in by_adapter if not bsmm.adapters_workspace_size(T, R, L)] == []
