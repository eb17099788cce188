"""Workspaces of the norms' gradients by rows: more rows never need less, up to what the GPU holds at once (these calls never touch the
device)."""
import pytest

from test_norms_abi import M, block_params, gate_params  # noqa: F401  (M is a fixture)

ROWS = sorted({1, 2, 7, 8, 9, 63, 64, 100, 151, 152, 153, 1000, 4863, 4864, 9727, 9728, 9729, 24319, 24320, 97280, 194559, 194560, 200001, 1 << 20,
               *(152 * per_sm * slots * k + d for per_sm in (1, 3, 5, 6, 20) for slots in (1, 4, 8, 16) for k in (1, 16) for d in (-1, 0, 1))})


@pytest.mark.parametrize("width,group", [(64, 64), (128, 128), (256, 256), (264, 264), (512, 512), (520, 520), (765, 765), (1280, 1280), (1536, 512), (2560, 2560),
                                         (2557, 2557), (5120, 64), (5120, 640), (8192, 8192), (8191, 8191), (16384, 8192), (3, 1), (111, 37)])
def test_gate_and_norm(M, width, group):  # noqa: F811
    size = lambda r: M.lib.ssd_gate_norm_bwd_workspace_size(gate_params(M, rows=r, width=width, group_size=group, z_stride=width, dz_stride=width))
    sizes = [size(r) for r in ROWS]
    assert sizes == sorted(sizes) and all(s % (4 * width) == 0 for s in sizes)
    assert all(s <= 4 * width * r for s, r in zip(sizes, ROWS))   # a slot has a row at least
    assert size(10 ** 7) == size(1 << 20) or group <= 256
    for dtype in (0, 1):   # and neither the type nor the strides matter
        p = gate_params(M, rows=5000, width=width, group_size=group, dtype=dtype, z_stride=width + 1, dz_stride=width + 3)
        assert M.lib.ssd_gate_norm_bwd_workspace_size(p) == size(5000)


@pytest.mark.parametrize("width", [1, 24, 64, 245, 256, 511, 513, 520, 1280, 1533, 2560, 4104, 8191, 8192])
def test_norm_after_a_block(M, width):  # noqa: F811
    size = lambda r, **kw: M.lib.ssd_block_norm_bwd_workspace_size(block_params(M, rows=r, width=width, gate_stride=width, dgate_stride=width, **kw))
    sizes = [size(r) for r in ROWS]
    assert sizes == sorted(sizes) and all(s % (8 * width) == 0 and s <= 8 * width * r for s, r in zip(sizes, ROWS))
    assert size(5000, dtype=0, out_dtype=0) == size(5000) == size(5000, residual_dtype=1)
