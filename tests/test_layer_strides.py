"""Which views of a wider matrix, and which streams, the operators around the scan take."""
import pytest
import torch


@pytest.fixture(scope="module")
def row_stride():
    from mamba_ssd_chunked_scan_gb300 import build
    build.build()
    from mamba_ssd_chunked_scan_gb300 import layer
    return layer._row_stride


M = torch.zeros(3, 50, 400)


@pytest.mark.parametrize("view,step", [
    (M, 400), (M[..., 64:192], 400), (M[:, -1:], 20000), (M[:, -1:, 8:72], 20000), (M[:, 7], 20000), (M[:1, :, :100], 400),
    (M[:1, 3:4, :100], 100), (M[:, :, None, :100], 400), (M[:, -1:, None, :100], 20000), (M[1, :, 5:9], 400), (M[..., 3:4], 400), (M[:, ::2], 800)])
def test_rows_at_one_stride(row_stride, view, step):
    assert row_stride("x", view) == step


@pytest.mark.parametrize("view", [M[:, :20, :100], M[:, ::3], M[..., ::2], M.transpose(0, 1), M.transpose(1, 2), M[0].t(),
                                  M[:1, :1].expand(3, 50, 400), M[:, :1].expand(3, 50, 400), M[0, 0, ::3]])
def test_others_are_refused(row_stride, view):
    with pytest.raises(ValueError):
        row_stride("x", view)


def test_stream_of_another_device_is_refused():
    """Made current, it would take the call to its own device, and the tensors' device would then get another stream."""
    from types import SimpleNamespace
    from mamba_ssd_chunked_scan_gb300 import build
    build.build()
    from mamba_ssd_chunked_scan_gb300 import layer
    with pytest.raises(ValueError, match="stream"):
        with layer._elsewhere(0, SimpleNamespace(device=torch.device("cuda", 1))):
            pass


@pytest.mark.gpu
def test_last_tokens_of_a_prompt():
    import mamba_ssd_chunked_scan_gb300 as ssd
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
    h, w, dy = r(6, 33, 256), r(96, 128), r(6, 1, 96)
    x = h[:, -1:, 64:192]
    y = ssd.linear(x, w)
    assert y.shape == (6, 1, 96) and torch.equal(y, ssd.linear(x.contiguous(), w))
    a, b = ssd.linear_bwd(dy, x, w), ssd.linear_bwd(dy, x.contiguous(), w)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    g, v = h[:, -1:, :128], h[:, -1:, 128:]
    state = torch.randn(6, 128, generator=gen, device="cuda")
    y, fin = ssd.gate_scan(g, v, state, return_final_states=True)
    y2, fin2 = ssd.gate_scan(g.contiguous(), v.contiguous(), state, return_final_states=True)
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    one, two = (ssd.gate_scan_bwd(p, q, y, torch.ones_like(y), state) for p, q in ((g, v), (g.contiguous(), v.contiguous())))
    assert all(torch.equal(one[k], two[k]) for k in ("dg", "dx", "dinit"))
