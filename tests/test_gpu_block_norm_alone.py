"""The norm after a block without a next norm: its gradient takes the stream after the block or not, and does not read it."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, F4, wide
from test_gpu_block_norm import EPS, SCALE, TYPES, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width,extra,offset", [(3, 24, 8, 0), (37, 2560, 80, 0), (9, 513, 0, 0), (6, 520, 8, 1), (700, 64, 0, 0)])
@pytest.mark.parametrize("dtype,rtype", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_the_stream_is_not_read(rows, width, extra, offset, dtype, rtype, gated, packed):
    t = make(rows, width, dtype, rtype, rows + 7 * width, extra, offset, gated)
    args = dict(x=t["x"], gate=t["gate"], weight=t["w"], scale=SCALE, eps=EPS)
    if packed:
        f = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], scale=SCALE, eps=EPS, pack=True)
        args.update(x=f["x"], gate=f["gate"], x_scales=f["x_scales"], gate_scales=f["gate_scales"], dtype=dtype)
    want = ssd.block_norm_bwd(None, t["dres"], h=None, **args)
    x = wide(args["x"], args.get("x_scales"))
    z = wide(args["gate"], args.get("gate_scales")) if gated else None
    check(want, t, x, z, None, dtype, rtype, False)
    codes, scales = ssd.pack_rows(t["res"])
    streams = (dict(h=t["res"]), dict(h=torch.full_like(t["res"], float("nan"))), dict(h=codes, h_scales=scales))
    for stream in streams:
        got = ssd.block_norm_bwd(None, t["dres"], **stream, **args)
        assert got.keys() == want.keys()
        for k in want:
            assert (got[k] is None) == (want[k] is None) and (got[k] is None or torch.equal(got[k], want[k])), k


def test_what_stays_refused():
    t = make(4, 64, BF, F4, 1, gated=False)
    scales = torch.ones(4, device="cuda")
    for bad in (dict(dout=t["dout"], h=t["res"]), dict(dout=t["dout"], h=None), dict(dout=None, h=None, next_weight=t["w2"]),
                dict(dout=None, h=t["res"], next_weight=t["w2"]), dict(dout=t["dout"], h=None, next_weight=t["w2"]),
                dict(dout=None, h=None, h_scales=scales)):
        with pytest.raises(ValueError):
            ssd.block_norm_bwd(dresidual=t["dres"], x=t["x"], weight=t["w"], **bad)
