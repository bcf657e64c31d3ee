"""The scored call's outputs beside those of the plain call on the same inputs."""
import pytest
import torch

import paged_kv_cache_250_gb300 as pkv
from ops_harness import DT, Paged, half_step
from test_scored_decode_gpu import expect, pool_of, scored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("lens", [[5000, 3, 700, 129], [20011], [0, 1, 16, 64]])
@pytest.mark.parametrize("cache,Hq,Hkv,d", [("f16", 4, 4, 64), ("bf16", 8, 2, 128),
                                            ("e4m3", 8, 1, 128), ("e4m3tok", 8, 4, 128)])
def test_outputs(cache, Hq, Hkv, d, lens, out_type):
    """Each is off by at most `tol` from the formula, and by half a step of the output's
    type where it was rounded."""
    p = Paged(lens, Hq, Hkv, d, cache, 25)
    q = p.queries(len(lens), 26, 2.0)
    out = scored(p, q, pool_of(p, 0.0), out_type=out_type)
    plain = torch.empty_like(out)
    n = pkv.pkv_decode_workspace_bytes(p.desc, len(lens), p.mbs)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode_attention(p.desc, q.cuda(), p.kc, p.vc, p.tables, p.ctx, p.scale, plain,
                                   ws)
    ref, tol, _, _ = expect(p, q, pool_of(p, 0.0), 1.0)
    bound = 2 * (tol[..., None] + half_step(ref.abs() + tol[..., None], out_type))
    assert ((out.double() - plain.double()).abs().cpu() <= bound).all()
    assert out.dtype == plain.dtype == DT[out_type]
