"""Every row of the packed kernel's output, against the kernel that does not pack."""
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import HALF_STEP
from test_gpu_grouped import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,hq,hkv,d,dtype", [([5003, 700, 1], 6, 2, 128, torch.bfloat16), ([4096], 8, 1, 64, torch.float16),
                                                 ([130] * 200, 10, 2, 64, torch.bfloat16), ([9000], 3, 1, 128, torch.float16)])
@pytest.mark.parametrize("causal", [True, False])
def test_every_row_is_written(lens, hq, hkv, d, dtype, causal):
    """Each side rounds o once and every p once (2 half steps a side at most, of |o| and of
    sum p |v|), and 2^-12 of sum p |v| covers scores, exponentials and sums in f32, as in
    cache_model.check_output; sum p |v| is itself taken with rounded p (1 + 2^-6)."""
    x, cu = make(lens, hq, hkv, d, dtype, 81)
    q, k, v = (x[n].cuda() for n in "qkv")
    out = torch.full_like(q, float("nan"))
    lse = torch.full((hq, q.shape[0]), float("nan"), device="cuda")
    attn.FwdCall(q, k, v, causal=causal, cu_seqlens_q=cu, out=out, lse=lse).run()
    assert attn.device_status() == 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    want, want_lse = attn.fwd(q, k, v, causal=causal, cu_seqlens_q=cu, num_splits=1, out_dtype=torch.float32)
    pv, _ = attn.fwd(q, k, v.abs(), causal=causal, cu_seqlens_q=cu, num_splits=1, out_dtype=torch.float32)
    step = HALF_STEP[dtype]
    bound = 2 * (step + 2.0 ** -12) * (1 + 2.0 ** -6) * pv + step * (want.abs() + 2 * step * pv) + 2.0 ** -22
    off = (out.float() - want).abs() - bound
    assert float(off.max()) <= 0, f"{float(off.max()):.3e} over the bound"
    assert float((lse - want_lse).abs().max()) <= 2e-3  # 1e-3 a side
