"""Arguments of the prepared calls that only the kernels can refuse, and what is refused on the host with tensors on the GPU."""
import pytest
import torch

import online_softmax_attention_gb300 as attn
from online_softmax_attention_gb300 import _abi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv", [4, 2])
@pytest.mark.parametrize("cu", [[0, (1 << 32) + 64], [0, -(1 << 32) + 64], [1 << 32, 64]])
def test_offsets_on_the_device_are_not_cut_to_32_bits(cu, hkv):
    """64-bit offsets whose low 32 bits would be good ones."""
    q, k, v = (torch.randn(64, h, 64, device="cuda").half() for h in (4, hkv, hkv))
    cu = torch.tensor(cu, device="cuda")
    o, lse = attn.fwd(q, k, v, causal=True)
    assert attn.device_status() == 0
    attn.fwd(q, k, v, causal=True, cu_seqlens_q=cu)
    assert attn.device_status() == _abi.ATTN_EINVAL
    attn.bwd(q, k, v, o, lse, q, causal=True, cu_seqlens_q=cu)
    assert attn.device_status() == _abi.ATTN_EINVAL
    got = attn.fwd(q, k, v, causal=True, cu_seqlens_q=torch.tensor([0, 64], device="cuda"))
    assert attn.device_status() == 0 and torch.equal(got[0], o)


def test_outputs_and_workspaces_of_a_forward():
    q, k, v = (torch.randn(64, h, 64, device="cuda").half() for h in (4, 2, 2))
    want = attn.fwd(q, k, v, causal=True)
    need = attn.FwdCall(q, k, v, causal=True).workspace.numel()
    for kw in (dict(out=torch.empty(64, 4, 64).half()), dict(out=torch.empty_like(k)), dict(lse=torch.empty(4, 64)),
               dict(workspace=torch.empty(need, dtype=torch.uint8)),
               dict(workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            attn.FwdCall(q, k, v, causal=True, **kw)
    with pytest.raises(ValueError):
        attn.fwd(q, k.cpu(), v)
    out, lse = torch.zeros(70, 6, 64, dtype=torch.float16, device="cuda"), torch.zeros(4, 64, device="cuda")
    attn.FwdCall(q, k, v, causal=True, out=out, lse=lse).run()
    assert torch.equal(out[:64, :4], want[0]) and torch.equal(lse, want[1])
    assert not out[64:].any() and not out[:, 4:].any()


def test_arguments_of_a_backward():
    q, k, v = (torch.randn(64, h, 64, device="cuda").half() for h in (4, 2, 2))
    o, lse = attn.fwd(q, k, v, causal=True)
    want = attn.bwd(q, k, v, o, lse, q, causal=True)
    need = attn.BwdCall(q, k, v, o, lse, q, causal=True).workspace.numel()
    for kw in (dict(dk=torch.empty(64, 2, 64).half()), dict(workspace=torch.empty(need, dtype=torch.uint8)),
               dict(workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            attn.BwdCall(q, k, v, o, lse, q, causal=True, **kw)
    for bad in ((q, k, v, k, lse, q), (q, k, v, o, lse, k), (q, k, v, o, lse.cpu(), q), (q, k, v, o, lse.t(), q),
                (q, k, v, o.cpu(), lse, q)):
        with pytest.raises(ValueError):
            attn.bwd(*bad, causal=True)
    with pytest.raises(TypeError):
        attn.bwd(q, k, v, o, lse, q.float(), causal=True)
    with pytest.raises(TypeError):
        attn.bwd(q, k.bfloat16(), v, o, lse, q, causal=True)
    dk = torch.zeros(70, 5, 64, dtype=torch.float16, device="cuda")
    got = attn.BwdCall(q, k, v, o, lse, q, causal=True, dk=dk[:, 1:]).run()
    assert torch.equal(got[0], want[0]) and torch.equal(dk[:64, 1:3], want[1]) and torch.equal(got[2], want[2])
    assert not dk[64:].any() and not dk[:, 0].any() and not dk[:, 3:].any()


@pytest.mark.parametrize("hkv", [4, 2])
def test_values_longer_than_the_keys(hkv):
    """A value buffer with room behind the last key."""
    q, k, v = (torch.randn(64, h, 64, device="cuda").half() for h in (4, hkv, hkv))
    want = attn.fwd(q, k[:40], v[:40].clone())
    o, lse = attn.fwd(q, k[:40], v)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for a, b in zip(attn.bwd(q, k[:40], v, o, lse, q), attn.bwd(q, k[:40], v[:40], o, lse, q)):
        assert torch.equal(a, b)
