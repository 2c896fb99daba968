"""Arguments that the prepared calls refuse on the host, before any pointer is followed
(CPU tensors: with good arguments the last refusal is that they are not on a GPU)."""
import pytest
import torch

import online_softmax_attention_gb300 as attn


def tensors(hq=4, hkv=2, n=8, d=64, dtype=torch.float16):
    return [torch.zeros(n, h, d, dtype=dtype) for h in (hq, hkv, hkv)]


def forward(**kw):
    q, k, v = tensors()
    return attn.fwd(q, k, v, causal=True, **kw)


def backward(**kw):
    q, k, v = tensors()
    return attn.bwd(q, k, v, q, torch.zeros(4, 8), q, causal=True, **kw)


@pytest.mark.parametrize("call", [forward, backward])
def test_good_arguments_only_lack_a_gpu(call):
    for cu in (None, [0, 3, 8], torch.tensor([0, 3, 8]), torch.tensor([0, 3, 8], dtype=torch.int32)):
        with pytest.raises(ValueError, match="CUDA"):
            call(cu_seqlens_q=cu)
        with pytest.raises(ValueError, match="CUDA"):
            call(cu_seqlens_q=cu, cu_seqlens_k=cu)


@pytest.mark.parametrize("call", [forward, backward])
def test_fewer_key_offsets_than_query_offsets(call):
    """The kernels read as many of one list as of the other."""
    for ck in ([0, 8], [0, 1, 3, 8], torch.tensor([0, 8], dtype=torch.int32)):
        with pytest.raises(ValueError, match="cu_seqlens_k must have 3"):
            call(cu_seqlens_q=[0, 3, 8], cu_seqlens_k=ck)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("far", [(1 << 32) + 8, -(1 << 32) + 8, 1 << 31])
def test_offsets_are_not_cut_to_32_bits(call, far):
    for cu in ([0, far], torch.tensor([0, far])):
        with pytest.raises(ValueError, match="cu_seqlens_q: entries must fit 32 bits"):
            call(cu_seqlens_q=cu)
    with pytest.raises(ValueError, match="cu_seqlens_k: entries must fit 32 bits"):
        call(cu_seqlens_q=[0, 8], cu_seqlens_k=[0, far])


def prepared(**kw):
    q, k, v = tensors()
    return attn.FwdCall(q, k, v, causal=True, **kw)


def test_outputs_that_a_forward_would_write_past():
    for out in (torch.empty(8, 2, 64), torch.empty(7, 4, 64), torch.empty(8, 4, 32), torch.empty(32, 64)):
        with pytest.raises(ValueError, match="out must be"):
            prepared(out=out.half())
    for lse in (torch.empty(4, 8).half(), torch.empty(2, 8), torch.empty(8, 4), torch.empty(4, 16)[:, ::2],
                torch.empty(31)):
        with pytest.raises(ValueError, match="lse must be"):
            prepared(lse=lse)
    for good in (torch.empty(9, 6, 64), torch.empty(8, 4, 64)):  # a buffer with room is written in part
        with pytest.raises(ValueError, match="CUDA"):
            prepared(out=good.half(), lse=torch.empty(4, 8))


def gradients(**kw):
    q, k, v = tensors()
    a = dict(q=q, k=k, v=v, o=q, lse=torch.zeros(4, 8), dout=q)
    a.update(kw)
    return attn.BwdCall(causal=True, **a)


def test_inputs_that_a_backward_would_read_past():
    for name, t in (("o", torch.empty(8, 2, 64)), ("o", torch.empty(7, 4, 64)), ("dout", torch.empty(8, 2, 64)),
                    ("dout", torch.empty(5, 4, 64)), ("dout", torch.empty(8, 4, 32))):
        with pytest.raises(ValueError, match=f"{name} must be"):
            gradients(**{name: t.half()})
    for lse in (torch.empty(2, 8), torch.empty(8, 4), torch.empty(4, 8).half(), torch.empty(4, 8, dtype=torch.float64),
                torch.empty(8, 4).t(), torch.empty(16)):
        with pytest.raises(ValueError, match="lse must be"):
            gradients(lse=lse)
    with pytest.raises(ValueError, match="CUDA"):
        gradients(o=torch.empty(9, 4, 64), lse=torch.empty(32))  # f32 outputs, room, a flat lse


def test_inputs_of_another_type_in_a_backward():
    """One type is passed on for q, k, v and dout: another's bits would be read as it."""
    for name, t in (("k", torch.empty(8, 2, 64)), ("v", torch.empty(8, 2, 64).bfloat16()), ("dout", torch.empty(8, 4, 64))):
        with pytest.raises(TypeError, match=f"{name} must be torch.float16"):
            gradients(**{name: t})


def test_gradients_that_a_backward_would_write_past():
    for name, t in (("dq", torch.empty(8, 2, 64)), ("dk", torch.empty(7, 2, 64)), ("dv", torch.empty(8, 1, 64))):
        with pytest.raises(ValueError, match=f"{name} must be"):
            gradients(**{name: t.half()})
        with pytest.raises(TypeError, match="torch.float32"):
            gradients(grad_dtype=torch.float32, **{name: torch.empty(8, 4, 64).half()})
    with pytest.raises(ValueError, match="CUDA"):
        gradients(grad_dtype=torch.float32, dk=torch.empty(9, 2, 64), dq=torch.empty(8, 4, 64))


def test_values_longer_than_the_keys_are_not_refused():
    q, k, v = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        attn.fwd(q, k[:5], v)
    with pytest.raises(ValueError, match="k and v must both"):
        attn.fwd(q, k, v[:5])
