"""Prompts over sliding windows with sinks: forward and backward against f64, for every
kernel that takes a window."""
import ctypes

import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import assert_output
from online_softmax_attention_gb300 import _abi
from parity_util import check_grad
from test_gpu_grouped import make
from window_model import gradients, reference

pytestmark = pytest.mark.gpu

WINDOWS = [(1, 0), (1, 1), (7, 3), (64, 0), (127, 1), (128, 4), (129, 128), (200, 300)]


def cuda(x):
    return {n: t.cuda() for n, t in x.items()}


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("lens,hq,hkv", [([1], 2, 1), ([600], 8, 2), ([127, 1, 0, 131, 400], 6, 2), ([330, 5], 2, 2),
                                         ([290, 61], 5, 1), ([17] * 9, 16, 2)])
def test_forward_tensor_cores(lens, hq, hkv, window, sinks, dtype, d):
    x, cu = make(lens, hq, hkv, d, dtype, 51)
    c = cuda(x)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=window, sinks=sinks, kernel="tc")
    assert_output(o, lse, reference(x, lens, d ** -0.5, window, sinks), dtype, f"{lens} {hq}/{hkv} {window}+{sinks}")
    assert attn.device_status() == 0


@pytest.mark.parametrize("n,window,sinks", [(2500, 300, 4), (2500, 40, 0), (1900, 1800, 500), (3000, 640, 700)])
def test_forward_of_long_prompts(n, window, sinks):
    """Windows behind a gap of many tiles, units cut between blocks."""
    x, cu = make([n, 700], 8, 2, 128, torch.bfloat16, 52)
    c = cuda(x)
    want = reference(x, [n, 700], 128 ** -0.5, window, sinks)
    first = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=window, sinks=sinks)
    assert_output(*first, want, torch.bfloat16)
    for _ in range(2):
        again = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=window, sinks=sinks)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("kernel,dtype,d", [("auto", torch.float32, 64), ("auto", torch.float32, 128),
                                            ("simt", torch.bfloat16, 64), ("simt", torch.float16, 128)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_forward_cuda_cores(kernel, dtype, d, window, sinks):
    lens = [130, 1, 377]
    x, cu = make(lens, 6, 2, d, dtype, 53)
    c = cuda(x)
    call = attn.FwdCall(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, kernel=kernel, window=window, sinks=sinks)
    assert call.selected_kernel() == "simt"
    assert_output(*call.run(), reference(x, lens, d ** -0.5, window, sinks), dtype)


@pytest.mark.parametrize("splits", [0, 1, 3, 20])
def test_forward_key_splits(splits):
    x, _ = make([700], 4, 2, 64, torch.float32, 54)
    c = cuda(x)
    for window, sinks in ((90, 5), (300, 0), (64, 200)):
        o, lse = attn.fwd(c["q"], c["k"], c["v"], causal=True, num_splits=splits, window=window, sinks=sinks)
        assert_output(o, lse, reference(x, [700], 0.125, window, sinks), torch.float32, f"{window}+{sinks}")


@pytest.mark.parametrize("scale", [0.3, -0.11, 0.0])
def test_forward_scaled_and_stored_in_f32(scale):
    x, _ = make([700], 8, 2, 128, torch.bfloat16, 55)
    c = cuda(x)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], causal=True, scale=scale, out_dtype=torch.float32, window=150, sinks=6)
    assert_output(o, lse, reference(x, [700], scale, 150, 6), torch.bfloat16)


def test_forward_strided_views_and_rows_behind_the_last_sequence():
    lens, hq, hkv, d = [200, 60], 8, 2, 64
    x, cu = make(lens + [40], hq, hkv, d, torch.float16, 56)
    both = torch.cat([x["q"], x["k"], x["v"]], 1).cuda()
    both[260:] = float("nan")
    call = attn.FwdCall(both[:, :hq], both[:, hq:hq + hkv], both[:, hq + hkv:], causal=True, cu_seqlens_q=cu[:3],
                        window=50, sinks=2)
    call.o.fill_(7.0)
    call.lse.fill_(7.0)
    o, lse = call.run()
    assert (o[260:] == 7).all() and (lse[:, 260:] == 7).all()
    assert_output(o[:260], lse[:, :260], reference({n: t[:260] for n, t in x.items()}, lens, 0.125, 50, 2), torch.float16)


def test_a_window_as_long_as_the_keys_is_none():
    x, cu = make([300, 200], 8, 2, 128, torch.bfloat16, 57)
    c = cuda(x)
    plain = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu)
    for window in (500, 2 ** 31 - 1):
        wide = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=window, sinks=3)
        assert all(torch.equal(a, b) for a, b in zip(plain, wide))
    # longer than every sequence, but not than all of them together
    assert_output(*attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=400, sinks=2 ** 31 - 1),
                  reference(x, [300, 200], 128 ** -0.5, None, 0), torch.bfloat16)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64), (torch.bfloat16, 64)])
@pytest.mark.parametrize("window,sinks", [(2, 0), (7, 3), (64, 0), (128, 4), (129, 130), (300, 20)])
@pytest.mark.parametrize("lens,hq,hkv", [([129, 1, 420], 6, 2), ([700], 5, 1), ([64, 0, 330], 4, 4)])
def test_backward_tensor_cores(lens, hq, hkv, window, sinks, dtype, d):
    x, cu = make(lens, hq, hkv, d, dtype, 58, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, kernel="tc", window=window, sinks=sinks)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], out_dtype=torch.float32, **w)
    got = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **w)
    for name, g, r in zip(("dq", "dk", "dv"), got, gradients(x, lens, d ** -0.5, window, sinks)):
        check_grad(g, r, f"{name} {lens} {window}+{sinks}")
    assert attn.device_status() == 0


@pytest.mark.parametrize("kernel,dtype,d", [("auto", torch.float32, 64), ("auto", torch.float32, 128), ("simt", torch.float16, 64)])
@pytest.mark.parametrize("window,sinks", [(2, 0), (7, 3), (64, 0), (100, 70)])
def test_backward_cuda_cores(kernel, dtype, d, window, sinks):
    lens = [70, 1, 240]
    x, cu = make(lens, 6, 2, d, dtype, 59, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, kernel=kernel, window=window, sinks=sinks)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], out_dtype=torch.float32, **w)
    got = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **w)
    for name, g, r in zip(("dq", "dk", "dv"), got, gradients(x, lens, d ** -0.5, window, sinks)):
        check_grad(g, r, f"{name} {window}+{sinks}")


@pytest.mark.parametrize("dtype,kernel", [(torch.bfloat16, "tc"), (torch.float32, "simt")])
def test_a_window_of_one_key(dtype, kernel):
    """Each query sees itself alone: p = 1, dv = dO summed over the group, and ds = 0, up to
    the f32 difference of two equal sums."""
    x, cu = make([300, 77], 4, 2, 64, dtype, 60, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, kernel=kernel, window=1)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], out_dtype=torch.float32, **w)
    dq, dk, dv = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **w)
    assert max(float(g.abs().max()) for g in (dq, dk)) < 1e-2
    check_grad(dv, x["do"].double().view(377, 2, 2, 64).sum(2).numpy(), "dv")


def test_gradients_against_differences():
    """As without a window: central differences of <o, dO> in f32, step 2^-5; the quotient's own
    error (below 1e-3 of the sum's size) and the forward's 1e-5 sqrt(n) / h lie within 2 % of
    the largest directional derivative."""
    lens = [9, 40]
    x, cu = make(lens, 4, 2, 64, torch.float32, 61, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, window=6, sinks=2)

    def loss(q, k, v):
        return float((attn.fwd(q, k, v, **w)[0].double() * c["do"].double()).sum())

    o, lse = attn.fwd(c["q"], c["k"], c["v"], **w)
    grads = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], **w)
    g = torch.Generator().manual_seed(62)
    h = 2.0 ** -5
    for i, name in enumerate("qkv"):
        for _ in range(3):
            u = torch.randn(c[name].shape, generator=g).cuda()
            u /= u.norm()
            hi, lo = ([c[n] for n in "qkv"] for _ in range(2))
            hi[i], lo[i] = hi[i] + h * u, lo[i] - h * u
            slope = (loss(*hi) - loss(*lo)) / (2 * h)
            want = float((grads[i].double() * u.double()).sum())
            assert abs(slope - want) <= 0.02 * float(grads[i].norm()), (name, slope, want)


def test_backward_of_many_blocks_is_the_same_every_time():
    lens = [90, 1300, 260, 0, 700]
    x, cu = make(lens, 8, 2, 64, torch.float16, 63, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, window=300, sinks=5)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], **w)
    got = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], **w)
    for name, g, r in zip(("dq", "dk", "dv"), got, gradients(x, lens, 0.125, 300, 5)):
        check_grad(g, r, name)
    for num_ctas in (0, 3):
        again = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], num_ctas=num_ctas, **w)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_a_step_in_a_graph_and_on_another_stream():
    lens = [400, 90]
    x, cu = make(lens, 8, 2, 64, torch.float16, 64, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, window=100, sinks=4)
    f = attn.FwdCall(c["q"], c["k"], c["v"], **w)
    f.run()
    b = attn.BwdCall(c["q"], c["k"], c["v"], f.o, f.lse, c["do"], **w)
    want = [t.clone() for t in (*f.run(), *b.run())]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.run()
        b.run()
    for t in (f.o, f.lse, b.dq, b.dk, b.dv):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, y) for a, y in zip(want, (f.o, f.lse, b.dq, b.dk, b.dv)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = attn.fwd(c["q"], c["k"], c["v"], **w)
        grads = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], **w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, y) for a, y in zip(want, (o, lse, *grads)))


def test_calls_that_are_refused():
    x, cu = make([200], 4, 2, 128, torch.bfloat16, 65, True)
    c = cuda(x)
    q, k, v = c["q"], c["k"], c["v"]

    def refused(code, fn, *args, **kw):
        with pytest.raises(attn.AttnError) as e:
            fn(*args, **kw)
        assert e.value.code == code

    refused(_abi.ATTN_EUNSUPPORTED, attn.fwd, q, k, v, window=20)  # the full relation
    refused(_abi.ATTN_EUNSUPPORTED, attn.fwd, q, k, v, causal=True, window=20, num_splits=2)
    refused(_abi.ATTN_EUNSUPPORTED, attn.fwd, q, k, v, causal=True, window=20, num_ctas=4)
    refused(_abi.ATTN_EUNSUPPORTED, attn.fwd, q.float(), k.float(), v.float(), causal=True, window=20, kernel="tc")
    q8, k8 = q.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn)
    refused(_abi.ATTN_EUNSUPPORTED, attn.fwd, q8, k8, v, causal=True, window=20)
    o, lse = attn.fwd(q, k, v, causal=True, window=20)
    refused(_abi.ATTN_EUNSUPPORTED, attn.bwd, q, k, v, o, lse, c["do"], causal=True, window=20, dq_mode="fused")
    refused(_abi.ATTN_EUNSUPPORTED, attn.bwd, q, k, v, o, lse, c["do"], window=20)
    for bad in (dict(window=0), dict(window=-1), dict(sinks=2), dict(window=3, sinks=-1)):
        with pytest.raises(ValueError):
            attn.fwd(q, k, v, causal=True, **bad)
        with pytest.raises(ValueError):
            attn.bwd(q, k, v, o, lse, c["do"], causal=True, **bad)


def test_without_allocation():
    """f32 windows have the fixed scratch; f16 ones need the packed kernel's workspace."""
    lib = _abi.load()
    for dtype, code in ((torch.float32, 0), (torch.float16, _abi.ATTN_EUNSUPPORTED)):
        x, _ = make([200], 4, 2, 64, dtype, 66)
        c = cuda(x)
        call = attn.FwdCall(c["q"], c["k"], c["v"], causal=True, window=30, sinks=1, num_splits=1)
        call.run()
        want = call.o.clone(), call.lse.clone()
        call.o.zero_()
        torch.cuda.synchronize()
        assert lib.attn_fwd_noalloc(ctypes.byref(call.args), torch.cuda.current_stream().cuda_stream) == code
        if code == 0:
            torch.cuda.synchronize()
            assert torch.equal(call.o, want[0]) and torch.equal(call.lse, want[1])


def test_offsets_that_do_not_fit_are_reported():
    x, _ = make([200], 4, 2, 64, torch.float16, 67)
    c = cuda(x)
    for cu in ([0, 150, 90], [0, 90, 300], [5, 100, 200]):
        attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=30)
        assert attn.device_status() == _abi.ATTN_EINVAL


def test_groups_of_more_than_a_tile():
    x, _ = make([150], 130, 1, 64, torch.float16, 68)
    c = cuda(x)
    call = attn.FwdCall(c["q"], c["k"], c["v"], causal=True, window=40, sinks=2)
    assert call.selected_kernel() == "simt"
    assert_output(*call.run(), reference(x, [150], 0.125, 40, 2), torch.float16)


def test_many_sequences():
    """More than the packed kernel takes without a window."""
    lens = list(np.random.default_rng(69).integers(0, 9, 2500))
    x, cu = make(lens, 4, 2, 64, torch.float16, 69)
    c = cuda(x)
    assert_output(*attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=3, sinks=1),
                  reference(x, lens, 0.125, 3, 1), torch.float16)


@pytest.mark.parametrize("scale", [0.3, -0.11])
@pytest.mark.parametrize("window,sinks", [(100, 3), (260, 300)])
def test_backward_scaled(scale, window, sinks):
    lens = [700, 90]
    x, cu = make(lens, 4, 2, 128, torch.bfloat16, 70, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, scale=scale, window=window, sinks=sinks)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], out_dtype=torch.float32, **w)
    got = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **w)
    for name, g, r in zip(("dq", "dk", "dv"), got, gradients(x, lens, scale, window, sinks)):
        check_grad(g, r, f"{name} {scale}")


def test_backward_of_a_scale_of_zero():
    """The uniform average of the admitted values: dq = dk = 0, dv as by the formula."""
    x, cu = make([400], 4, 2, 64, torch.float16, 79, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, scale=0.0, window=150, sinks=2)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], out_dtype=torch.float32, **w)
    dq, dk, dv = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **w)
    assert (dq == 0).all() and (dk == 0).all()
    check_grad(dv, gradients(x, [400], 0.0, 150, 2)[2], "dv")


@pytest.mark.parametrize("kernel,dtype,d", [("simt", torch.float32, 64), ("simt", torch.float32, 128), ("tc", torch.bfloat16, 128),
                                            ("tc", torch.float16, 64)])
@pytest.mark.parametrize("window,sinks", [(5, 1), (60, 200), (130, 4), (3, 900)])
def test_backward_of_sinks_that_many_queries_see(kernel, dtype, d, window, sinks):
    """Key blocks with a sink cut into several items: rows that are cut beside ones that are not, more
    than one block of sinks, chunks behind the last query."""
    lens = [90, 1100, 300, 700] if kernel == "tc" else [90, 600, 270, 300]
    x, cu = make(lens, 4, 2, d, dtype, 80, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, kernel=kernel, window=window, sinks=sinks)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], out_dtype=torch.float32, **w)
    call = attn.BwdCall(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **w)
    plain = attn.BwdCall(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **{**w, "sinks": 0})
    assert call.workspace.numel() > plain.workspace.numel()
    call.workspace.fill_(255)  # (NaN, where a slot is read that was not written)
    for t in (call.dq, call.dk, call.dv):
        t.fill_(float("nan"))
    for name, g, r in zip(("dq", "dk", "dv"), call.run(), gradients(x, lens, d ** -0.5, window, sinks)):
        check_grad(g, r, f"{name} {window}+{sinks}")
    assert attn.device_status() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
def test_values_that_a_window_hides_stay_out_of_the_units_behind(dtype, d):
    """A value of infinity beside the sinks reaches the rows that see it and their tiles, no others."""
    x, _ = make([1500], 8, 2, d, dtype, 60)
    c = cuda(x)
    want = attn.fwd(c["q"], c["k"], c["v"], causal=True, window=100, sinks=5)
    c["v"][6:12] = torch.inf
    got = attn.fwd(c["q"], c["k"], c["v"], causal=True, window=100, sinks=5)
    assert torch.equal(got[0][256:], want[0][256:]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,kernel", [(torch.bfloat16, "tc"), (torch.float32, "simt")])
def test_a_step_with_more_sinks_than_keys(dtype, kernel):
    x, cu = make([500, 90], 4, 2, 64, dtype, 61, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, kernel=kernel, window=5, sinks=2 ** 31 - 1)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], out_dtype=torch.float32, **w)
    assert_output(o, lse, reference(x, [500, 90], 0.125, None, 0), dtype)
    got = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], grad_dtype=torch.float32, **w)
    for name, g, r in zip(("dq", "dk", "dv"), got, gradients(x, [500, 90], 0.125, None, 0)):
        check_grad(g, r, name)
    assert attn.device_status() == 0


def test_two_steps_at_once():
    x, cu = make([900, 300], 8, 2, 64, torch.float16, 62, True)
    c = cuda(x)
    calls, want = [], []
    for window, sinks in ((100, 4), (300, 0)):
        f = attn.FwdCall(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, window=window, sinks=sinks)
        o, lse = f.run()
        b = attn.BwdCall(c["q"], c["k"], c["v"], o, lse, c["do"], causal=True, cu_seqlens_q=cu, window=window, sinks=sinks)
        want.append([t.clone() for t in (o, lse, *b.run())])
        calls.append((f, b))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [None] * 2
    for _ in range(5):
        for i, (s, (f, b)) in enumerate(zip(streams, calls)):
            with torch.cuda.stream(s):
                got[i] = [*f.run(), *b.run()]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(y, z) for y, z in zip(a, b))


@pytest.mark.parametrize("lens,hq,hkv,d,dtype", [([900, 33, 300], 8, 2, 64, torch.float16), ([2000], 4, 4, 128, torch.bfloat16)])
def test_steps_over_the_same_buffers(lens, hq, hkv, d, dtype):
    """Steps one behind the other in the same buffers and workspaces, with other inputs each time: no kernel reads what
    the step before left there."""
    sets = [make(lens, hq, hkv, d, dtype, 63 + i, True) for i in range(2)]
    cu = sets[0][1]
    c = cuda(sets[0][0])
    w = dict(causal=True, cu_seqlens_q=cu, window=150, sinks=2)
    f = attn.FwdCall(c["q"], c["k"], c["v"], **w)
    b = attn.BwdCall(c["q"], c["k"], c["v"], f.o, f.lse, c["do"], **w)
    inputs, want = [cuda(s[0]) for s in sets], []
    for x in inputs:
        o, lse = attn.fwd(x["q"], x["k"], x["v"], **w)
        want.append([o, lse, *attn.bwd(x["q"], x["k"], x["v"], o, lse, x["do"], **w)])
    for i in range(24):
        for n in c:
            c[n].copy_(inputs[i % 2][n])
        got = [t.clone() for t in (*f.run(), *b.run())]
        assert all(torch.equal(x, y) for x, y in zip(got, want[i % 2])), i


@pytest.mark.parametrize("num_ctas", [1, 7, 151, 400])
def test_backward_of_any_grid(num_ctas):
    x, cu = make([700, 90, 400], 8, 2, 64, torch.bfloat16, 66, True)
    c = cuda(x)
    w = dict(causal=True, cu_seqlens_q=cu, window=130, sinks=3)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], **w)
    want = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], **w)
    call = attn.BwdCall(c["q"], c["k"], c["v"], o, lse, c["do"], num_ctas=num_ctas, **w)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call.run(), want))
