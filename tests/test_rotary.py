"""Rotary positions: the plan (CPU) and vattn_rotate against 64-bit rotations (GPU)."""
import ctypes as C
import math

import pytest
import torch

from tests.serving import amplitude, frequencies, rotate64
from verified_sparse_attention_b200 import _abi
from verified_sparse_attention_b200.decoder import SparseDecoder
from verified_sparse_attention_b200.rotary import Rotary

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SCALINGS = {
    "none": {},
    "linear": dict(factor=4.0),
    "base": dict(factor=8.0),
    "bands": dict(factor=8.0, original_ctx=8192, low=1.0, high=4.0),
    "yarn": dict(factor=16.0, original_ctx=4096, slow=1.0, fast=32.0),
}


# ------------------------------------------------------------ the plan
@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rot", [2, 6, 34, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_plan_frequencies(scaling, rot, base):
    r = Rotary(head_dim=128, rot_dim=rot, base=base, scaling=scaling, **SCALINGS[scaling])
    ref = frequencies(rot, base=base, scaling=scaling, **SCALINGS[scaling])
    for i in range(rot // 2):
        turns = r.plan.turns[i] / 2**64
        # the reference's own double rounding: a few units of 2^-53 relative, |ln f| amplified
        assert abs(turns - float(ref[i]) / (2 * math.pi)) <= 2**-64 + 1e-14 * turns
    assert r.plan.amplitude == pytest.approx(amplitude(scaling, SCALINGS[scaling].get("factor", 1.0)), rel=2**-23)


def test_plan_amplitude_is_taken():
    assert Rotary(head_dim=64, scaling="yarn", factor=4.0, amplitude=0.5).plan.amplitude == 0.5


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling="linear", factor=0.0), dict(scaling="yarn", factor=float("inf")),
    dict(scaling="bands", low=4.0, high=4.0), dict(scaling="bands", original_ctx=0), dict(scaling="yarn", slow=0.0),
    dict(scaling="yarn", slow=33.0)])
def test_plan_refusals(bad):
    with pytest.raises(_abi.VattnError):
        Rotary(**{"head_dim": 128, **bad})


@pytest.mark.parametrize("bad", [dict(layout="other"), dict(scaling="other"), dict(amplitude=0.0),
                                 dict(amplitude=-1.0)])
def test_plan_names_and_amplitude_refusals(bad):
    with pytest.raises(ValueError):
        Rotary(head_dim=128, **bad)


def _call(plan, tokens=4, heads=8, dtype=_abi.VATTN_BF16, xs=(1024, 128), os=(1024, 128), x=1 << 20, out=1 << 21,
          pos=1 << 22):
    return _abi.vattn_rotate(plan, x, out, pos, tokens, heads, dtype, xs, os, stream=0, check=False)


def test_rotate_refusals_before_any_launch():
    plan = Rotary(head_dim=128).plan
    bad = [dict(tokens=-1), dict(heads=-1), dict(tokens=(1 << 30) + 1), dict(heads=(1 << 16) + 1), dict(dtype=2),
           dict(x=0), dict(out=0), dict(pos=0), dict(os=(1024, 127)), dict(os=(1023, 128)), dict(os=(127, 4096)),
           dict(os=(128, 511)), dict(xs=(-1, 128)),
           dict(xs=(1024, -128)), dict(out=1 << 20, xs=(2048, 128)), dict(out=1 << 20, xs=(1024, 256))]
    for kw in bad:
        assert _call(plan, **kw) == _abi.VATTN_EINVAL, kw
    assert _call(_abi.vattn_rope()) == _abi.VATTN_EINVAL          # not filled by vattn_rope_init
    assert _call(plan, tokens=0, x=0, out=0, pos=0) == _abi.VATTN_OK
    assert _call(plan, heads=0, x=0, out=0, pos=0) == _abi.VATTN_OK


def test_rotate_refuses_pointers_between_elements():
    plan = Rotary(head_dim=128).plan
    for dtype, off in ((_abi.VATTN_BF16, 1), (_abi.VATTN_FP32, 1), (_abi.VATTN_FP32, 2)):
        for name, base in (("x", 1 << 20), ("out", 1 << 21)):
            assert _call(plan, dtype=dtype, **{name: base + off}) == _abi.VATTN_EINVAL, (dtype, name, off)
    for off in (1, 2, 3):
        assert _call(plan, pos=(1 << 22) + off) == _abi.VATTN_EINVAL


def test_rotate_wrapper_refuses_host_tensors_and_shapes():
    r = Rotary(head_dim=64)
    x = torch.zeros(3, 2, 64)
    pos = torch.zeros(3, dtype=torch.int32)
    for bad in (x, x[..., :32], x.double(), x[0]):
        with pytest.raises(ValueError):
            r.rotate(bad, pos)


def test_rotate_refuses_what_autograd_would_have_to_follow():
    r = Rotary(head_dim=64)
    x = torch.zeros(3, 2, 64, requires_grad=True)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="gradient"):
        r.rotate(x, pos)
    with pytest.raises(ValueError, match="gradient"):
        r.rotate(x * 2, pos, out=torch.zeros(3, 2, 64))
    for call in (lambda: r.rotate(x.detach(), pos), torch.no_grad()(lambda: r.rotate(x, pos))):
        with pytest.raises(ValueError, match="CUDA device"):    # a host tensor is all that is wrong with it
            call()


@pytest.mark.gpu
def test_rotate_takes_leaves_without_autograd():
    r = Rotary(head_dim=64)
    x = torch.randn(3, 2, 64, device="cuda", requires_grad=True)
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    with torch.no_grad():
        got = r.rotate(x, pos)
    assert not got.requires_grad and torch.equal(got, r.rotate(x.detach(), pos))


# ------------------------------------------------------------ on the GPU
# fp32: cos and sin to 2^-22 (angle 2^-32 turns + 2^-25 relative, sincospif, the amplitude's product), two
# products and a sum of half an ulp each: |err| <= 2^-21 (|a| + |b|) A. bf16 adds half an ulp of the result.
def _check(got, ref, x, dtype, amp):
    mag = x.double().abs().amax(-1, keepdim=True).cpu() * 2 * amp
    tol = 2**-21 * mag + (2**-8 * ref.abs() if dtype == "bf16" else 0)
    err = (got.double().cpu() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (64, 16), (64, 6), (128, 128), (128, 64), (128, 34), (128, 2)])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 32), (37, 5), (300, 9)])
def test_rotate(layout, dtype, d, rot, tokens, heads):
    scaling = ["none", "linear", "base", "bands", "yarn"][(rot + tokens) % 5]
    kw = SCALINGS[scaling]
    r = Rotary(head_dim=d, rot_dim=rot, layout=layout, scaling=scaling, **kw)
    g = torch.Generator().manual_seed(tokens * 7 + rot)
    x = torch.randn(tokens, heads, d, generator=g).to(DT[dtype])
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (tokens,), generator=g).int()
    pos[0] = 0
    pos[-1] = (1 << 24) - 1
    amp = amplitude(scaling, kw.get("factor", 1.0))
    freq = frequencies(rot, scaling=scaling, **kw)
    # far positions: reduce the angle by the plan's own turns, exact in integers, so that the reference keeps 64 bits
    ang = torch.tensor([[((r.plan.turns[i] * int(p)) % 2**64) / 2**64 * 2 * math.pi for i in range(rot // 2)]
                        for p in pos], dtype=torch.float64)
    near = pos.abs() < 1 << 20
    assert torch.allclose(torch.cos(ang[near]), torch.cos(pos[near].double()[:, None] * freq), atol=1e-8)
    one = torch.ones(tokens)
    for transpose in (False, True):
        ref = torch.stack([rotate64(x[t:t + 1], one[t:t + 1], rot, layout, ang[t], amp, transpose)[0]
                           for t in range(tokens)])
        got = r.rotate(x.cuda(), pos.cuda(), transpose=transpose)
        _check(got, ref, x, dtype, amp)
        assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotate_views_in_place_and_unaligned(dtype):
    r = Rotary(head_dim=128)
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(33, 12, 128, generator=g).to(DT[dtype]).cuda()
    pos = torch.arange(5, 38, dtype=torch.int32).cuda()
    x = wide[:, 3:8]
    ref = r.rotate(x.contiguous(), pos)
    keep = wide.clone()
    assert torch.equal(r.rotate(x, pos), ref)                     # a view of a wider row
    out = torch.full((33, 7, 128), 9.0, dtype=DT[dtype], device="cuda")
    r.rotate(x, pos, out=out[:, 1:6])                             # into a view
    assert torch.equal(out[:, 1:6], ref) and (out[:, 0] == 9).all() and (out[:, 6] == 9).all()
    r.rotate(x, pos, out=x)                                       # in place, neighbours untouched
    assert torch.equal(wide[:, 3:8], ref)
    assert torch.equal(wide[:, :3], keep[:, :3]) and torch.equal(wide[:, 8:], keep[:, 8:])
    flat = torch.zeros(33 * 5 * 128 + 1, dtype=DT[dtype], device="cuda")
    odd = flat[1:].view(33, 5, 128)                               # not 16-byte aligned
    odd.copy_(keep[:, 3:8])
    assert torch.equal(r.rotate(odd, pos), ref)
    heads_first = keep[:, 3:8].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(r.rotate(heads_first, pos), ref)
    out = torch.empty(5, 33, 128, dtype=DT[dtype], device="cuda")
    assert torch.equal(r.rotate(x.contiguous(), pos, out=out.transpose(0, 1)), r.rotate(x.contiguous(), pos))
    assert torch.equal(r.rotate(heads_first, pos, out=heads_first), ref)    # in place, heads first


@pytest.mark.gpu
def test_rotate_gradient_is_the_transpose():
    r = Rotary(head_dim=64, rot_dim=48, layout="interleaved", scaling="yarn", **SCALINGS["yarn"])
    g = torch.Generator().manual_seed(2)
    x, w = (torch.randn(19, 3, 64, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 100000, (19,), generator=g).int().cuda()
    grad = r.rotate(w, pos, transpose=True)
    # <R x, w> = <x, R^T w>, and central differences of <R x, w> in random directions (the map is linear, so
    # the only error is fp32 rounding: 2^-21 of the summed magnitudes, twice, over the step)
    y = r.rotate(x, pos)
    mag = float((y.double() * w.double()).abs().sum())
    assert abs(float((y.double() * w.double()).sum() - (x.double() * grad.double()).sum())) <= 2**-20 * 2 * mag
    for k in range(3):
        e = torch.randn(19, 3, 64, generator=g).cuda()
        diff = (r.rotate(x + 0.5 * e, pos).double() - r.rotate(x - 0.5 * e, pos).double())
        num, ana = float((diff * w.double()).sum()), float((e.double() * grad.double()).sum())
        assert abs(num - ana) <= 2**-20 * 4 * (mag + float((e * w).abs().sum()))


@pytest.mark.gpu
def test_rotate_on_another_stream_and_captured():
    r = Rotary(head_dim=128)
    x = torch.randn(50, 4, 128, device="cuda").bfloat16()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    ref = r.rotate(x, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = r.rotate(x, pos)
    s.synchronize()
    assert torch.equal(got, ref)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.rotate(x, pos, out=out)
    pos += 3
    graph.replay()
    assert torch.equal(out, r.rotate(x, pos))


@pytest.mark.gpu
def test_rotate_failure_leaves_nothing_for_the_next_call():
    # a stream whose capture was spoiled (by waiting for it on the host) refuses launches
    rt = C.CDLL("libcudart.so.12")
    stream, graph = C.c_void_p(), C.c_void_p()
    x = torch.randn(5, 4, 64, device="cuda").bfloat16()
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    r = Rotary(head_dim=64)
    ref, out = r.rotate(x, pos), torch.empty_like(x)
    dec = SparseDecoder(num_q_heads=4, num_kv_heads=4, head_dim=64, dtype=torch.bfloat16, page_size=16, max_batch=1,
                        max_ctx=16)
    cache = torch.randn(1, 4, 16, 64, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.zeros(1, 1, **i32), torch.full((1,), 9, **i32)
    torch.cuda.synchronize()
    assert rt.cudaStreamCreateWithFlags(C.byref(stream), 1) == 0
    assert rt.cudaStreamBeginCapture(stream, 2) == 0
    try:
        assert rt.cudaStreamSynchronize(stream) != 0
        with pytest.raises(_abi.VattnError):
            r.rotate(x, pos, out=out, stream=stream.value)
    finally:
        rt.cudaStreamEndCapture(stream, C.byref(graph))
        rt.cudaGetLastError()
        rt.cudaStreamDestroy(stream)
    dec.dense(x[:1], cache, cache, table, lens, 1)       # reported the failure of the rotation
    assert dec.last_error() == 0 and torch.equal(r.rotate(x, pos), ref)
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [0, 1, 2])
def test_rotate_takes_the_default_streams_handles(stream):
    # the legacy default stream's two and the thread's own
    r = Rotary(head_dim=64)
    x = torch.randn(7, 3, 64, device="cuda")
    pos = torch.arange(7, dtype=torch.int32, device="cuda")
    want = r.rotate(x, pos)
    torch.cuda.synchronize()
    got = r.rotate(x, pos, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
