"""Rotary positions (sage_rope, sage_rotary, sage_attention(rope=...)) against the formula in
extended precision.

Tolerance of a turned value, from the arithmetic: with s = |x0| + |x1| and u = 2^-24,
  - the half turns are cut to 32 bits and rounded to float32: at most pi (2^-31 + 2^-25) of angle,
    1.6 u; freq / 2 pi in float64 is off by 2^-52 of itself: |p freq| 2^-52 of angle;
  - sincospif is within 2 units in the last place: 2 u;
  - each product and the sum round once: u s and u s;
so |error| <= s (6 u + |p freq| 2^-52), and the output type's rounding adds eps / 2 of the value
(half a subnormal step of fp16 at least).
"""
import numpy as np
import pytest
import torch

from tests.gpu_common import make_case, rel_l2, to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def reference(x, pos, rope, inverse=False):
    """(values, tolerance) of the turned x (B,H,N,d); pos (axes,B or 1,N) int64."""
    B, H, N, d = x.shape
    x = x.astype(np.longdouble)
    y, tol = x.copy(), np.zeros(x.shape)
    axis = np.repeat(np.arange(rope.axes), rope.sections)
    half = rope.rotary // 2
    for j in range(half):
        angle = pos[axis[j]].astype(np.longdouble) * np.longdouble(rope.freqs[j])         # (B or 1, N)
        angle = np.broadcast_to(angle, (B, N))[:, None, :]
        c, s = np.cos(angle), np.sin(angle)
        s = -s if inverse else s
        c0, c1 = (2 * j, 2 * j + 1) if rope.interleaved else (j, j + half)
        x0, x1 = x[..., c0], x[..., c1]
        y[..., c0], y[..., c1] = x0 * c - x1 * s, x0 * s + x1 * c
        t = (np.abs(x0) + np.abs(x1)) * (6 * U + np.abs(angle) * 2.0 ** -52)
        tol[..., c0] = tol[..., c1] = t
    return y, tol


def check(got, want, tol):
    eps = torch.finfo(got.dtype).eps / 2
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[got.dtype]
    err = np.abs(got.double().cpu().numpy() - want).astype(np.float64)
    bound = tol + eps * np.abs(want).astype(np.float64) * (1 + 2.0 ** -20) + tiny
    assert np.all(err <= bound), float((err / bound).max())


CASES = [
    # B, H, Hk, N, d, sections, dtype, interleaved, pos_batch1, far
    (2, 4, 2, 65, 128, (16, 24, 24), torch.bfloat16, False, False, 1 << 20),
    (1, 1, 1, 1, 64, (32,), torch.float16, False, False, 1 << 24),
    (3, 5, 0, 7, 64, (3, 0, 5), torch.float32, True, False, 100),          # partial: 16 of 64 channels
    (2, 3, 3, 130, 128, (9, 11, 13, 7), torch.float16, True, True, 5000),  # 80 of 128 channels
    (1, 2, 7, 33, 128, (1, 2, 5), torch.bfloat16, False, True, 1 << 30),
    (16, 32, 8, 1, 128, (16, 24, 24), torch.bfloat16, False, False, 1 << 17),
]


@pytest.mark.parametrize("B,H,Hk,N,d,sections,dtype,inter,shared,far", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_formula(B, H, Hk, N, d, sections, dtype, inter, shared, far, inverse):
    import bit_trainable_attention_sage_gb300 as sg
    g = torch.Generator().manual_seed(N * d + H)
    rope = sg.make_rope(d, sections, interleaved=inter)
    Q = torch.randn(B, H, N, d, generator=g).to(dtype)
    K = torch.randn(B, Hk, N, d, generator=g).to(dtype) if Hk else None
    pos = torch.randint(-far, far, (rope.axes, 1 if shared else B, N), generator=g, dtype=torch.int64)
    Qo, Ko = sg.sage_rope(Q.cuda(), None if K is None else K.cuda(), pos.int().cuda(), rope, inverse=inverse)
    for x, y in ((Q, Qo), (K, Ko)):
        if x is not None:
            check(y, *reference(x.double().numpy(), pos.numpy(), rope, inverse))
    assert (Ko is None) == (K is None)


def test_rope_extreme_positions_and_freqs():
    """The ends of int32, and frequencies above a turn a position, negative and zero."""
    import bit_trainable_attention_sage_gb300 as sg
    rope = sg.make_rope(64, (8,), freqs=[1.0, -1.0, 0.0, 7.25, 1e-9, 2.0 ** -40, 3.0, 0.125])
    pos = torch.tensor([[[2 ** 31 - 1, -2 ** 31, 0, -1, 1, 123456789]]], dtype=torch.int64)
    Q = torch.randn(1, 2, 6, 64, generator=torch.Generator().manual_seed(0))
    Qo, _ = sg.sage_rope(Q.cuda(), None, pos.int().cuda(), rope)
    check(Qo, *reference(Q.double().numpy(), pos.numpy(), rope))


def test_rope_in_place_streams_and_large():
    """In place gives the same bits; so does another stream; and a training-sized call, where a
    thread visits several heads, equals the same heads called one by one."""
    import bit_trainable_attention_sage_gb300 as sg
    rope = sg.make_rope(128, (16, 24, 24))
    g = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.randn(2, 19, 4100, 128, device="cuda", generator=g).half()
    K = torch.randn(2, 3, 4100, 128, device="cuda", generator=g).half()
    pos = torch.randint(0, 9000, (3, 2, 4100), device="cuda", generator=g, dtype=torch.int32)
    Qo, Ko = sg.sage_rope(Q, K, pos, rope)
    for h in (0, 8, 18):
        one, _ = sg.sage_rope(Q[:, h:h + 1].contiguous(), None, pos, rope)
        assert torch.equal(one[:, 0], Qo[:, h])
    one, _ = sg.sage_rope(K[:, 2:].contiguous(), None, pos, rope)
    assert torch.equal(one[:, 0], Ko[:, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Qs, Ks = sg.sage_rope(Q, K, pos, rope, stream=side)
    side.synchronize()
    assert torch.equal(Qs, Qo) and torch.equal(Ks, Ko)
    sg.sage_rope(Q, K, pos, rope, out=(Q, K))
    assert torch.equal(Q, Qo) and torch.equal(K, Ko)


def test_rope_captured():
    import bit_trainable_attention_sage_gb300 as sg
    rope = sg.make_rope(64, (32,))
    Q = torch.randn(2, 4, 3, 64, device="cuda")
    pos = torch.zeros(1, 2, 3, dtype=torch.int32, device="cuda")
    sg.sage_rope(Q, None, pos, rope)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Qo, _ = sg.sage_rope(Q, None, pos, rope)
    pos.fill_(41)
    Q.normal_()
    graph.replay()
    want, _ = sg.sage_rope(Q, None, pos, rope)
    assert torch.equal(Qo, want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_rotary_gradient(dtype):
    """The gradient is the inverse turn of the output's gradient (the same call), and agrees with
    differences: the map is linear, so <f(x + h e) - f(x), dy> / h is exact up to rounding."""
    import bit_trainable_attention_sage_gb300 as sg
    rope = sg.make_rope(64, (8, 12, 12), interleaved=dtype == torch.float16)
    g = torch.Generator().manual_seed(3)
    Q, K = (torch.randn(2, h, 9, 64, generator=g).to(dtype).cuda().requires_grad_() for h in (4, 2))
    pos = torch.randint(0, 1000, (3, 2, 9), generator=g, dtype=torch.int32).cuda()
    Qo, Ko = sg.sage_rotary(Q, K, pos, rope)
    dQo, dKo = torch.randn(Qo.shape, generator=g).to(dtype).cuda(), torch.randn(Ko.shape, generator=g).to(dtype).cuda()
    torch.autograd.backward([Qo, Ko], [dQo, dKo])
    want = sg.sage_rope(dQo, dKo, pos, rope, inverse=True)
    assert torch.equal(Q.grad, want[0]) and torch.equal(K.grad, want[1])
    for dy, grad in ((dQo, Q.grad), (dKo, K.grad)):
        check(grad, *reference(dy.double().cpu().numpy(), pos.cpu().numpy().astype(np.int64), rope, inverse=True))
    # differences along random directions, the perturbed points exact in the type (h = 1, x = 0)
    for _ in range(4):
        e = torch.randint(-3, 4, Q.shape, generator=g).to(dtype).cuda()
        f, _ = sg.sage_rope(e, None, pos, rope)
        lhs = (f.double() * dQo.double()).sum().item()
        rhs = (e.double() * Q.grad.double()).sum().item()
        eps = torch.finfo(dtype).eps / 2 + 8 * U
        # each term of either sum is off by at most eps of its factor's size, s <= 6 and |dy0| + |dy1|
        bound = eps * ((f.double().abs() * dQo.double().abs()).sum() + 6 * dQo.double().abs().sum()
                       + (e.double().abs() * Q.grad.double().abs()).sum() + 3 * 2 * dQo.double().abs().sum()).item()
        assert abs(lhs - rhs) <= bound


def test_rotary_second_derivative():
    """f = sum of x'^4 / 12 over the turned x' = R x: the gradient R^T x'^3 / 3 is itself differentiable, and its
    product with t is R^T (x'^2 R t).  float32: with ey, et the tolerances of the turned x and t and a rounding each,
    x'^2 R t is off by 2 |y t| ey + y^2 et (1 + 2^-10 for their products) and its own arithmetic: powers of at most
    2 units in the last place, and fewer than 12 further roundings, 16 u; the last turn adds both channels' errors,
    its own tolerance and a rounding."""
    import bit_trainable_attention_sage_gb300 as sg
    rope = sg.make_rope(64, [8, 24])
    g = torch.Generator().manual_seed(0)
    Q, K, tq, tk = (torch.randn(2, h, 33, 64, generator=g) for h in (3, 2, 3, 2))
    pos = torch.randint(0, 5000, (2, 1, 33), generator=g, dtype=torch.int32)
    Qc, Kc = Q.cuda().requires_grad_(), K.cuda().requires_grad_()
    Qo, Ko = sg.sage_rotary(Qc, Kc, pos.cuda(), rope)
    dQ, dK = torch.autograd.grad((Qo ** 4).sum() / 12 + (Ko ** 4).sum() / 12, (Qc, Kc), create_graph=True)
    hQ, hK = torch.autograd.grad((dQ * tq.cuda()).sum() + (dK * tk.cuda()).sum(), (Qc, Kc))
    p = pos.numpy().astype(np.int64)
    for x, t, got in ((Q, tq, hQ), (K, tk, hK)):
        (y, ey), (ty, et) = reference(x.numpy(), p, rope), reference(t.numpy(), p, rope)
        ey, et = ey + U * np.abs(y), et + U * np.abs(ty)
        e = (2 * np.abs(y * ty) * ey + y * y * et) * (1 + 2.0 ** -10) + 16 * U * np.abs(y * y * ty)
        half = rope.rotary // 2
        e = np.concatenate([e[..., :half] + e[..., half:]] * 2, -1)
        want, tol = reference(y * y * ty, p, rope, inverse=True)
        check(got, want, (e + tol) * (1 + 2.0 ** -10))


@pytest.mark.parametrize("causal,dtype,norm", [(False, "fp16", False), (True, "bf16", True)])
def test_attention_with_rope_equals_its_calls(causal, dtype, norm):
    """sage_attention(rope=...) is turn -> quantise -> forward, and backward -> turn back in float32."""
    import bit_trainable_attention_sage_gb300 as sg
    w, x = make_case(256, 64, dtype, causal)
    Q, K, V, dO = (to_dev(x[k], w.dtype) for k in ("Q", "K", "V", "dO"))
    rope = sg.make_rope(64, (8, 12, 12))
    pos = torch.randint(0, 500, (3, 1, 256), generator=torch.Generator().manual_seed(0), dtype=torch.int32).cuda()
    Qr, Kr, Vr = (t.clone().requires_grad_(True) for t in (Q, K, V))
    O = sg.sage_attention(Qr, Kr, Vr, causal=causal, qk_norm=norm, rope=rope, positions=pos)
    O.backward(dO)
    Qt, Kt = sg.sage_rope(Q, K, pos, rope)
    q = sg.sage_quantize_smooth_qknorm(Qt, Kt, V) if norm else sg.sage_quantize_smooth(Qt, Kt, V)
    O2, L2 = sg.sage_attn_fwd(q, causal=causal)
    dQ, dK, dV = sg.sage_attn_bwd(q, V, O2, L2, dO, causal=causal)
    if norm:
        dQ, dK = sg.sage_qknorm_bwd(Qt, q.rQ, dQ)[0], sg.sage_qknorm_bwd(Kt, q.rK, dK)[0]
    dQ, dK = sg.sage_rope(dQ, dK, pos, rope, inverse=True)
    assert sg.sage_device_status() == 0
    assert torch.equal(O, O2)
    assert torch.equal(Kr.grad, dK.to(Q.dtype)) and torch.equal(Vr.grad, dV.to(Q.dtype))
    # dQ is summed with float32 reductions in any order
    assert rel_l2(Qr.grad.float().cpu().numpy(), dQ.to(Q.dtype).float().cpu().numpy()) <= 1e-3
