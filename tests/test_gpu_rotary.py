"""orthrus_rotary on the GPU against its definition in float64.

Bound of one value y = gain (x1 cos a - x2 sin a), derived: the angle is off by at most half a step
of the fp32 remainder (2^-26 turns, 2 pi 2^-26 < 2^-23 rad) and, at |pos| <= 2^24, less than 2^-29
turns from the fp64 product; sincospi adds 2 ulp (2^-23) and the gain, the two products and their
sum a rounding each (4 x 2^-24). Together below 2^-21 gain (|x1| + |x2|); then the roundings to bf16
(when asked) and to the destination's type, half a step each.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F32, F16, B16 = torch.float32, torch.float16, torch.bfloat16


def lib():
    from shared_kv_draft_b200 import orthrus
    return orthrus


def normal(shape, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(t)


def reference(x, pos, rope, inverse=False, copy=False):
    """x [B][T][h][d], pos [B][T]: (float64 result, |x1| + |x2| of every value's pair)."""
    x = x.double()
    if copy:
        return x, torch.zeros_like(x)
    rot = rope.rot_dim
    f = torch.tensor(list(rope.turns[:rot // 2]), dtype=torch.float64, device="cuda") * (2 * math.pi)
    a = pos.double().cuda()[..., None] * f * (-1 if inverse else 1)
    c, s = (torch.cos(a) * rope.gain)[:, :, None], (torch.sin(a) * rope.gain)[:, :, None]
    y, mag = x.clone(), torch.zeros_like(x)
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if rope.interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    x1, x2 = x[..., one], x[..., two]
    y[..., one], y[..., two] = x1 * c - x2 * s, x2 * c + x1 * s
    mag[..., one] = mag[..., two] = rope.gain * (x1.abs() + x2.abs())
    return y, mag


def check(got, x, pos, rope, inverse=False, copy=False, bf16_values=False):
    ref, mag = reference(x, pos, rope, inverse, copy)
    u = HALF_STEP[got.dtype] + (2.0 ** -8 if bf16_values else 0.0)
    tol = 2.0 ** -21 * mag * 1.01 + 1.01 * u * (ref.abs() + 2.0 ** -20 * mag) + (2.0 ** -25 if got.dtype is F16 else 0.0)
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (128, 64), (128, 32), (64, 16), (256, 256), (80, 48), (96, 20), (10, 2), (6, 6)])
def test_layouts_and_partial_heads(d, rot, interleaved):
    o = lib()
    rope = o.rope(d, rot, 1.0e4, interleaved=interleaved)
    x = normal((2, 7, 5, d), F32, d + rot)
    y = torch.empty_like(x)
    o.rotary(rope, [(x, y)])
    check(y, x, torch.arange(7).expand(2, 7), rope)
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dst", [F32, F16, B16], ids=str)
@pytest.mark.parametrize("src", [F32, F16, B16], ids=str)
def test_types(src, dst):
    o = lib()
    for interleaved in (False, True):
        rope = o.rope(128, 96, interleaved=interleaved)
        x, z = normal((1, 33, 8, 128), src, 1), normal((1, 33, 2, 128), src, 2)
        y, w = torch.empty((1, 33, 8, 128), dtype=dst, device="cuda"), torch.empty((1, 33, 2, 128), dtype=dst, device="cuda")
        o.rotary(rope, [(x, y), (z, w, o.ROTARY_BF16_VALUES)])
        pos = torch.arange(33)[None]
        check(y, x, pos, rope)
        check(w, z, pos, rope, bf16_values=True)
        o.rotary(rope, [(x, y, o.ROTARY_COPY)])
        assert torch.equal(y, x.to(dst))


@pytest.mark.parametrize("B,T,H,Hkv", [(1, 1, 1, 1), (1, 1, 32, 8), (3, 5, 6, 3), (1, 33, 32, 8), (2, 700, 8, 2), (1, 5000, 4, 1)])
def test_sizes(B, T, H, Hkv):
    o = lib()
    rope = o.rope(128, theta=1.0e6)
    q, k = normal((B, T, H, 128), B16, 3), normal((B, T, Hkv, 128), B16, 4)
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    base = torch.tensor([1000 * b for b in range(B)], dtype=torch.int32, device="cuda")
    o.rotary(rope, [(q, yq), (k, yk)], len=base)
    pos = base.cpu()[:, None] + torch.arange(T)
    check(yq, q, pos, rope)
    check(yk, k, pos, rope)


@pytest.mark.parametrize("B,T", [(0, 5), (2, 0)])
def test_no_tokens(B, T):
    o = lib()
    x, cache = normal((B, T, 4, 64), B16, 19), torch.zeros((B, 8, 4, 64), device="cuda")
    y = torch.empty_like(x)
    o.rotary(o.rope(64), [(x, y), (x, cache, o.ROTARY_APPEND)], len=torch.zeros(B, dtype=torch.int32, device="cuda"))
    assert not cache.any()


def test_broadcast_source_and_destination():
    o = lib()
    rope = o.rope(64)
    x = normal((1, 1, 2, 64), F32, 20).expand(3, 5, 2, 64)
    y = torch.empty((3, 5, 2, 64), device="cuda")
    o.rotary(rope, [(x, y)])
    check(y, x, torch.arange(5).expand(3, 5), rope)
    for flat in (y[:1].expand(3, 5, 2, 64), y[:, :1].expand(3, 5, 2, 64), y[:, :, :1].expand(3, 5, 2, 64)):
        with pytest.raises(o.OrthrusError):
            o.rotary(rope, [(y.clone(), flat)])


@pytest.mark.parametrize("d", [128, 20])
@pytest.mark.parametrize("T", [2367, 2368, 5000, 20001])
def test_one_head_of_many_tokens(T, d):
    o = lib()
    rope = o.rope(d)
    x = normal((1, T, 1, d), B16, 18)
    y = torch.empty_like(x)
    o.rotary(rope, [(x, y)])
    check(y, x, torch.arange(T)[None], rope)


@pytest.mark.parametrize("scaling", ["none", "linear", "by_parts", "by_index"])
def test_far_positions_and_stretched_contexts(scaling):
    """Positions up to 16 million, negative ones among them."""
    o = lib()
    rope = o.rope(128, theta=1.0e6, scaling=scaling, factor=4.0, original=32768)
    x = normal((1, 9, 2, 128), F32, 5)
    off = torch.tensor([[0, 1, -1, 131071, 999_983, -999_983, 2 ** 24 - 1, 8_388_609, 40_000]], dtype=torch.int32)
    y = torch.empty_like(x)
    o.rotary(rope, [(x, y)], offsets=off.cuda())
    check(y, x, off, rope)
    o.rotary(rope, [(x, y)], len=torch.tensor([-5], dtype=torch.int32, device="cuda"), offsets=off.cuda())
    check(y, x, off - 5, rope)


def test_gradient_is_the_inverse_call():
    """For y = R x: <g, R x> = <R^T g, x>, and the difference quotient of <g, R x> along a direction."""
    o = lib()
    for interleaved in (False, True):
        rope = o.rope(128, 64, 1.0e4, interleaved=interleaved, scaling="by_parts", factor=8.0, original=4096)
        x, g, v = (normal((2, 19, 3, 128), F32, s) for s in (6, 7, 8))
        turn = lambda t, inverse=False: _turned(o, rope, t, inverse)  # noqa: E731
        gx = turn(g, True)
        check(gx, g, torch.arange(19).expand(2, 19), rope, inverse=True)
        dot = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
        scale = float(g.double().norm() * x.double().norm())
        assert abs(dot(g, turn(x)) - dot(gx, x)) <= 2.0 ** -19 * scale
        h = 2.0 ** -3  # the map is linear: any step gives the derivative, up to the rounding of x + h v
        slope = (dot(g, turn(x + h * v)) - dot(g, turn(x - h * v))) / (2 * h)
        assert abs(slope - dot(gx, v)) <= 2.0 ** -16 * scale
        # there and back: the gain squared on the rotated dims
        back = turn(turn(x), True)
        want = x.clone()
        want[..., :64] *= rope.gain ** 2
        assert float((back - want).abs().max()) <= 2.0 ** -18 * float(want.abs().max()) * 4


def _turned(o, rope, t, inverse):
    y = torch.empty_like(t)
    o.rotary(rope, [(t, y)], inverse=inverse)
    return y


@pytest.mark.parametrize("odd", [False, True], ids=["aligned", "odd"])
def test_strided_views_and_in_place(odd):
    """Views of a fused projection with any strides; elements around them stay as they were."""
    o = lib()
    rope = o.rope(64)
    pad = 3 if odd else 16
    buf = normal((2, 11, 9 * 64 + pad), F32, 9)
    before = buf.clone()
    x = buf[:, :, :6 * 64].unflatten(2, (6, 64))
    big = torch.full((2, 6, 15, 64 + pad), 5.0, device="cuda")
    y = big[:, :, 2:13, pad:].transpose(1, 2)
    o.rotary(rope, [(x, y)])
    pos = torch.arange(11).expand(2, 11)
    check(y, x, pos, rope)
    assert torch.equal(buf, before)
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[:, :, 2:13, pad:] = False
    assert (big[mask] == 5.0).all()
    x0 = x.clone()
    o.rotary(rope, [(x, x)])  # in place
    check(x, x0, pos, rope)
    assert torch.equal(buf[:, :, 6 * 64:], before[:, :, 6 * 64:])
    # every other head, reversed use of memory through an expanded source
    one = normal((1, 1, 6, 64), F32, 10).expand(2, 11, 6, 64)
    y2 = torch.empty((2, 11, 6, 64), device="cuda")
    o.rotary(rope, [(one, y2)])
    check(y2, one, pos, rope)


def test_append_to_a_cache_and_the_attention_q_layout():
    o = lib()
    B, T, Hkv, G, d, cap = 3, 9, 2, 4, 128, 40
    rope = o.rope(d)
    qkv = normal((B, T, Hkv * (G + 2), d), F32, 11)
    q, k, v = qkv.split((Hkv * G, Hkv, Hkv), 2)
    lens, depth = torch.tensor([0, 13, 31], dtype=torch.int32), torch.randint(0, 9, (B, T), dtype=torch.int32)
    kc, vc = (torch.full((B, Hkv, cap, d), 3.0, dtype=F16, device="cuda") for _ in range(2))
    qo = torch.zeros((B, Hkv, T * G, d), dtype=F16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    flags = o.ROTARY_APPEND | o.ROTARY_BF16_VALUES
    parts = [(q, qo.view(B, Hkv, T, G, d).permute(0, 2, 1, 3, 4)), (k, kc.transpose(1, 2), flags),
             (v, vc.transpose(1, 2), flags | o.ROTARY_COPY)]
    o.rotary(rope, parts, len=lens.cuda(), offsets=depth.cuda(), status=status)
    assert int(status.item()) == 0
    pos = lens[:, None] + depth
    check(qo.view(B, Hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, d), q, pos, rope)
    for b in range(B):
        n = int(lens[b])
        check(kc[b:b + 1, :, n:n + T].transpose(1, 2), k[b:b + 1], pos[b:b + 1], rope, bf16_values=True)
        assert torch.equal(vc[b, :, n:n + T].transpose(0, 1), v[b].bfloat16().half())
        for c in (kc, vc):
            assert (c[b, :, :n] == 3.0).all() and (c[b, :, n + T:] == 3.0).all()


@pytest.mark.parametrize("d", [64, 10])
def test_append_without_room(d):
    """Rows past the end (or before the start) are not written, the others are, and the status says so."""
    o = lib()
    rope = o.rope(d)
    k = normal((2, 5, 2, d), F32, 12)
    for lens, keep in (([7, 0], [3, 5]), ([0, 12], [5, 0]), ([-2, 1], [3, 5])):
        cache = torch.full((2, 2, 10, d), 3.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o.rotary(rope, [(k, cache.transpose(1, 2), o.ROTARY_APPEND)],
                 len=torch.tensor(lens, dtype=torch.int32, device="cuda"), status=status)
        assert int(status.item()) == o.ERR_CAPACITY
        want = torch.full_like(cache, 3.0)
        full = torch.empty((2, 5, 2, d), device="cuda")
        o.rotary(rope, [(k, full)], len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        for b in range(2):
            for t in range(5):
                if 0 <= lens[b] + t < 10:
                    want[b, :, lens[b] + t] = full[b, t]
        assert torch.equal(cache, want)


def test_matches_the_decode_path_frequencies():
    """The table of the decoder's own rotary embedding: oracle.model.rope at the cache's positions."""
    from oracle.model import rope as turned
    o = lib()
    x = normal((1, 6, 4, 128), F32, 13)
    y = torch.empty_like(x)
    o.rotary(o.rope(128, theta=1.0e6), [(x, y)], len=torch.tensor([1021], dtype=torch.int32, device="cuda"))
    ref = turned(x[0].double().cpu(), torch.arange(1021, 1027), 1.0e6)
    assert float((y[0].cpu().double() - ref).abs().max()) <= 2.0 ** -20 * 2 * float(x.abs().max())


def test_offsets_past_32_bits():
    """A head past 2^31 elements of a large cache."""
    o = lib()
    rope = o.rope(128)
    cap = 17_000_000
    cache = torch.empty((1, 2, cap, 128), dtype=F16, device="cuda")
    k = normal((1, 4, 2, 128), F32, 14)
    n = cap - 4
    o.rotary(rope, [(k, cache.transpose(1, 2), o.ROTARY_APPEND | o.ROTARY_BF16_VALUES)],
             len=torch.tensor([n], dtype=torch.int32, device="cuda"))
    pos = n + torch.arange(4)[None]
    # 17 million positions: the fp64 product is off by up to 2^-53 x 2.7 million turns, still far below 2^-26
    check(cache[:, :, n:].transpose(1, 2), k, pos, rope, bf16_values=True)


def test_captured_and_on_another_stream():
    o = lib()
    rope = o.rope(128)
    x, y = normal((2, 40, 8, 128), F32, 15), torch.zeros((2, 40, 8, 128), dtype=F16, device="cuda")
    base = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o.rotary(rope, [(x, y)], len=base, stream=side)
    side.synchronize()
    check(y, x, torch.arange(40).expand(2, 40), rope)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.rotary(rope, [(x, y)], len=base)
    for step in (100, 200_000):
        base.fill_(step)
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        check(y, x, step + torch.arange(40).expand(2, 40), rope)


def test_binding_refuses_what_does_not_fit():
    o = lib()
    rope = o.rope(64)
    x = normal((1, 3, 2, 64), F32, 16)
    y = torch.empty_like(x)
    for parts in ([(x.double(), y)], [(x, y.double())], [(x[..., :32], y)], [(x, y[..., :32])], [(x, y[:, :2])],
                  [(x, y[:, :, :1])], [(x.transpose(2, 3), y)], [(x, y.cpu())], [(x[0], y)], [(x, y)] * 4,
                  [(x, y), (x[:, :2], y[:, :2])]):
        with pytest.raises(ValueError):
            o.rotary(rope, parts)
    with pytest.raises(ValueError):
        o.rotary(rope, [(x, y)], offsets=torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        o.rotary(rope, [(x, y)], len=torch.zeros(1, device="cuda"))
    with pytest.raises(o.OrthrusError):
        o.rotary(rope, [(x, y, 64)])
