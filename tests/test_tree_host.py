"""Draft trees and rotary positions on the host: argument checks of the C entry points and of
the binding, the frequency tables, the scratch sizes. No GPU: every refusal comes before a launch."""
import ctypes as C
import math

import pytest
import torch

import synth
from shared_kv_draft_b200 import orthrus
from shared_kv_draft_b200.build import build

P = C.c_void_p(1 << 20)   # an aligned address that no call gets as far as reading
ODD = C.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    build()
    return orthrus.load()


def attention_args(**kw):
    a = dict(q=P, k_cache=P, v_cache=P, k_blk=P, v_blk=P, len=P, n_nodes=None, mask=P, batch=1, n_kv_heads=2, group=4,
             nodes=9, head_dim=128, capacity=64, blk_stride=9, type=orthrus.FP16, out_type=orthrus.BF16, scale=0.0, out=P,
             workspace=P, workspace_bytes=1 << 30, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad,code", [
    ({k: None}, orthrus.ERR_ARG) for k in ("q", "k_cache", "v_cache", "k_blk", "v_blk", "len", "mask", "out", "workspace")
] + [({k: ODD}, orthrus.ERR_ARG) for k in ("q", "k_cache", "v_cache", "k_blk", "v_blk", "out", "mask", "workspace")] + [
    (dict(batch=0), orthrus.ERR_ARG), (dict(batch=1025), orthrus.ERR_ARG), (dict(n_kv_heads=0), orthrus.ERR_ARG),
    (dict(group=0), orthrus.ERR_ARG), (dict(group=33), orthrus.ERR_UNSUPPORTED), (dict(nodes=0), orthrus.ERR_ARG),
    (dict(nodes=257, blk_stride=257), orthrus.ERR_ARG), (dict(head_dim=96), orthrus.ERR_UNSUPPORTED),
    (dict(capacity=0), orthrus.ERR_ARG), (dict(blk_stride=8), orthrus.ERR_ARG), (dict(type=orthrus.FP32), orthrus.ERR_ARG),
    (dict(type=7), orthrus.ERR_ARG), (dict(out_type=orthrus.FP32), orthrus.ERR_ARG), (dict(out_type=-1), orthrus.ERR_ARG),
    (dict(scale=-1.0), orthrus.ERR_ARG), (dict(scale=math.nan), orthrus.ERR_ARG), (dict(scale=math.inf), orthrus.ERR_ARG),
    (dict(workspace_bytes=0), orthrus.ERR_WORKSPACE), (dict(n_kv_heads=1 << 21), orthrus.ERR_UNSUPPORTED),
], ids=str)
def test_tree_attention_refuses(lib, bad, code):
    assert lib.orthrus_tree_attention(*attention_args(**bad)) == code


def test_tree_attention_workspace(lib):
    for args in [(1, 8, 4, 33, 128), (1024, 8, 32, 256, 128), (1, 1, 1, 1, 64), (16, 8, 4, 64, 128)]:
        n = orthrus.tree_attention_workspace_bytes(*args)
        assert 0 < n <= 64 << 20, args
    for args in [(0, 8, 4, 33, 128), (1, 8, 4, 33, 96), (1, 8, 33, 33, 128), (1, 8, 4, 257, 128), (1025, 8, 4, 33, 128)]:
        assert orthrus.tree_attention_workspace_bytes(*args) == 0, args


def commit_args(**kw):
    a = dict(parents=P, tokens=P, argmax=P, n_nodes=None, k_blk=P, v_blk=P, blk_stride=9, k_cache=P, v_cache=P, n_layers=2,
             batch=1, n_kv_heads=2, capacity=64, head_dim=64, nodes=9, len=P, new_len=P, pending=P, accept_len=P, path=P,
             committed=P, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad,code", [
    ({k: None}, orthrus.ERR_ARG) for k in ("parents", "tokens", "argmax", "k_blk", "v_blk", "k_cache", "v_cache", "len",
                                           "new_len", "pending", "accept_len", "path", "committed")
] + [({k: ODD}, orthrus.ERR_ARG) for k in ("k_blk", "v_blk", "k_cache", "v_cache")] + [
    (dict(nodes=0), orthrus.ERR_ARG), (dict(nodes=257, blk_stride=300), orthrus.ERR_ARG), (dict(blk_stride=8), orthrus.ERR_ARG),
    (dict(n_layers=0), orthrus.ERR_ARG), (dict(batch=0), orthrus.ERR_ARG), (dict(batch=2000), orthrus.ERR_ARG),
    (dict(n_kv_heads=0), orthrus.ERR_ARG), (dict(capacity=0), orthrus.ERR_ARG), (dict(head_dim=0), orthrus.ERR_ARG),
    (dict(head_dim=60), orthrus.ERR_UNSUPPORTED), (dict(head_dim=1032), orthrus.ERR_UNSUPPORTED),
    (dict(n_layers=1 << 20, batch=1024, n_kv_heads=64), orthrus.ERR_UNSUPPORTED),
], ids=str)
def test_tree_commit_refuses(lib, bad, code):
    assert lib.orthrus_tree_commit(*commit_args(**bad)) == code


@pytest.mark.parametrize("args", [(None, None, 1, 4, P, P), (P, None, 1, 4, None, P), (P, None, 1, 4, P, None),
                                  (P, None, 0, 4, P, P), (P, None, 1025, 4, P, P), (P, None, 1, 0, P, P),
                                  (P, None, 1, 257, P, P), (P, None, 1, 4, P, ODD)], ids=str)
def test_tree_layout_refuses(lib, args):
    assert lib.orthrus_tree_layout(*args, None, None) == orthrus.ERR_ARG


def test_plan_calls_refuse_a_null_plan(lib):
    assert lib.orthrus_verify_tree(None, P, P, P, None, 4, P, None, None) == orthrus.ERR_ARG
    assert lib.orthrus_accept_commit_tree(None, P, P, P, None, P, 4, P, P, P, None) == orthrus.ERR_ARG


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g2", [0, 1])
def test_the_tree_view_has_kernels_of_its_own(lib, d, g2):
    """The draft and verify views run without the tree view's masks: their kernel has no third view."""
    with open(orthrus.LIB_PATH, "rb") as f:
        built = f.read()
    for tree in (0, 1):
        assert f"orthrus14forward_kernelILi{d}ELb0ELb{g2}ELb{tree}EEE".encode() in built


def test_plans_whose_trees_run_in_one_launch_hold_no_scratch_for_them(lib):
    """Beside the block's depths and visibility words, a plan holds the tree attention's scratch only where a block takes
    the per-op kernels."""
    size = lambda shape, B, cap, K: orthrus.workspace_bytes(orthrus.make_config(shape), B, cap, K, B * (K + 1))  # noqa: E731
    # a whole plan of one sequence of the tiny shape took 22.8 MB before there were trees, with the scratch 42.6 MB
    assert size(synth.TINY, 1, 64, 4) < 23_000_000
    assert size(synth.QWEN3_8B, 1, 64, 4) < 53_100_000


# ---- rotary ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [
    dict(head_dim=0), dict(head_dim=65), dict(head_dim=258), dict(rot_dim=130), dict(rot_dim=3), dict(rot_dim=0),
    dict(theta=1.0), dict(theta=math.nan), dict(theta=math.inf), dict(gain=-1.0), dict(gain=math.inf),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.nan), dict(scaling="by_parts", factor=2.0, original=0),
    dict(scaling="by_parts", factor=2.0, original=100, slow=0.0), dict(scaling="by_index", factor=2.0, original=100, slow=3.0, fast=3.0),
], ids=str)
def test_rope_refuses(lib, kw):
    with pytest.raises(orthrus.OrthrusError) as e:
        orthrus.rope(**{"head_dim": 128, **kw})
    assert e.value.code == orthrus.ERR_ARG


def test_rope_refuses_an_unknown_scaling(lib):
    with pytest.raises(ValueError):
        orthrus.rope(128, scaling="dynamic")


def formula(rot, theta, scaling, factor, original, slow, fast):
    """Turns per position and the gain, from the definition."""
    out = []
    index = lambda r: rot * math.log(original / (2 * math.pi * r)) / (2 * math.log(theta))  # noqa: E731
    for p in range(rot // 2):
        f = theta ** (-2 * p / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_parts":
            k = min(max((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0)
            f *= k + (1 - k) / factor
        elif scaling == "by_index":
            lo = max(math.floor(index(fast)), 0)
            hi = max(min(math.ceil(index(slow)), rot - 1), lo + 1e-3)
            k = 1 - min(max((p - lo) / (hi - lo), 0.0), 1.0)
            f *= k + (1 - k) / factor
        out.append(f / (2 * math.pi))
    return out, (0.1 * math.log(factor) + 1 if scaling.startswith("by") else 1.0)


@pytest.mark.parametrize("scaling", ["none", "linear", "by_parts", "by_index"])
@pytest.mark.parametrize("rot,theta,factor,original,slow,fast", [
    (128, 1.0e6, 4.0, 32768, 1.0, 32.0), (64, 1.0e4, 8.0, 8192, 1.0, 4.0), (2, 1.0e4, 2.0, 100, 0.5, 2.0),
    (128, 5.0e5, 1.0, 4096, 1.0, 32.0), (32, 1.0e4, 40.0, 16, 1.0, 32.0)])
def test_rope_table_is_the_formula(lib, scaling, rot, theta, factor, original, slow, fast):
    r = orthrus.rope(128, rot, theta, scaling=scaling, factor=factor, original=original, slow=slow, fast=fast)
    turns, gain = formula(rot, theta, scaling, factor, original, slow, fast)
    assert (r.head_dim, r.rot_dim, r.interleaved) == (128, rot, 0)
    assert list(r.turns[:rot // 2]) == pytest.approx(turns, rel=1e-14)
    assert r.gain == pytest.approx(gain, rel=2 ** -23)
    assert not any(r.turns[rot // 2:])


@pytest.mark.parametrize("scaling", ["none", "linear", "by_parts", "by_index"])
@pytest.mark.parametrize("rot,theta,factor,original,slow,fast", [
    (128, 17143.79, 1.3, 32768, 1.1, 31.7), (64, 500000.1, 2.7, 8191, 0.9, 3.3), (128, 1.0e6 + 0.1, 1.0 + 1e-9, 100, 0.1, 0.3)])
def test_rope_table_of_parameters_that_fp32_does_not_hold(lib, scaling, rot, theta, factor, original, slow, fast):
    """Rounded to fp32 first they would be off by up to 6e-8, which is 0.06 rad at position 10^6; each of the about
    ten fp64 operations adds 2^-53, and the power's logarithm (below 14) multiplies by 28: 1e-14 in all."""
    r = orthrus.rope(128, rot, theta, scaling=scaling, factor=factor, original=original, slow=slow, fast=fast)
    turns, gain = formula(rot, theta, scaling, factor, original, slow, fast)
    assert list(r.turns[:rot // 2]) == pytest.approx(turns, rel=1e-14)
    assert r.gain == pytest.approx(gain, rel=2 ** -23)


def test_rope_init_takes_the_same_numbers_in_fp32(lib):
    r = orthrus.Rope()
    assert lib.orthrus_rope_init(C.byref(r), 128, 64, 0, 5.0e5, 3, 8.0, 4096, 1.0, 32.0, 0.0) == orthrus.OK
    assert bytes(r) == bytes(orthrus.rope(128, 64, 5.0e5, scaling="by_index", factor=8.0, original=4096))
    assert lib.orthrus_rope_init(None, 128, 64, 0, 5.0e5, 0, 1.0, 1, 1.0, 32.0, 0.0) == orthrus.ERR_ARG
    assert lib.orthrus_rope_init_from(C.byref(r), 128, 64, 0, None, 0, 1, 0.0) == orthrus.ERR_ARG


def test_rope_gain_can_be_set(lib):
    assert orthrus.rope(64, scaling="by_parts", factor=4.0, original=100, gain=1.0).gain == 1.0
    assert orthrus.rope(64, gain=0.5).gain == 0.5


def test_rope_tables_are_the_callers_own(lib):
    r = orthrus.rope(64, theta=1.0e4)
    want = bytes(r)
    r.gain, r.turns[3], r.interleaved = 2.0, 7.0, 1
    assert bytes(orthrus.rope(64, theta=1.0e4)) == want


def rotary_part(**kw):
    a = dict(src=P, dst=P, src_type=orthrus.FP32, dst_type=orthrus.FP16, heads=4, group=1, flags=0, rows=0, src_batch=512,
             src_token=512, src_head=128, dst_batch=512, dst_token=512, dst_kv=128, dst_head=0)
    a.update(kw)
    part = orthrus.RotaryPart()
    for k, v in a.items():
        setattr(part, k, v.value if isinstance(v, C.c_void_p) else v)
    return part


@pytest.mark.parametrize("bad", [
    dict(src=None), dict(dst=None), dict(heads=0), dict(group=0), dict(group=3), dict(src_type=3), dict(dst_type=-1),
    dict(flags=8), dict(flags=orthrus.ROTARY_APPEND, rows=0), dict(heads=65537), dict(src=C.c_void_p(1025)),
    dict(src=ODD), dict(dst=C.c_void_p(1025)), dict(dst_kv=0), dict(group=2)], ids=str)
def test_rotary_refuses_a_part(lib, bad):
    rope = orthrus.rope(128)
    part = (orthrus.RotaryPart * 1)(rotary_part(**bad))
    assert lib.orthrus_rotary(C.byref(rope), part, 1, 1, 1, None, None, 0, None, None) == orthrus.ERR_ARG


def test_rotary_refuses(lib):
    rope, part = orthrus.rope(128), (orthrus.RotaryPart * 4)(*[rotary_part() for _ in range(4)])
    call = lambda r, p, n, b, t: lib.orthrus_rotary(r, p, n, b, t, None, None, 0, None, None)  # noqa: E731
    ref = C.byref(rope)
    assert call(None, part, 1, 1, 1) == orthrus.ERR_ARG
    assert call(ref, None, 1, 1, 1) == orthrus.ERR_ARG
    assert call(ref, part, 0, 1, 1) == orthrus.ERR_ARG
    assert call(ref, part, 4, 1, 1) == orthrus.ERR_ARG
    assert call(ref, part, 1, -1, 1) == orthrus.ERR_ARG
    assert call(ref, part, 1, 1, -1) == orthrus.ERR_ARG
    many = (orthrus.RotaryPart * 2)(rotary_part(heads=16384), rotary_part(heads=1))  # more than 16384 heads in all
    assert call(ref, many, 2, 1, 1) == orthrus.ERR_UNSUPPORTED
    assert call(ref, part, 1, 1 << 16, 1 << 16) == orthrus.ERR_ARG  # more than 2^31 - 1 tokens
    bad = orthrus.Rope(128, 130, 0, 1.0)
    assert call(C.byref(bad), part, 1, 1, 1) == orthrus.ERR_ARG
    assert call(ref, part, 1, 0, 5) == orthrus.OK and call(ref, part, 1, 5, 0) == orthrus.OK  # nothing to do
    flat = (orthrus.RotaryPart * 2)(rotary_part(dst_batch=0), rotary_part(dst_token=0))  # broadcast destinations
    assert call(ref, C.byref(flat, 0), 1, 2, 1) == orthrus.ERR_ARG
    assert call(ref, C.byref(flat, C.sizeof(orthrus.RotaryPart)), 1, 1, 2) == orthrus.ERR_ARG
    empty = (orthrus.RotaryPart * 1)(rotary_part(src=None, dst=None))
    assert call(ref, empty, 1, 0, 5) == orthrus.OK and call(ref, empty, 1, 5, 0) == orthrus.OK
    assert call(ref, empty, 1, 1, 1) == orthrus.ERR_ARG


# ---- the binding's checks (tensors on the CPU are refused before anything else) ------------------------

def test_binding_refuses_cpu_tensors(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    with pytest.raises(ValueError):
        orthrus.tree_layout(i32(1, 4), i32(1, 4), torch.zeros((1, 4, 1), dtype=torch.int64))
    with pytest.raises(ValueError):
        orthrus.tree_attention(f16(1, 2, 8, 64), f16(1, 2, 16, 64), f16(1, 2, 16, 64), f16(1, 2, 4, 64), f16(1, 2, 4, 64),
                               i32(1), torch.zeros((1, 4, 1), dtype=torch.int64), f16(4, 256), f16(8))
    with pytest.raises(ValueError):
        orthrus.tree_commit(i32(1, 4), i32(1, 4), i32(1, 4), f16(1, 1, 2, 4, 64), f16(1, 1, 2, 4, 64), f16(1, 1, 2, 16, 64),
                            f16(1, 1, 2, 16, 64), i32(1), i32(1), i32(1), i32(1), i32(1, 4), i32(1, 4))
    with pytest.raises(ValueError):
        orthrus.rotary(orthrus.rope(64), [(torch.zeros(1, 2, 3, 64), torch.zeros(1, 2, 3, 64))])
    with pytest.raises(ValueError):
        orthrus.rotary(orthrus.rope(64), [])
