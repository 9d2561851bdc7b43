"""Draft trees on the GPU against definitions in float64 / plain Python.

* Layout: depths and visibility words of chains, stars, forests, random and invalid trees.
* Attention: every row against a float64 softmax over the same 16-bit inputs. The bound is
  elementwise and derived, see `attention_bound`.
* Commit: the walk and the K/V rows, exactly, everything else of the cache unchanged.
* The operators one after another, as a layer uses them; the plan's tree step against the
  oracle; captured, on a second stream, with stale scratch.
"""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import Oracle, greedy_ar, top2_margin

pytestmark = pytest.mark.gpu

CUDA = dict(device="cuda")
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def lib():
    from shared_kv_draft_b200 import orthrus
    return orthrus


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def random_parents(B, N, seed, spread=8):
    rng = np.random.default_rng(seed)
    return np.array([[-1] + [int(rng.integers(max(0, i - spread), i)) for i in range(1, N)] for _ in range(B)], np.int32)


def visibility(parents, counts=None):
    B, N = parents.shape
    see = np.zeros((B, N, N), bool)
    for b in range(B):
        for i in range(N if counts is None else counts[b]):
            j = i
            while j >= 0:
                see[b, i, j] = True
                j = parents[b, j] if parents[b, j] < j else -1
    return see


def words_of(see):
    B, N, _ = see.shape
    W = (N + 63) // 64
    bits = np.zeros((B, N, W * 64), np.uint8)
    bits[:, :, :N] = see
    return torch.from_numpy(np.packbits(bits, axis=2, bitorder="little").view("<i8").reshape(B, N, W).copy()).cuda()


# ---- layout --------------------------------------------------------------------------------------

def run_layout(parents, counts=None):
    o = lib()
    B, N = parents.shape
    depth = torch.full((B, N), -7, dtype=torch.int32, **CUDA)
    mask = torch.full((B, N, (N + 63) // 64), -7, dtype=torch.int64, **CUDA)
    status = torch.zeros(1, dtype=torch.int32, **CUDA)
    o.tree_layout(i32(parents), depth, mask, n_nodes=None if counts is None else i32(counts), status=status)
    return depth.cpu().numpy(), mask, int(status.item())


@pytest.mark.parametrize("B,N", [(1, 1), (1, 2), (3, 31), (2, 33), (1, 64), (2, 65), (5, 100), (2, 128), (1, 200), (3, 256)])
def test_layout(B, N):
    trees = {"random": random_parents(B, N, N), "chain": np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1)),
             "star": np.tile(np.array([-1] + [0] * (N - 1), np.int32), (B, 1)), "forest": np.full((B, N), -1, np.int32),
             "wide": random_parents(B, N, N + 1, spread=N)}
    for name, parents in trees.items():
        counts = [max(0, N - 3 * b) for b in range(B)]
        for c in (None, counts):
            depth, mask, status = run_layout(parents, c)
            see = visibility(parents, c)
            assert status == 0
            assert torch.equal(mask, words_of(see)), name
            assert (depth == np.maximum(see.sum(2) - 1, 0)).all(), name


def test_layout_flags_invalid_parents():
    parents = np.array([[-1, 0, 2, 5, -2, 3]], np.int32)  # 2 and 3 point at or past themselves, 4 below -1
    depth, mask, status = run_layout(parents)
    assert status == lib().ERR_ARG
    fixed = np.array([[-1, 0, -1, -1, -1, 3]], np.int32)
    assert torch.equal(mask, words_of(visibility(fixed)))
    assert depth.tolist() == [[0, 1, 0, 0, 0, 1]]


def test_layout_flags_node_counts_out_of_range():
    for bad in (-1, 7):
        depth, mask, status = run_layout(random_parents(1, 6, 0), [bad])
        assert status == lib().ERR_ARG
        assert bool(mask.any()) == (bad == 7)


# ---- attention ------------------------------------------------------------------------------------

def attention_bound(q, keys, vals, seen, scale, n_keys, t, u_out):
    """Float64 result and the elementwise bound of one KV head.

    out = sum p v / sum p. Per key, |error of p / p| is at most
      scores: fp32 accumulation of d products, (d + 2) 2^-24 scale sum|q k|, and as much for the
              reference point, plus the multiplications by the scale (2 x 2^-24 |s|);
      exp2:   2^-21 (2 ulp and the argument's rounding near zero are below that);
      sums:   at most n / 128 + 160 additions in a row, 2^-24 each, for l and for the products;
      P:      half a step of the type for the weights that multiply V (a weight below 2^-14 of the
              type's normal range: 2^-25 absolute, scaled up by at least 2^6 against the row's maximum).
    The numerator's error is then at most that times sum p|v|, the denominator's that times out,
    and sum p|v| >= |out|. The result is rounded once more on the way out.
    """
    z = (q @ keys.T) * scale
    mag = (q.abs() @ keys.abs().T * scale).masked_fill(~seen, 0.0).amax(1, keepdim=True) if keys.shape[0] else q.new_zeros(q.shape[0], 1)
    z = z.masked_fill(~seen, -math.inf)
    any_seen = seen.any(1, keepdim=True)
    p = torch.where(any_seen, torch.softmax(z, 1), torch.zeros((), dtype=z.dtype, device=z.device))
    vals = torch.where(seen.any(0)[:, None], vals, torch.zeros((), dtype=z.dtype, device=z.device))
    out, spread = p @ vals, p @ vals.abs()
    d = q.shape[1]
    rel = 2 * ((d + 4) * 2.0 ** -24 * mag + 2.0 ** -21 + (n_keys / 128 + 160) * 2.0 ** -24) + HALF_STEP[t]
    tiny = 2.0 ** -31 * (seen.double() @ vals.abs())  # weights under the type's range
    return out, rel * spread * 1.01 + tiny + u_out * out.abs() + 2.0 ** -24


def make_attention(B, Hkv, G, N, d, cap, lens, t=torch.float16, seed=0, counts=None, see=None, blk_stride=None, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (torch.randn(s, generator=g, **CUDA) * std).to(t)  # noqa: E731
    S = blk_stride or N
    parents = random_parents(B, N, seed)
    see = visibility(parents, counts) if see is None else see
    return dict(q=r(B, Hkv, N * G, d), k_cache=r(B, Hkv, cap, d), v_cache=r(B, Hkv, cap, d), k_blk=r(B, Hkv, S, d),
                v_blk=r(B, Hkv, S, d), len=i32(lens), mask=words_of(see), see=see, counts=counts, lens=list(lens), G=G, N=N)


def call_attention(a, out_type=None, planes=False, scale=0.0, workspace=None, out=None, stream=None):
    o = lib()
    B, Hkv, R, d = a["q"].shape
    N, G = a["N"], a["G"]
    t = out_type or a["q"].dtype
    if out is None:
        shape = (2, B * N, Hkv * G * d) if planes else (B * N, Hkv * G * d)
        out = torch.full(shape, 7.0, dtype=torch.bfloat16 if planes else t, **CUDA)
    if workspace is None:  # stale scratch: the kernels may not read what they have not written
        n = o.tree_attention_workspace_bytes(B, Hkv, G, N, d)
        workspace = torch.full((n,), 0xff, dtype=torch.uint8, **CUDA)
    status = torch.zeros(1, dtype=torch.int32, **CUDA)
    o.tree_attention(a["q"], a["k_cache"], a["v_cache"], a["k_blk"], a["v_blk"], a["len"], a["mask"], out, workspace,
                     n_nodes=None if a["counts"] is None else i32(a["counts"]), scale=scale, status=status, stream=stream)
    return out, status


def check_attention(a, out, planes=False, scale=0.0):
    B, Hkv, R, d = a["q"].shape
    N, G = a["N"], a["G"]
    t = a["q"].dtype
    assert torch.isfinite(out).all()
    got = (out[0].double() + out[1].double() if planes else out.double()).view(B, N, Hkv, G, d)
    u_out = 2.0 ** -16 if planes else HALF_STEP[out.dtype]
    scale = scale or d ** -0.5
    worst = 0.0
    for b in range(B):
        n, live = a["lens"][b], N if a["counts"] is None else a["counts"][b]
        if live < N:  # padding rows are left as they were
            left = out[:, b * N + live:(b + 1) * N] if planes else out[b * N + live:(b + 1) * N]
            assert (left == 7.0).all()
        if live == 0:
            continue
        see = torch.from_numpy(a["see"][b, :live, :live].copy()).cuda()
        seen = torch.cat([torch.ones((live, n), dtype=torch.bool, **CUDA), see], 1).repeat_interleave(G, 0)
        for h in range(Hkv):
            keys = torch.cat([a["k_cache"][b, h, :n], a["k_blk"][b, h, :live]]).double()
            vals = torch.cat([a["v_cache"][b, h, :n], a["v_blk"][b, h, :live]]).double()
            q = a["q"][b, h, :live * G].double()
            ref, tol = attention_bound(q, keys, vals, seen, scale, n + live, t, u_out)
            err = (got[b, :live, h].reshape(live * G, d) - ref).abs()
            worst = max(worst, float((err / tol).max()))
            assert (err <= tol).all(), (b, h, float((err / tol).max()))
    return worst


def run_attention(*args, planes=False, out_type=None, scale=0.0, **kw):
    a = make_attention(*args, **kw)
    out, status = call_attention(a, planes=planes, out_type=out_type, scale=scale)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check_attention(a, out, planes, scale)
    again, _ = call_attention(a, planes=planes, out_type=out_type, scale=scale)
    assert torch.equal(out, again)  # the same inputs, the same bits
    return a, out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 127, 128, 129, 255, 300, 1000, 2111])
def test_attention_cache_lengths(n, d):
    run_attention(1, 2, 4, 9, d, 2112, [n], seed=n)


@pytest.mark.parametrize("N", [1, 2, 16, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200, 256])
def test_attention_tree_sizes(N):
    run_attention(1, 2, 4, N, 128, 384, [200], seed=N)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 32])
def test_attention_groups(G, d):
    run_attention(2, 3, G, 11, d, 320, [37, 250], seed=G)


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("out_type,planes", [(torch.float16, False), (torch.bfloat16, False), (None, True)],
                         ids=["to_fp16", "to_bf16", "to_planes"])
def test_attention_types(t, out_type, planes):
    run_attention(2, 2, 4, 33, 128, 700, [650, 129], t=t, seed=3, out_type=out_type, planes=planes)


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_attention_ragged_batch(t):
    """Lengths from none to several thousand keys in one batch, trees of different sizes, one
    idle sequence, a scratch block with more rows than nodes."""
    run_attention(7, 2, 4, 33, 128, 4000, [0, 3963, 1, 128, 2049, 700, 64], t=t, seed=5,
                  counts=[33, 20, 1, 0, 33, 32, 7], blk_stride=40)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_units_of_both_kinds(d):
    """40 nodes x 8 heads are 320 rows, one unit of 256 rows and one of 64 for each KV head; with other sequences
    of 1 to 39 nodes a CTA goes from units of more than 128 rows to smaller ones and back."""
    B = 20
    run_attention(B, 4, 8, 40, d, 1600, [(397 * b) % 1500 for b in range(B)], seed=20, counts=[40 - (b * 7) % 40 for b in range(B)])


def test_attention_random_cases():
    """Sizes, lengths, types and node counts drawn at random, everything dead poisoned."""
    import random
    rng = random.Random(23)
    for _ in range(60):
        d, G, N = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 8, 16, 32]), rng.choice([1, 2, 7, 16, 33, 64, 65, 90, 130, 256])
        B, H, most = rng.choice([1, 1, 2, 5, 20, 70]), rng.choice([1, 2, 3, 8]), rng.choice([0, 5, 70, 300, 1500])
        if B * H * N * G * (most + N) > 3e8:
            continue
        lens = [rng.randint(0, most) for _ in range(B)]
        counts = None if rng.random() < 0.4 else [rng.randint(0, N) for _ in range(B)]
        a = make_attention(B, H, G, N, d, max(1, max(lens)) + rng.choice([0, 1, 50]), lens, seed=rng.randint(0, 10 ** 6),
                           t=rng.choice([torch.float16, torch.bfloat16]), counts=counts, blk_stride=N + rng.choice([0, 3]))
        for b in range(B):
            live = N if counts is None else counts[b]
            for x in (a["k_cache"], a["v_cache"]):
                x[b, :, lens[b]:] = float("nan")
            for x in (a["k_blk"], a["v_blk"]):
                x[b, :, live:] = float("nan")
            a["q"][b, :, live * G:] = float("nan")
        planes = rng.random() < 0.3
        out, status = call_attention(a, planes=planes)
        assert int(status.item()) == 0
        check_attention(a, out, planes)


def test_attention_many_sequences():
    run_attention(200, 1, 2, 5, 64, 192, [(37 * b) % 180 for b in range(200)], seed=6, counts=[b % 6 for b in range(200)])


def test_attention_long_cache():
    run_attention(1, 2, 4, 17, 128, 33000, [32777], seed=7)


def test_attention_scale_and_large_scores():
    """A given scale; scores of up to about +-100, so that the maximum moves by far between tiles."""
    run_attention(1, 2, 4, 9, 128, 1400, [1300], seed=8, scale=0.031)
    run_attention(1, 2, 4, 9, 128, 1400, [1300], seed=9, std=3.0)


def test_attention_rising_and_falling_maximum():
    """Keys whose scores rise (then fall) steadily along the cache: the running maximum changes in
    every tile, or never after the first."""
    for sign in (1.0, -1.0):
        a = make_attention(1, 2, 2, 7, 128, 1600, [1555], seed=10)
        ramp = torch.linspace(-4.0, 4.0, 1600, **CUDA) * sign
        a["q"] = (a["q"] * 0 + 1.0).contiguous()
        a["k_cache"] = (a["k_cache"] * 0.05 + ramp[None, None, :, None]).to(torch.float16).contiguous()
        out, status = call_attention(a)
        assert int(status.item()) == 0
        check_attention(a, out)


def test_attention_arbitrary_masks_and_empty_rows():
    """Visibility that is no tree: random, full, none; rows that see nothing at all are zero."""
    N = 70
    rng = np.random.default_rng(11)
    for lens in ([0, 0, 90], [5, 0, 200]):
        see = rng.random((3, N, N)) < 0.1
        see[0, :N // 2] = False
        see[1] = False
        see[2] = True
        a = make_attention(3, 2, 4, N, 128, 256, lens, seed=12, see=see)
        out, status = call_attention(a)
        assert int(status.item()) == 0
        check_attention(a, out)
        rows = out.view(3, N, -1)
        if lens[0] == 0:
            assert (rows[0, :N // 2] == 0).all()
        assert (rows[1] == 0).all()


def test_attention_never_reads_dead_rows():
    """NaN and infinities past the live rows of the cache, in padding nodes' K, V and q, in scratch
    rows past the tree; words with bits set for nodes that do not exist."""
    B, Hkv, G, N, d = 3, 2, 4, 33, 128
    lens, counts = [130, 0, 257], [33, 20, 1]
    a = make_attention(B, Hkv, G, N, d, 640, lens, seed=13, counts=counts, blk_stride=50)
    for b in range(B):
        for x, y in ((a["k_cache"], a["v_cache"]), (a["k_blk"], a["v_blk"])):
            lo = lens[b] if x is a["k_cache"] else counts[b]
            x[b, :, lo:] = float("nan")
            y[b, :, lo::2] = float("inf")
            y[b, :, lo + 1::2] = float("nan")
        a["q"][b, :, counts[b] * G:] = float("nan")
    words = a["mask"].cpu().numpy().view(np.uint64)
    for b in range(B):
        words[b, :, 0] |= np.uint64(((1 << 64) - 1) ^ ((1 << counts[b]) - 1))
    a["mask"] = torch.from_numpy(words.view(np.int64)).cuda()
    out, status = call_attention(a)
    assert int(status.item()) == 0
    check_attention(a, out)


def test_attention_nan_of_one_branch_stays_there():
    """A node whose K or V is not finite reaches the nodes that see it and no others. (An infinite K may
    give the score -inf, a weight of zero: only NaN is tried there.)"""
    N, G = 24, 4
    for which, value in (("k_blk", float("nan")), ("v_blk", float("nan")), ("v_blk", float("inf"))):
        a = make_attention(1, 2, G, N, 128, 256, [140], seed=14)
        ref, _ = call_attention(a)
        ref = ref.view(N, 2, G, 128)
        a[which][0, 1, 5, 3] = value
        out, status = call_attention(a)
        assert int(status.item()) == 0
        got = out.view(N, 2, G, 128)
        sees = torch.from_numpy(a["see"][0, :, 5].copy()).cuda()
        assert sees.any() and not sees.all()
        assert not torch.isfinite(got[sees][:, 1]).all(dim=-1).any()
        assert torch.equal(got[~sees], ref[~sees])
        assert torch.equal(got[:, 0], ref[:, 0])


def test_attention_flags_lengths_out_of_range():
    for bad, code in ((-3, lib().ERR_ARG), (300, lib().ERR_CAPACITY)):
        a = make_attention(2, 2, 4, 9, 128, 256, [bad, 40], seed=15)
        out, status = call_attention(a)
        assert int(status.item()) == code
        a["lens"] = [min(max(bad, 0), 256), 40]
        check_attention(a, out)  # clamped, and the other sequence is right


def test_attention_offsets_past_32_bits():
    """A cache of 2 heads x 17 million rows: the second head starts past 2^31 elements."""
    cap, n, N, G, d = 17_000_000, 300, 9, 4, 128
    a = make_attention(1, 2, G, N, d, 512, [n], seed=16)
    small = a["k_cache"], a["v_cache"]
    big = []
    for x in small:
        y = torch.empty((1, 2, cap, d), dtype=torch.float16, **CUDA)
        y[:, :, :512] = x
        big.append(y)
    ref, _ = call_attention(a)
    a["k_cache"], a["v_cache"] = big
    out, status = call_attention(a)
    assert int(status.item()) == 0
    check_attention({**a, "k_cache": small[0], "v_cache": small[1]}, out)
    # and with the live rows at the far end of a cache that is full past 2^31 bytes of one head
    n2 = 9_000_000
    a["len"], a["lens"] = i32([n2]), [n2]
    big[0][:, :, 512:n2].normal_()
    big[1][:, :, 512:n2].normal_()
    out, status = call_attention(a)
    assert int(status.item()) == 0
    h, see = 1, torch.from_numpy(a["see"][0].copy()).cuda().repeat_interleave(G, 0)
    keys = torch.cat([big[0][0, h, :n2], a["k_blk"][0, h]])
    vals = torch.cat([big[1][0, h, :n2], a["v_blk"][0, h]])
    q = a["q"][0, h].double()
    m = torch.full((N * G, 1), -math.inf, dtype=torch.float64, **CUDA)
    l, acc = torch.zeros_like(m), torch.zeros((N * G, d), dtype=torch.float64, **CUDA)
    for lo in range(0, n2 + N, 1_000_000):
        hi = min(lo + 1_000_000, n2 + N)
        z = q @ keys[lo:hi].double().T * d ** -0.5
        if hi > n2:
            z[:, n2 - lo:] = z[:, n2 - lo:].masked_fill(~see, -math.inf)
        m2 = torch.maximum(m, z.amax(1, keepdim=True))
        p, f = torch.exp(z - m2), torch.exp(m - m2)
        l, acc, m = l * f + p.sum(1, keepdim=True), acc * f + p @ vals[lo:hi].double(), m2
    got = out.view(N, 2, G, d)[:, h].reshape(N * G, d).double()
    # nine million random values average out to about 1e-3: compare with the scale of one weighted value
    assert (got - acc / l).abs().max() <= 2.0 ** -11 * 3.0


def test_attention_rows_past_32_bits_decide():
    """One head of 16.9 million rows whose result comes from 128 of them: 64 past 2^31 bytes of K and V, 64 past 2^32,
    their V values far apart. All other K and V are zero: a row that is skipped, or read from 2^31 or 2^32 bytes before
    its place, moves the result, about 0.5, towards 2 or -1: by far more than the bound."""
    n, N, G, d = 16_900_001, 3, 4, 128
    a = make_attention(1, 1, G, N, d, 64, [0], seed=24, see=np.eye(N, dtype=bool)[None])
    g = torch.Generator(device="cuda").manual_seed(25)
    r = lambda *s: torch.randn(s, generator=g, **CUDA)  # noqa: E731
    lo, hi = 2 ** 31 // (2 * d), 2 ** 32 // (2 * d)
    far = torch.cat([torch.arange(lo, lo + 32), torch.arange(hi - 32, hi), torch.arange(hi, hi + 32),
                     torch.arange(n - 32, n)]).cuda()
    q = 1.5 + 0.1 * r(1, 1, N * G, d)                       # scores of 1.5 x 1 x 128 / sqrt(128) = 17
    keys, vals = 1.0 + 0.01 * r(128, d), 0.1 * r(128, d) + torch.where(torch.arange(128, **CUDA) < 64, 2.0, -1.0)[:, None]
    a["q"], keys, vals = q.half(), keys.half(), vals.half()
    a["k_cache"], a["v_cache"] = (torch.zeros((1, 1, n + 3, d), dtype=torch.float16, **CUDA) for _ in range(2))
    a["k_cache"][0, 0, far], a["v_cache"][0, 0, far] = keys, vals
    a["k_cache"][0, 0, n:], a["v_cache"][0, 0, n:] = math.nan, math.nan
    a["len"] = i32([n])
    out, status = call_attention(a)
    assert int(status.item()) == 0
    got = out.view(N, G, d).reshape(N * G, d).double()
    kb, vb = (a[k][0, 0].double() for k in ("k_blk", "v_blk"))
    qd, kd, vd = a["q"][0, 0].double(), keys.double(), vals.double()
    node = torch.arange(N * G, **CUDA) // G
    own = (qd * kb[node]).sum(1, keepdim=True) * d ** -0.5  # a node sees itself alone

    def result(rows):
        z = qd @ kd[rows].T * d ** -0.5
        m = torch.maximum(z.amax(1, keepdim=True), own)
        p, po = torch.exp(z - m), torch.exp(own - m)
        total = p.sum(1, keepdim=True) + po + (n - rows.numel()) * torch.exp(-m)
        return (p @ vd[rows] + po * vb[node]) / total, (p @ vd[rows].abs() + po * vb[node].abs()) / total

    ref, spread = result(torch.arange(128, **CUDA))
    mag = (qd.abs() @ kd.abs().T).amax() * d ** -0.5
    rel = 2 * ((d + 4) * 2.0 ** -24 * mag + 2.0 ** -21 + (n / 128 + 160) * 2.0 ** -24) + HALF_STEP[torch.float16]
    tol = rel * spread * 1.01 + HALF_STEP[torch.float16] * ref.abs() + 2.0 ** -24  # as in attention_bound
    assert ((got - ref).abs() <= tol).all(), float(((got - ref).abs() / tol).max())
    for part in (slice(0, 64), slice(64, 128)):  # what a kernel that misses either half would give
        keep = torch.ones(128, dtype=torch.bool, **CUDA)
        keep[part] = False
        assert ((result(keep.nonzero()[:, 0])[0] - ref).abs() > 10 * tol).all()


def test_attention_captured_and_on_two_streams():
    """A captured call replayed on new inputs; two calls at once on two streams, each with its scratch."""
    a, b = (make_attention(2, 2, 4, 33, 128, 1500, lens, seed=s) for lens, s in (([1400, 30], 17), ([0, 900], 18)))
    o = lib()
    ws = [torch.empty(o.tree_attention_workspace_bytes(2, 2, 4, 33, 128), dtype=torch.uint8, **CUDA) for _ in range(2)]
    outs = [torch.zeros((66, 1024), dtype=torch.float16, **CUDA) for _ in range(2)]
    refs = [call_attention(x)[0] for x in (a, b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        call_attention(a, workspace=ws[0], out=outs[0], stream=s1)
        call_attention(b, workspace=ws[1], out=outs[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], refs[0]) and torch.equal(outs[1], refs[1])
    status = torch.zeros(1, dtype=torch.int32, **CUDA)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.tree_attention(a["q"], a["k_cache"], a["v_cache"], a["k_blk"], a["v_blk"], a["len"], a["mask"], outs[0], ws[0],
                         status=status)
    for x in (b, a, b):  # the captured call reads its tensors anew
        for k in ("q", "k_cache", "v_cache", "k_blk", "v_blk", "len", "mask"):
            if x is not a:
                a_saved = {k2: a[k2].clone() for k2 in ("q", "k_cache", "v_cache", "k_blk", "v_blk", "len", "mask")}
                break
        if x is b:
            for k in a_saved:
                a[k].copy_(b[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], refs[1] if x is b else refs[0])
        if x is b:
            for k in a_saved:
                a[k].copy_(a_saved[k])
    assert int(status.item()) == 0


def test_attention_agrees_with_block_attention():
    """A chain (every node sees the ones before it) and a full mask are what orthrus_attention computes
    in verify and in draft mode."""
    o = lib()
    B, Hkv, G, N, d, cap = 2, 2, 4, 33, 128, 700
    for full in (False, True):
        see = np.ones((B, N, N), bool) if full else np.tile(np.tril(np.ones((N, N), bool)), (B, 1, 1))
        a = make_attention(B, Hkv, G, N, d, cap, [600, 77], seed=19, see=see)
        mine, _ = call_attention(a, planes=True)
        kc, vc = a["k_cache"].clone(), a["v_cache"].clone()
        for b in range(B):
            kc[b, :, a["lens"][b]:a["lens"][b] + N] = a["k_blk"][b]
            vc[b, :, a["lens"][b]:a["lens"][b] + N] = a["v_blk"][b]
        out = torch.zeros_like(mine)
        ws = torch.empty(o.attention_workspace_bytes(B, Hkv, G, N, d, cap), dtype=torch.uint8, **CUDA)
        status = torch.zeros(1, dtype=torch.int32, **CUDA)
        o.attention(a["q"], kc, vc, a["k_blk"], a["v_blk"], a["len"], B, Hkv, G, N, d, cap, N, 0 if full else 1, out, ws,
                    status)
        x, y = mine[0].double() + mine[1].double(), out[0].double() + out[1].double()
        assert float((x - y).norm() / y.norm()) <= 2 * 2.0 ** -11  # both round P to fp16


# ---- commit ---------------------------------------------------------------------------------------

def walk(parents, tokens, argmax, n):
    path = [0]
    while True:
        nxt = [j for j in range(path[-1] + 1, n) if parents[j] == path[-1] and tokens[j] == argmax[path[-1]]]
        if not nxt:
            return path
        path.append(nxt[0])


def make_commit(B, N, L, Hkv, d, cap, lens, seed, counts=None, vocab=3, t=torch.float16, blk_stride=None):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, **CUDA).to(t)  # noqa: E731
    return dict(parents=random_parents(B, N, seed), tokens=rng.integers(0, vocab, (B, N)).astype(np.int32),
                argmax=rng.integers(0, vocab, (B, N)).astype(np.int32), counts=counts, lens=list(lens),
                k_blk=r(L, B, Hkv, blk_stride or N, d), v_blk=r(L, B, Hkv, blk_stride or N, d), k_cache=r(L, B, Hkv, cap, d),
                v_cache=r(L, B, Hkv, cap, d))


def check_commit(c, in_place=False, status_in=0, want_status=0):
    o = lib()
    B, N = c["parents"].shape
    cap = c["k_cache"].shape[3]
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    z = lambda *s: torch.full(s, -9, dtype=torch.int32, **CUDA)  # noqa: E731
    length, pending, acc, path, com = i32(c["lens"]), z(B), z(B), z(B, N), z(B, N)
    new_len = length if in_place else z(B)
    status = i32([status_in])
    o.tree_commit(i32(c["parents"]), i32(c["tokens"]), i32(c["argmax"]), c["k_blk"], c["v_blk"], kc, vc, length, new_len,
                  pending, acc, path, com, n_nodes=None if c["counts"] is None else i32(c["counts"]), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == want_status
    want_k, want_v = c["k_cache"].clone(), c["v_cache"].clone()
    for b in range(B):
        n = N if c["counts"] is None else c["counts"][b]
        p = walk(c["parents"][b], c["tokens"][b], c["argmax"][b], n) if 0 < n <= N else []
        if status_in or not p or c["lens"][b] < 0 or c["lens"][b] + len(p) > cap:
            assert int(acc[b]) == -1 and int(new_len[b]) == c["lens"][b] and int(pending[b]) == -9
            assert (path[b] == -1).all() and (com[b] == -1).all()
            continue
        a, final = len(p) - 1, int(c["argmax"][b][p[-1]])
        assert int(acc[b]) == a and int(pending[b]) == final and int(new_len[b]) == c["lens"][b] + a + 1
        assert path[b].tolist() == p + [-1] * (N - a - 1)
        assert com[b].tolist() == [int(c["tokens"][b][j]) for j in p[1:]] + [final] + [-1] * (N - a - 1)
        for j, node in enumerate(p):
            want_k[:, b, :, c["lens"][b] + j] = c["k_blk"][:, b, :, node]
            want_v[:, b, :, c["lens"][b] + j] = c["v_blk"][:, b, :, node]
    assert torch.equal(kc.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))
    return acc


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,N,L,Hkv,d", [(1, 1, 1, 1, 64), (1, 33, 3, 2, 128), (3, 2, 2, 2, 8), (5, 64, 2, 4, 128),
                                         (2, 65, 1, 3, 72), (40, 17, 2, 1, 64), (2, 256, 2, 2, 128)])
def test_commit(B, N, L, Hkv, d, in_place):
    """Three tokens only, so that siblings repeat one another and long paths occur."""
    for vocab in (1, 2, 3):
        c = make_commit(B, N, L, Hkv, d, 600, [(7 * b) % 40 for b in range(B)], seed=N + vocab, vocab=vocab)
        acc = check_commit(c, in_place)
        if vocab == 1 and N > 2:
            assert int(acc.max()) > 0


def test_commit_ragged_idle_and_full():
    """Padded and idle trees; a path that just fits, and one that is one row too long."""
    c = make_commit(6, 20, 2, 2, 64, 64, [0, 10, 63, 64, 30, -1], seed=3, counts=[20, 1, 1, 1, 0, 9], vocab=2, blk_stride=31)
    # a missing row and a negative length occur in one call: whichever warp is first records its own
    check_commit(c, want_status=_Either(lib().ERR_CAPACITY, lib().ERR_ARG))
    chain = make_commit(2, 8, 1, 1, 64, 40, [32, 33], seed=4, vocab=1)
    chain["parents"][:] = np.arange(-1, 7)
    acc = check_commit(chain, want_status=lib().ERR_CAPACITY)
    assert acc.tolist() == [7, -1]


class _Either:
    def __init__(self, *codes):
        self.codes = codes

    def __eq__(self, other):
        return other in self.codes


def test_commit_after_an_error_changes_nothing():
    c = make_commit(3, 16, 2, 2, 64, 64, [0, 5, 9], seed=5, vocab=1)
    check_commit(c, status_in=lib().ERR_NAN, want_status=lib().ERR_NAN)


def test_commit_node_counts_out_of_range():
    c = make_commit(2, 8, 1, 1, 64, 64, [0, 5], seed=6, counts=[9, 8], vocab=1)
    check_commit(c, want_status=lib().ERR_ARG)


def test_commit_walk_ends_on_parents_that_are_no_tree():
    c = make_commit(1, 64, 1, 1, 64, 128, [3], seed=7, vocab=1)
    c["parents"][:] = np.random.default_rng(8).integers(-5, 70, (1, 64))
    check_commit(c)


def test_commit_bf16_cache():
    check_commit(make_commit(2, 33, 2, 2, 128, 128, [3, 50], seed=9, vocab=2, t=torch.bfloat16))


# ---- together ---------------------------------------------------------------------------------------

def test_operators_one_after_another():
    """One layer's tree step from the single operators: projection, layout, rotary positions into the q layout
    and the scratch block, tree attention; then the commit, and the next step's attention over the grown cache."""
    o = lib()
    B, N, Hkv, G, d, D, cap, n0 = 2, 21, 2, 4, 64, 256, 128, [50, 17]
    H, dev = Hkv * G, dict(device="cuda")
    g = torch.Generator(device="cuda").manual_seed(21)
    W = (torch.randn((H + 2 * Hkv) * d, D, generator=g, **dev) * 0.05).bfloat16()
    kc, vc = (torch.randn(1, B, Hkv, cap, d, generator=g, **dev).bfloat16().half() for _ in range(2))
    kb, vb = (torch.zeros(1, B, Hkv, N, d, dtype=torch.float16, **dev) for _ in range(2))
    length, rope = i32(n0), o.rope(d, theta=1.0e4)
    status, words = torch.zeros(1, dtype=torch.int32, **dev), (N + 63) // 64
    ws = torch.empty(o.tree_attention_workspace_bytes(B, Hkv, G, N, d), dtype=torch.uint8, **dev)
    gemm_ws = torch.empty(o.linear_workspace_bytes(B * N, W.shape[0], D), dtype=torch.uint8, **dev)
    lens = list(n0)
    for step in range(2):
        X = torch.randn(B * N, D, generator=g, **dev).bfloat16()
        parents = random_parents(B, N, 30 + step)
        depth = torch.zeros((B, N), dtype=torch.int32, **dev)
        mask = torch.zeros((B, N, words), dtype=torch.int64, **dev)
        Y = torch.empty(B * N, W.shape[0], dtype=torch.float32, **dev)
        q = torch.empty(B, Hkv, N * G, d, dtype=torch.float16, **dev)
        out = torch.empty(2, B * N, H * d, dtype=torch.bfloat16, **dev)
        o.tree_layout(i32(parents), depth, mask, status=status)
        o.linear(X, W, Y, gemm_ws, status)
        heads = Y.view(B, N, H + 2 * Hkv, d)
        o.rotary(rope, [(heads[:, :, :H], q.view(B, Hkv, N, G, d).permute(0, 2, 1, 3, 4)),
                        (heads[:, :, H:H + Hkv], kb[0].transpose(1, 2), o.ROTARY_BF16_VALUES),
                        (heads[:, :, H + Hkv:], vb[0].transpose(1, 2), o.ROTARY_BF16_VALUES | o.ROTARY_COPY)],
                 len=length, offsets=depth, status=status)
        o.tree_attention(q, kc[0], vc[0], kb[0], vb[0], length, mask, out, ws, status=status)
        # the same in float64
        see = visibility(parents)
        pos = torch.tensor(lens, **dev)[:, None] + torch.from_numpy(see.sum(2) - 1).cuda()
        y = (X.double() @ W.double().T).view(B, N, H + 2 * Hkv, d)
        from oracle.model import rope as turned
        for b in range(B):
            qk = turned(y[b, :, :H + Hkv].cpu(), pos[b].cpu(), 1.0e4).cuda()
            keys = torch.cat([kc[0, b, :, :lens[b]].double(), qk[:, H:].transpose(0, 1)], 1)
            vals = torch.cat([vc[0, b, :, :lens[b]].double(), y[b, :, H + Hkv:].transpose(0, 1)], 1)
            seen = torch.cat([torch.ones((N, lens[b]), dtype=torch.bool), torch.from_numpy(see[b])], 1).cuda()
            got = (out[0].double() + out[1].double()).view(B, N, Hkv, G, d)[b]
            for h in range(Hkv):
                z = torch.einsum("ngd,kd->ngk", qk[:, h * G:(h + 1) * G], keys[h]) * d ** -0.5
                p = torch.softmax(z.masked_fill(~seen[:, None], -math.inf), -1)
                ref = torch.einsum("ngk,kd->ngd", p, vals[h])
                # K and V of the block are rounded to bf16 (half a step 2^-8), q and P to fp16
                assert float((got[:, h] - ref).norm() / ref.norm()) <= 2 * 2.0 ** -8 + 2 * 2.0 ** -11
        tokens = np.random.default_rng(40 + step).integers(0, 2, (B, N)).astype(np.int32)
        argmax = np.random.default_rng(50 + step).integers(0, 2, (B, N)).astype(np.int32)
        z = lambda *s: torch.zeros(s, dtype=torch.int32, **dev)  # noqa: E731
        pending, acc, path, com = z(B), z(B), z(B, N), z(B, N)
        o.tree_commit(i32(parents), i32(tokens), i32(argmax), kb, vb, kc, vc, length, length, pending, acc, path, com,
                      status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for b in range(B):
            p = walk(parents[b], tokens[b], argmax[b], N)
            for j, node in enumerate(p):
                assert torch.equal(kc[0, b, :, lens[b] + j], kb[0, b, :, node])
                assert torch.equal(vc[0, b, :, lens[b] + j], vb[0, b, :, node])
            lens[b] += len(p)
        assert length.tolist() == lens


# ---- with a plan ------------------------------------------------------------------------------------

MARGIN, LOGITS = 0.1, 5e-2


@pytest.mark.parametrize("shape", [synth.TINY, synth.TINY_QK], ids=["tiny", "tiny_qk"])
def test_plan_tree_step_matches_oracle(shape):
    """Two sequences, trees of different sizes. Every node's logits equal the oracle's verify view of the
    tokens on its path; the committed stream continues as greedy decoding does."""
    o = lib()
    B, K, N, cap = 2, 16, 14, 96
    w = synth.make_weights(shape, 61, 62, gain_std=0.1 if shape.qk_norm else 0.0)
    dev = o.DeviceModel(shape, w, batch=B, capacity=cap, max_block=K, max_rows=64)
    ref = Oracle(shape, w, capacity=cap)
    plens = [11, 24]
    prompts = [synth.make_prompt(shape, p, 63 + b) for b, p in enumerate(plens)]
    toks = np.zeros((B, max(plens)), np.int32)
    for b in range(B):
        toks[b, :plens[b]] = prompts[b]
    pending = torch.zeros(B, dtype=torch.int32, **CUDA)
    dev.prefill(torch.from_numpy(toks).cuda(), plens, pending)
    states = []
    for b in range(B):
        st = ref.new_state()
        ref.prefill(st, prompts[b])
        st.y = int(pending[b])
        st.out = [st.y]
        states.append(st)
    counts, rng = [N, 9], np.random.default_rng(64)
    accepted = 0
    for step in range(4):
        parents, tokens = random_parents(B, N, 70 + step, spread=4), rng.integers(0, shape.vocab, (B, N)).astype(np.int32)
        for b in range(B):  # plant the oracle's greedy continuation on a path of the tree
            import copy
            s2, node = copy.deepcopy(states[b]), 0
            for i in range(1, counts[b]):
                if parents[b, i] == node and rng.random() < 0.8:
                    tokens[b, i] = ref.ar_step(s2)
                    node = i
        argmax = torch.full((B, N), -5, dtype=torch.int32, **CUDA)
        logits = torch.zeros((B, N, shape.vocab), dtype=torch.float32, **CUDA)
        z = lambda *s: torch.zeros(s, dtype=torch.int32, **CUDA)  # noqa: E731
        acc, path, com = z(B), z(B, N), z(B, N)
        before = dev.lens.tolist()
        dev.verify_tree(pending, i32(tokens), i32(parents), argmax, n_nodes=i32(counts), logits=logits)
        torch.cuda.synchronize()
        assert dev.read_status() == 0 and dev.lens.tolist() == before
        got = argmax.cpu().numpy()
        for b in range(B):
            for i in range(counts[b]):
                chain, j = [], i
                while j > 0:
                    chain.append(int(tokens[b, j]))
                    j = parents[b, j]
                import copy
                _, lg = ref.verify_block(copy.deepcopy(states[b]), chain[::-1])
                row = lg[-1]
                assert float((logits[b, i].cpu().double() - row).abs().max()) <= LOGITS, (step, b, i)
                best = int(torch.argmax(row))
                if top2_margin(row) > MARGIN:
                    assert int(got[b, i]) == best
                else:
                    assert float(row[int(got[b, i])]) >= float(row[best]) - MARGIN
        dev.accept_commit_tree(pending, i32(tokens), i32(parents), argmax, acc, path, com, n_nodes=i32(counts))
        torch.cuda.synchronize()
        assert dev.read_status() == 0
        for b in range(B):
            p = walk(parents[b], tokens[b], got[b], counts[b])
            drafts = [int(tokens[b, j]) for j in p[1:]]
            a = len(drafts)
            accepted += a
            assert int(acc[b]) == a and path[b].tolist()[:a + 1] == p
            assert com[b].tolist() == drafts + [int(got[b, p[-1]])] + [-1] * (N - a - 1)
            ref.verify_block(states[b], drafts)
            ref.accept_commit(states[b], drafts, [int(got[b, j]) for j in p])
            assert int(pending[b]) == states[b].y and int(dev.lens[b]) == states[b].n
            for l in range(shape.n_layers):  # the cache rows of the path are those of decoding its tokens in a chain
                for mine, want in ((dev.k_cache, states[b].k), (dev.v_cache, states[b].v)):
                    x = mine[l, b, :, before[b]:states[b].n].double().cpu()
                    y = want[l][:, before[b]:states[b].n].double()
                    assert float((x - y).abs().max()) <= 2.0 ** -7 * max(1.0, float(y.abs().max()))
    assert accepted >= 4


def test_plan_tree_chain_and_block_agree():
    """A tree that is a chain is the verify block: the same argmaxes and commit, then decoding goes on
    with the chain's calls."""
    o, shape = lib(), synth.TINY_QK
    K, P, cap = 8, 20, 80
    w = synth.make_weights(shape, 71, 72, gain_std=0.1)
    prompt = synth.make_prompt(shape, P, 73)
    stream = greedy_ar(Oracle(shape, w, capacity=cap), prompt, 40)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, **CUDA)  # noqa: E731
    results = []
    for tree in (False, True):
        dev = o.DeviceModel(shape, w, batch=1, capacity=cap, max_block=K + 1, max_rows=64)
        pending, ar, acc, com = z(1), z(1, K + 1), z(1), z(1, K + 1)
        dev.prefill(torch.from_numpy(prompt).view(1, P).cuda(), [P], pending)
        drafts = np.array(stream[1:K + 1], np.int32)
        drafts[4] = (drafts[4] + 1) % shape.vocab
        logits = torch.zeros((1, K + 1, shape.vocab), **CUDA)
        if tree:
            tokens = i32([[0] + drafts.tolist()])
            parents, path = i32([list(range(-1, K))]), z(1, K + 1)
            dev.verify_tree(pending, tokens, parents, ar, logits=logits)
            dev.accept_commit_tree(pending, tokens, parents, ar, acc, path, com)
        else:
            dev.verify_block(pending, i32([drafts.tolist()]), K, ar, logits)
            dev.accept_commit(pending, i32([drafts.tolist()]), ar, K, acc, com)
        first = (ar.tolist(), acc.tolist(), com.tolist(), dev.lens.tolist(), pending.tolist())
        dev.decode_step(pending, K, None, acc, com)
        torch.cuda.synchronize()
        assert dev.read_status() == 0
        results.append((first, com[0, :int(acc) + 1].tolist(), logits))
    assert results[0][0] == results[1][0] and results[0][0][1] == [4]
    assert float((results[0][2] - results[1][2]).abs().max()) <= 2 * LOGITS


WIDE = synth.ModelShape("wide_heads", 2, 512, 8, 2, 128, 768, 1024, qk_norm=True)


@pytest.mark.parametrize("shape", [synth.TINY_QK, WIDE], ids=["d64", "d128"])
@pytest.mark.parametrize("P", [3, 200])
@pytest.mark.parametrize("N", [1, 16, 33, 47, 64])
def test_plan_tree_in_one_launch_and_in_many(N, P, shape):
    """Few rows run through the persistent kernel, more than 128 through the kernels of each step: the same tree
    in a batch of one and in a batch of many, with two roots and padding, gives the same logits up to rounding."""
    o, cap = lib(), 320
    w = synth.make_weights(shape, 91, 92, gain_std=0.1)
    prompt = synth.make_prompt(shape, P, 93)
    parents, rng = random_parents(1, N, 94 + N, spread=12), np.random.default_rng(95)
    if N > 12:
        parents[0, 12] = -1
    tokens, live = rng.integers(0, shape.vocab, (1, N)).astype(np.int32), max(1, N - 3)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, **CUDA)  # noqa: E731
    got = []
    for B in (1, 128 // N + 1):
        dev = o.DeviceModel(shape, w, batch=B, capacity=cap, max_block=N, max_rows=max(256, B * (N + 1)))
        pending, ar = z(B), z(B, N)
        dev.prefill(torch.from_numpy(np.tile(prompt, (B, 1))).cuda(), [P] * B, pending)
        logits = torch.zeros((B, N, shape.vocab), **CUDA)
        dev.verify_tree(pending, i32(np.tile(tokens, (B, 1))), i32(np.tile(parents, (B, 1))), ar, n_nodes=i32([live] * B),
                        logits=logits)
        torch.cuda.synchronize()
        assert dev.read_status() == 0 and dev.lens.tolist() == [P] * B
        assert torch.equal(ar[:, :live].long(), logits[:, :live].argmax(-1))
        assert float((logits[:, :live] - logits[:1, :live]).abs().max()) <= 2 * LOGITS
        got.append((logits[0, :live].clone(), dev))
    assert float((got[0][0] - got[1][0]).abs().max()) <= 2 * LOGITS


def test_plan_tree_refusals():
    o, shape = lib(), synth.TINY
    w = synth.make_weights(shape, 81, 82)
    dev = o.DeviceModel(shape, w, batch=1, capacity=64, max_block=4)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, **CUDA)  # noqa: E731
    pending, tokens, parents = z(1), z(1, 5), i32([[-1, 0, 0, 1, 2]])
    with pytest.raises(o.OrthrusError):  # more nodes than the plan's block limit
        dev.verify_tree(pending, tokens, parents, z(1, 5))
    with pytest.raises(o.OrthrusError):
        dev.accept_commit_tree(pending, tokens, parents, z(1, 5), z(1), z(1, 5), z(1, 5))
    # a token outside the vocabulary and a parent that is none set the status, and nothing is committed
    dev.prefill(z(1, 6), [6], pending)
    for bad_tokens, bad_parents in (([0, shape.vocab, 1, 2], [-1, 0, 0, 1]), ([0, 1, 1, 2], [-1, 0, 3, 1])):
        dev.clear_status()
        ar, acc, path, com = z(1, 4), z(1), z(1, 4), z(1, 4)
        dev.verify_tree(pending, i32([bad_tokens]), i32([bad_parents]), ar)
        dev.accept_commit_tree(pending, i32([bad_tokens]), i32([bad_parents]), ar, acc, path, com)
        torch.cuda.synchronize()
        assert dev.read_status() == o.ERR_ARG
        assert acc.tolist() == [-1] and dev.lens.tolist() == [6]


def test_plan_goes_on_after_an_error():
    """A tree whose parents are none stops the forward on its way; once the status is cleared, trees and
    chains give the bits that they give without it."""
    o, shape, N, P = lib(), synth.TINY_QK, 9, 40
    w = synth.make_weights(shape, 96, 97, gain_std=0.1)
    prompt = torch.from_numpy(synth.make_prompt(shape, P, 98)).view(1, P).cuda()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, **CUDA)  # noqa: E731
    tokens, parents = i32(np.arange(5, 5 + N)[None]), i32(random_parents(1, N, 99))
    results = []
    for bad in (0, 1, 5):
        dev = o.DeviceModel(shape, w, batch=1, capacity=96, max_block=N, max_rows=64)
        pending, ar, chain = z(1), z(1, N), z(1, N)
        dev.prefill(prompt, [P], pending)
        for _ in range(bad):
            dev.verify_tree(pending, tokens, i32([[-1] + [7] * (N - 1)]), ar)
            torch.cuda.synchronize()
            assert dev.read_status() == o.ERR_ARG
            dev.clear_status()
        logits, more = torch.zeros((1, N, shape.vocab), **CUDA), torch.zeros((1, N, shape.vocab), **CUDA)
        dev.verify_tree(pending, tokens, parents, ar, logits=logits)
        dev.verify_block(pending, tokens[:, 1:].contiguous(), N - 1, chain, more)
        torch.cuda.synchronize()
        assert dev.read_status() == 0
        results.append((logits, more))
    for logits, more in results[1:]:
        assert torch.equal(logits, results[0][0]) and torch.equal(more, results[0][1])


def test_binding_refuses_what_does_not_fit():
    o = lib()
    a = make_attention(1, 2, 4, 9, 64, 128, [20], seed=1)
    out, ws = torch.zeros((9, 512), dtype=torch.float16, **CUDA), torch.zeros(1 << 20, dtype=torch.uint8, **CUDA)

    def call(**kw):
        x = {**a, "out": out, "ws": torch.zeros(64 << 20, dtype=torch.uint8, **CUDA), **kw}
        o.tree_attention(x["q"], x["k_cache"], x["v_cache"], x["k_blk"], x["v_blk"], x["len"], x["mask"], x["out"], x["ws"])

    call()
    for kw in (dict(q=a["q"].float()), dict(k_cache=a["k_cache"].bfloat16()), dict(v_cache=a["v_cache"][:, :, :100].contiguous()),
               dict(k_cache=a["k_cache"].transpose(1, 2)), dict(k_blk=a["k_blk"][:, :, :8].contiguous()), dict(len=a["len"].long()),
               dict(len=a["len"].cpu()), dict(mask=a["mask"].int()), dict(mask=a["mask"][:, :8].contiguous()),
               dict(out=out[:8]), dict(out=out.float()), dict(out=torch.zeros((2, 9, 512), dtype=torch.float16, **CUDA))):
        with pytest.raises(ValueError):
            call(**kw)
    if o.tree_attention_workspace_bytes(1, 2, 4, 9, 64) > 256:
        with pytest.raises(o.OrthrusError) as e:
            call(ws=ws[:256])
        assert e.value.code == o.ERR_WORKSPACE
