"""ar_cache_attention on the GPU against the definition in binary64.

Bound.  A score is a sum of D products (those of a step in a tensor core may lose what
lies below 4 units of 2^-24 of the step's magnitudes; D / 16 + 4 such steps, or D + 8
single additions: (D + 32) u of scale * sum |q||k| covers both), is scaled by at most four
more products, and enters the exponential with its own size: a weight is off by
  e = (D + 40) u S + 8 u,   S = the largest scale * sum |q||k| of the row.
(The binary16 form of q keeps 11 bits of numbers of at most 11 bits.)  With keys and values
of one or two bytes a weight is held with 16 bits more: 2^-16.  Sums over j are chains of at
most n / 16 + 128 additions.  Numerator and denominator carry these alike:
  |out - want| <= 2 (e + chain) sum p|v| + half a unit of the output.
Below 2^-126 a rounding is no longer relative: a value code * scale and its product with a
weight are each off by up to 2^-150 (their sums, multiples of 2^-149 there, are exact), and
so are a row's sum at each of its n / 16 rescalings and the quotient:
  (1 + n + n / 16 + 1) 2^-150 <= (2 n + 2) 2^-150 more."""
import math

import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from cache_helpers import Cache
from gpu_helpers import need_gpu
from layer_helpers import TORCH, U, assert_within, f64, half, placed, randn, untouched

pytestmark = pytest.mark.gpu


def _work(D):
    return torch.full((ar.AR_CACHE_WORK_ROWS * (D + 2),), float("nan"), device="cuda")


def _exact(c, q, scale, window):
    """out, lse, bounds (without the output's rounding) in binary64."""
    B, heads, D = q.shape
    group = heads // c.heads
    K, V = c.values(0), c.values(1)
    out, err = np.zeros((B, heads, D)), np.zeros((B, heads, D))
    lse, lerr = np.full((B, heads), -np.inf), np.zeros((B, heads))
    for b in range(B):
        n = min(max(c.lens_host[b], 0), c.width * c.page)
        pages, slots = c.places(b, n - window if window else 0, n)
        on = pages >= 0
        if not on.any():
            continue
        k, v = K[pages[on], :, slots[on]], V[pages[on], :, slots[on]]       # n, kv, D
        for h in range(heads):
            kh, vh = k[:, h // group], v[:, h // group]
            s = scale * (kh @ q[b, h])
            size = (abs(scale) * (np.abs(kh) @ np.abs(q[b, h]))).max()
            p = np.exp(s - s.max())
            total = p.sum()
            p /= total
            out[b, h] = p @ vh
            lse[b, h] = s.max() + math.log(total)
            e = (D + 40) * U * size + 8 * U + (len(p) / 16 + 128) * U
            lerr[b, h] = e + 8 * U * (abs(lse[b, h]) + 1)
            if c.dtype != "fp32" or c.eight:
                e += 2.0 ** -16
            err[b, h] = 2 * e * (p @ np.abs(vh)) + (2 * len(p) + 2) * 2.0 ** -150
    return out, lse, err, lerr


def _check(lens, heads, kv, D, page, dtype, cache, window=0, scale=None, qpad=0, shift=0, q_std=1.0,
           spoil=None, with_lse=True, **kw):
    need_gpu()
    c = Cache(lens, kv, D, page, dtype, cache, **kw)
    if spoil is not None:
        spoil(c)
    scale = D ** -0.5 if scale is None else scale
    cols = heads * D
    q, _ = placed((q_std * randn(7, c.B, cols)).to(TORCH[dtype]).cuda(), qpad, shift)
    out, buf = placed(torch.full((c.B, cols), float("nan"), device="cuda").to(TORCH[dtype]), qpad,
                      shift)
    lse = torch.full((c.B, heads), float("nan"), device="cuda") if with_lse else None
    work = _work(D)
    ar.ar_cache_attention(q, *c.args(), scale, out, lse, work, 4 * work.numel(), c.B, heads, kv, D,
                          dtype, cache, window=window, ldq=cols + qpad, ldout=cols + qpad,
                          **c.strides())
    torch.cuda.synchronize()
    want, wlse, err, lerr = _exact(c, f64(q).reshape(c.B, heads, D), np.float32(scale), window)

    def compare(what):
        assert untouched(buf, c.B, cols, qpad, shift)
        assert_within(f64(out).reshape(want.shape), want, err + half(want, dtype) * (1 + 1e-6),
                      what)
        if with_lse:
            got = lse.double().cpu().numpy()
            empty = np.isinf(wlse)
            assert (got[empty] == -np.inf).all()
            assert_within(got[~empty], wlse[~empty], lerr[~empty], what + ", lse")
    compare("out")
    # a table with room for far more, of which the lengths use as much: how units are shared
    # out goes by what the host knows, the table's width; the result holds either way.  (A
    # length past the table means another one then.)
    if all(n <= c.width * c.page for n in c.lens_host):
        first = out.clone()
        width = c.width + 20000 // c.page + 1
        table = torch.full((c.B, width), -1, dtype=torch.int32, device="cuda")
        table[:, :c.width] = c.table[:, :c.width]
        args = list(c.args())
        args[6], args[7] = table, width
        out.fill_(float("nan"))
        ar.ar_cache_attention(q, *args, scale, out, lse, work, 4 * work.numel(), c.B, heads, kv, D,
                              dtype, cache, window=window, ldq=cols + qpad, ldout=cols + qpad,
                              ldpage=c.ldpage)
        torch.cuda.synchronize()
        compare("out, wide table")
        return c, first
    return c, out


KINDS = [("bf16", "bf16"), ("bf16", "e4m3"), ("fp16", "fp16"), ("fp16", "e4m3"), ("fp32", "fp32"),
         ("fp32", "e4m3")]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 1000, 3001])
def test_lengths(dtype, cache, n):
    _check([n], 8, 1, 128, 16, dtype, cache, seed=n)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [1, 3, 8, 16, 24, 40, 64, 72, 80, 96, 100, 112, 128, 136, 160, 192,
                               250, 256])
def test_head_sizes(dtype, cache, D):
    _check([70, 9, 300], 6, 2, D, 16, dtype, cache, seed=D)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 1), (7, 1), (8, 8), (9, 1), (16, 1), (17, 1),
                                      (32, 2), (33, 1), (64, 1), (40, 8), (48, 24), (128, 4)])
def test_head_layouts(dtype, cache, heads, kv):
    _check([5, 130, 77], heads, kv, 64, 32, dtype, cache, seed=heads)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("page", [1, 2, 3, 16, 17, 50, 64, 100, 128])
def test_pages(dtype, cache, page):
    """Pages that end inside a tile, and tiles inside a page."""
    _check([333, 1, 64], 8, 2, 128, page, dtype, cache, seed=page, extra_columns=page % 3)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 500, 10 ** 6])
def test_windows(dtype, cache, window):
    _check([1, 64, 500, 129, 0], 4, 2, 64, 16, dtype, cache, window=window, seed=window % 97)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0, 5, 0, 0, 1, 0], [1] * 40, [-3, 4],
                                  [2000] + [3] * 20, [1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144, 233],
                                  [64] * 300], ids=lambda x: "%dx%d" % (len(x), max(x)))
def test_batches(dtype, cache, lens):
    """Empty and idle sequences, one token, uneven ones, more units than CTAs."""
    _check(lens, 8, 2, 64, 16, dtype, cache, seed=len(lens))


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
@pytest.mark.parametrize("heads,kv,D", [(8, 1, 128), (16, 1, 256), (4, 4, 64), (24, 1, 96)])
def test_long_sequences_are_split(dtype, cache, heads, kv, D):
    _check([20000], heads, kv, D, 64, dtype, cache, seed=D)
    _check([9000, 1, 4000, 0, 12345], heads, kv, D, 64, dtype, cache, seed=D, window=8000)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("qpad,shift,gap,both", [
    (0, 0, 0, True), (8, 0, 64, False), (3, 0, 0, False), (0, 1, 0, False), (0, 0, 1, False),
    (5, 3, 8, True), (0, 0, 3, True)])
def test_strides_and_alignment(dtype, cache, qpad, shift, gap, both):
    _check([70, 200], 4, 2, 64, 16, dtype, cache, qpad=qpad, shift=shift, gap=gap, both=both,
           extra_columns=2, with_lse=shift == 0)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_sharp_and_large_scores(dtype, cache):
    """One position takes all of the weight, scores in the hundreds, either sign of scale."""
    _check([300, 40], 4, 2, 64, 16, dtype, cache, q_std=30.0)
    _check([300, 40], 4, 2, 64, 16, dtype, cache, scale=-1.5)
    _check([300, 40], 4, 2, 64, 16, dtype, cache, scale=0.0)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_positions_outside_the_pool(dtype, cache):
    """Pages that are not there, among them all of a sequence's; lengths past the table."""
    def spoil(c):
        c.table[0, 1], c.table[0, 3] = -1, c.pages
        c.table[1] = -2 ** 31
        c.table[2, 0] = 2 ** 31 - 1
        c.lens_host[2] = 2 ** 31 - 1
        c.lens.copy_(torch.tensor(c.lens_host, dtype=torch.int32))
    _check([70, 33, 80], 4, 2, 64, 16, dtype, cache, spoil=spoil)
    _check([70, 33, 80], 4, 2, 64, 16, dtype, cache, spoil=spoil, window=20)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_what_lies_behind_the_length_is_not_seen(dtype, cache):
    """NaN and infinities in every slot but the sequences' own, and in unused scales."""
    need_gpu()
    lens = [37, 1, 64, 90]
    clean = _check(lens, 8, 2, 128, 16, dtype, cache, window=30)[1]

    def spoil(c):
        own = [torch.zeros(c.pages, c.page, dtype=torch.bool, device="cuda") for _ in "kv"]
        for b, n in enumerate(lens):
            p, s = c.places(b, max(0, n - 30), n)
            for o in own:
                o[torch.tensor(p).cuda(), torch.tensor(s).cuda()] = True
        for pool, scale, o in zip(c.pools, c.scales, own):
            mask = ~o[:, None, :, None].expand(pool.shape)
            pool[mask] = 0x7F if c.eight else float("nan")
            if c.eight:
                scale[~o[:, None].expand(scale.shape)] = float("inf")

    out = []

    def keep(c):
        spoil(c)
        c.values = lambda which, f=c.values: np.nan_to_num(f(which), nan=0, posinf=0, neginf=0)
    out = _check(lens, 8, 2, 128, 16, dtype, cache, window=30, spoil=keep)[1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_nan_and_infinities_of_a_sequence_stay_in_it(dtype, cache):
    need_gpu()
    lens = [100, 100, 100, 100]
    clean = _check(lens, 4, 2, 64, 16, dtype, cache)[1]
    c = Cache(lens, 2, 64, 16, dtype, cache)
    bad = 0x7F if c.eight else float("nan")
    p, s = c.places(1, 70, 71)
    c.pools[0][int(p[0]), 0, int(s[0]), 3] = bad             # a key of sequence 1, head 0
    p, s = c.places(2, 5, 6)
    c.pools[1][int(p[0]), 1, int(s[0]), 9] = bad             # a value of sequence 2, head 1
    q = randn(7, 4, 256).to(TORCH[dtype]).cuda()
    q[3, 64:128] = float("inf")
    out, lse, work = torch.zeros_like(q), torch.zeros(4, 4, device="cuda"), _work(64)
    ar.ar_cache_attention(q, *c.args(), 0.125, out, lse, work, 4 * work.numel(), 4, 4, 2, 64, dtype,
                          cache, **c.strides())
    bad = torch.zeros(4, 4, 64, dtype=torch.bool, device="cuda")
    bad[1, :2] = True
    bad[2, 2:, 9] = True
    bad[3, 1] = True
    out = out.view(4, 4, 64)
    assert bool(torch.isnan(out[bad]).all())
    assert torch.equal(out[~bad], clean.view(4, 4, 64)[~bad])


def test_scores_of_minus_infinity_alone():
    """No weight at all: zeros and -inf, as for no position; beside others they weigh nothing."""
    need_gpu()
    for dtype in ("bf16", "fp32"):
        c = Cache([70, 70], 1, 64, 16, dtype, dtype)
        c.pools[0].zero_()
        c.pools[0][..., 0] = float("-inf")
        p, s = c.places(1, 66, 67)
        c.pools[0][int(p[0]), 0, int(s[0]), 0] = 1.0
        q = torch.zeros(2, 64, dtype=TORCH[dtype], device="cuda")
        q[:, 0] = 1.0
        # 0 * -inf of the other elements of q is NaN: they have no part in the keys
        c.pools[0][..., 1:] = 0
        out, lse, work = torch.ones_like(q), torch.ones(2, 1, device="cuda"), _work(64)
        ar.ar_cache_attention(q, *c.args(), 1.0, out, lse, work, 4 * work.numel(), 2, 1, 1, 64,
                              dtype, dtype, **c.strides())
        assert bool((out[0] == 0).all()) and float(lse[0]) == -math.inf
        assert torch.equal(out[1], c.pools[1][int(p[0]), 0, int(s[0])]) and float(lse[1]) == 1.0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ks,vs", [(1e-30, 1e-30), (1e-3, 1e30), (1e-38, 1e-33), (1.0, 3e35),
                                   (0.0, 1.0), (1e-3, 0.0)])
def test_scales_of_any_size(dtype, ks, vs):
    """Values whose scales are far from one another by many powers of two."""
    def spoil(c):
        c.scales[0].mul_(ks / 0.01)
        if ks == 0.0:
            c.scales[0].zero_()
        c.scales[1].mul_(vs / 0.01)
        c.scales[1][1::2] *= 2.0 ** -40
    if dtype != "fp32" and vs > 1e10 and dtype == "fp16":
        pytest.skip("beyond binary16")
    _check([200, 31], 4, 1, 64, 16, dtype, "e4m3", spoil=spoil)


def test_same_bits_every_time_and_in_a_graph():
    """The parts of a split depend on nothing that varies; one capture serves any lengths."""
    need_gpu()
    lens = [5000, 1, 0, 777]
    c = Cache(lens, 2, 128, 64, "bf16", "e4m3")
    q = randn(1, 4, 16 * 128).bfloat16().cuda()
    work = _work(128)

    def call(out, lse, stream=None):
        ar.ar_cache_attention(q, *c.args(), 0.1, out, lse, work, 4 * work.numel(), 4, 16, 2, 128,
                              "bf16", "e4m3", stream=stream, **c.strides())
    out, lse = torch.empty_like(q), torch.empty(4, 16, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(out, lse, s)
    for now in ([5000, 1, 0, 777], [4999, 0, 0, 1], [0, 0, 0, 0], [3, 1, 0, 2]):
        c.lens.copy_(torch.tensor(now, dtype=torch.int32))
        first, first_lse = torch.full_like(q, 7), torch.full_like(lse, 7)
        call(first, first_lse)
        for _ in range(5):
            out.fill_(9)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first) and torch.equal(lse, first_lse)


def test_two_calls_at_once_with_a_workspace_each():
    need_gpu()
    sets = []
    for i in range(2):
        c = Cache([3000 + i, 200], 2, 128, 64, "bf16", "bf16", seed=i)
        q = randn(i, 2, 1024).bfloat16().cuda()
        sets.append((c, q, torch.empty_like(q), _work(128), torch.cuda.Stream()))

    def call(c, q, out, work, s):
        ar.ar_cache_attention(q, *c.args(), 0.1, out, None, work, 4 * work.numel(), 2, 8, 2, 128,
                              "bf16", stream=s, **c.strides())
    want = []
    for x in sets:
        call(*x[:4], None)
        want.append(x[2].clone())
    torch.cuda.synchronize()
    for _ in range(20):
        for x in sets:
            call(*x)
    torch.cuda.synchronize()
    for x, w in zip(sets, want):
        assert torch.equal(x[2], w)


def test_zero_sequences():
    ar.ar_cache_attention(None, None, None, None, None, 0, 16, None, 1, None, 1.0, None, None, None,
                          0, 0, 8, 2, 64, "bf16", stream=0)
