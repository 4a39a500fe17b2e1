"""Attention over packed sequences against FP64 within derived bounds
(attn_harness.py): lengths, head layouts, masks, strides, paths."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import attn_harness as ah  # noqa: E402


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 300])
def test_one_sequence(tg, n, dim, dtype):
    ah.check_forward(tg, ah.Problem([n], heads=2, kv=1, dim=dim, dtype=dtype, causal=n % 2 == 1))


@pytest.mark.parametrize("dim", [8, 16, 40, 72, 80, 96, 120])
def test_head_sizes_between_tiles(tg, dim):
    ah.check_forward(tg, ah.Problem([130, 7], heads=4, kv=2, dim=dim, dtype="fp16"))


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (5, 1), (7, 7), (12, 4), (40, 2), (128, 1), (96, 2)])
def test_groups_of_heads(tg, heads, kv):
    ah.check_forward(tg, ah.Problem([70, 3], heads=heads, kv=kv, dim=64))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,k_len", [
    ([5, 0, 300, 1, 64], None),
    ([5, 0, 300, 1, 64], [9, 17, 411, 0, 64]),
    ([200, 130], [100, 3]),            # causal: rows without keys
    ([0, 0], [5, 0]),
    ([1, 1, 1], [700, 1, 129]),
    ([4, 4], [1000, 30]),
])
def test_packed_lengths(tg, q_len, k_len, causal):
    ah.check_forward(tg, ah.Problem(q_len, k_len, heads=4, kv=2, dim=64, causal=causal))


def test_many_tiles_two_a_cta(tg):
    """More row tiles than SMs: two a CTA, with odd counts and ragged ends."""
    ah.check_forward(tg, ah.Problem([700, 129, 385, 1, 0, 1000], heads=16, kv=16, dim=64, dtype="fp16"))
    ah.check_forward(tg, ah.Problem([1111, 260], heads=16, kv=8, dim=128))
    ah.check_forward(tg, ah.Problem([900, 513], [300, 1200], heads=16, kv=16, dim=128))
    ah.check_forward(tg, ah.Problem([640, 300], [257, 64], heads=24, kv=12, dim=96, causal=False))


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
def test_single_tokens_over_a_cache(tg, dim, dtype):
    """Slabs of 5000 rows, filled unevenly; long ones are cut into key ranges."""
    k = [5000, 1, 0, 4097, 640, 129]
    at = [5000 * i for i in range(6)]
    p = ah.Problem([1] * 6, k, heads=8, kv=2, dim=dim, dtype=dtype, k_at=at, k_rows=30000,
                   q_at=list(range(6)))
    assert tg.tg_attention_workspace_bytes(*p.sizes(), p.max_q, p.max_k, dtype) > 0
    ah.check_forward(tg, p)


@pytest.mark.parametrize("shape", [dict(pad=8), dict(gap=8), dict(pad=24, gap=16), dict(heads_first=True),
                                   dict(heads_first=True, pad=8, gap=64)])
def test_strides(tg, shape):
    ah.check_forward(tg, ah.Problem([150, 33], [170, 33], heads=4, kv=2, dim=72, **shape))


def test_rows_of_no_sequence(tg):
    """Gaps before, between and behind the sequences hold NaN and stay so."""
    p = ah.Problem([100, 37], [130, 1], heads=2, kv=2, dim=64, q_at=[7, 200], k_at=[3, 300], q_rows=260,
                   k_rows=320)
    ah.check_forward(tg, p)


@pytest.mark.parametrize("sigma,scale", [(4.0, 1.0), (0.01, 1.0), (1.0, 30.0), (1.0, 1e-6)])
def test_score_magnitudes(tg, sigma, scale):
    ah.check_forward(tg, ah.Problem([300], heads=2, kv=1, dim=64, sigma=sigma, scale=scale))


def test_growing_maxima(tg):
    """Later keys outgrow the reference again and again: every block rescales."""
    p = ah.Problem([400], heads=2, kv=2, dim=64, causal=False, scale=1.0)
    p.Q.t.fill_(0.25)
    ramp = torch.arange(400, device="cuda").float()[:, None, None] / 16
    p.K.t.copy_(ramp.expand(400, 2, 64).to(torch.bfloat16))
    ah.check_forward(tg, p)


def plan(tg, p):
    text = tg.tg_attention_plan_describe(*p.sizes(), p.max_q, p.max_k, p.dtype)
    return dict((k, int(v)) for k, v in (x.split("=") for x in text.split()))


@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("tiles,ranges", [(1, False), (1, True), (2, False), (2, True)])
def test_every_plan(tg, tiles, ranges, dim, dtype):
    """One and two row tiles a CTA, whole keys and ranges of them."""
    if tiles == 1:
        p = ah.Problem([3, 1, 2], [2000, 700, 1500] if ranges else [5, 300, 128], heads=8, kv=2, dim=dim, dtype=dtype)
    elif ranges:
        p = ah.Problem([300, 200], [3000, 2900], heads=16, kv=16, dim=dim, dtype=dtype)
    else:
        p = ah.Problem([700, 300], heads=32, kv=16, dim=dim, dtype=dtype)
    got = plan(tg, p)
    assert got["tiles"] == tiles and (got["ranges"] > 1) == ranges, got
    ah.check_forward(tg, p)


def test_outgrown_reference(tg):
    """Sums far beyond what the first block's maximum can hold: scores that jump within
    a block, in its first half, its second half, and in single rows, with FP16's limit
    and with BF16's."""
    for dtype, jump in (("fp16", 30.0), ("bf16", 30.0), ("bf16", 200.0), ("fp16", 300.0)):
        for at in (130, 200, 255, 256, 390):
            p = ah.Problem([3], [400], heads=2, kv=2, dim=64, dtype=dtype, causal=False, scale=1.0, sigma=0.25)
            # key `at` scores `jump` for row 1 alone
            p.Q.t[1, :, 0] = jump ** 0.5
            p.K.t[:, :, 0] = 0.0
            p.K.t[at, :, 0] = jump ** 0.5
            ah.check_forward(tg, p, f"{dtype} jump {jump} at key {at}")


def test_shared_keys_and_mixed_arrays(tg):
    """Two sequences over the same keys (a common prefix), lengths for one side only."""
    p = ah.Problem([64, 5], [200, 130], heads=4, kv=2, dim=64, k_at=[0, 0], k_rows=200)
    p.K.before, p.V.before = p.K.buf.clone(), p.V.buf.clone()
    ah.check_forward(tg, p)
    q = ah.Problem([64, 5], [200, 130], heads=4, kv=2, dim=64)
    qa, ql, ka, kl = q.dev
    want, _ = ah.run_forward(tg, q)
    for arrays in ((qa, ql, ka, None), (qa, None, ka, kl), (qa, ql, ka, kl)):
        q.arrays = lambda a=arrays: a
        got, _ = ah.run_forward(tg, q)
        assert torch.equal(got.t, want.t)


def test_arrays_that_point_outside(tg):
    """Entries are cut to the tensors: nothing outside is touched, other sequences keep
    their results."""
    p = ah.Problem([50, 60], [50, 60], heads=2, kv=1, dim=64, q_at=[0, 50], k_at=[0, 50], q_rows=110, k_rows=110)
    want, _ = ah.run_forward(tg, p)
    big = 1 << 40
    for starts, lengths in (([0, 5000], [50, 60]), ([0, -3], [50, 60]), ([0, big], [50, big]), ([0, 50], [50, -7]),
                            ([0, -big], [50, big])):
        dev = [torch.tensor(v, dtype=torch.int64, device="cuda") for v in (starts + [0], lengths)]
        p.arrays = lambda d=dev: (d[0], d[1], d[0], d[1])
        got, z = ah.run_forward(tg, p)
        assert torch.equal(got.t[:50], want.t[:50])
        assert bool(torch.isnan(got.t[50:]).all()) and bool(torch.isnan(z[:, 50:]).all())
    # a length that runs past the end is cut there
    dev = [torch.tensor(v, dtype=torch.int64, device="cuda") for v in ([0, 50, 0], [50, big])]
    p.arrays = lambda: (dev[0], dev[1], dev[0], dev[1])
    got, _ = ah.run_forward(tg, p)
    assert torch.equal(got.t, want.t)


def test_infinities_behind_a_sequence(tg):
    """Keys and values of other sequences in the same block never matter."""
    for bad in (float("inf"), float("-inf"), float("nan")):
        p = ah.Problem([40, 30], [70, 90], heads=2, kv=1, dim=128, q_at=[0, 40], k_at=[0, 200], q_rows=70, k_rows=300)
        want, _ = ah.run_forward(tg, p)
        for x in (p.K, p.V):
            x.t[70:200] = bad
            x.t[290:] = bad
        got, _ = ah.run_forward(tg, p)
        assert torch.equal(got.t, want.t)


@pytest.mark.parametrize("causal", [True, False])
def test_shared_keys(tg, causal):
    """Sequences that read the same rows of a cache: a common prefix."""
    ah.check_forward(tg, ah.Problem([1, 5, 40], [300, 300, 170], heads=4, kv=2, dim=64, causal=causal,
                                    q_at=[0, 1, 6], k_at=[0, 0, 130], q_rows=46, k_rows=300))


@pytest.mark.parametrize("q_len,heads,dtype", [([3], 2, "bf16"), ([3], 2, "fp16"), ([300, 700], 32, "bf16")])
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_of_minus_infinity_before_low_ones(tg, q_len, heads, dtype, dim):
    """Two blocks of keys whose scores are all -infinity, then scores of -240 and
    less: the keys before have no part, bit for bit."""
    n = [200] * len(q_len)
    k_at = [256 + 500 * i for i in range(len(n))]

    def problem(at, length):
        p = ah.Problem(q_len, length, heads=heads, kv=heads, dim=dim, dtype=dtype, causal=False, scale=1 / 8,
                       k_at=at, k_rows=500 * len(n), max_k=456, seed=5)
        g = ah.gen(6)
        p.Q.t.copy_(torch.rand(p.Q.t.shape, generator=g, device="cuda") + 1)
        p.V.t.copy_(torch.randn(p.V.t.shape, generator=g, device="cuda"))
        p.K.t.copy_(-30 - torch.rand(p.K.t.shape, generator=g, device="cuda"))
        return p

    p = problem(k_at, n)
    want, z = ah.run_forward(tg, p)
    ah.check_forward(tg, p)
    late = problem([a - 256 for a in k_at], [m + 256 for m in n])
    for a in k_at:
        late.K.t[a - 256: a] = float("-inf")
    got, y = ah.run_forward(tg, late)
    assert torch.equal(got.t, want.t) and torch.equal(y, z)


def test_rows_past_32_bit_offsets(tg):
    """A cache whose later rows lie beyond 2^31 elements."""
    ld, rows = 1 << 21, 1100
    buf = torch.zeros(rows * ld // 4 + 4096, 4, dtype=torch.bfloat16, device="cuda").view(-1)
    p = ah.Problem([1, 9], [600, 500], heads=4, kv=2, dim=64, k_at=[0, 600], k_rows=rows)
    for name, at in (("K", 0), ("V", 512)):
        small = getattr(p, name)
        view = torch.as_strided(buf, (rows, 2, 64), (ld, 64, 1), at)
        view.copy_(small.t)

        class Wide:
            t, lay = view, (view, ld, 64)

            @staticmethod
            def d(x=view):
                return x.double()

        setattr(p, name, Wide)
    ah.check_forward(tg, p)


def test_repeats_streams_and_graphs(tg):
    """Bitwise the same again, on two streams at once, and replayed with other lengths."""
    cases = [ah.Problem([1] * 4, [900, 3000, 1, 2000], heads=8, kv=2, dim=128, seed=5),
             ah.Problem([700, 300], heads=32, kv=16, dim=64, dtype="fp16", seed=6)]
    want = [ah.run_forward(tg, p) for p in cases]
    side = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for p, s in zip(cases, side):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                o = ah.Tensor3(p.q_rows, p.heads, p.dim, p.dtype)
                z = torch.empty(p.heads, p.q_rows, device="cuda")
                ws = ah.space(tg.tg_attention_workspace_bytes(*p.sizes(), p.max_q, p.max_k, p.dtype))
                tg.check(tg.tg_attention(*p.sizes(), *p.Q.lay, *p.K.lay, *p.V.lay, *p.arrays(), p.max_q, p.max_k,
                                         p.causal, p.scale, *o.lay, z, p.dtype, ws, s))
                got.append((o, z, ws))
        torch.cuda.synchronize()
        for (o, z, _), (wo, wz) in zip(got, want):
            assert torch.equal(o.t, wo.t) and torch.equal(z, wz)
    # captured once, replayed after the lengths have changed on the device
    p = ah.Problem([1] * 4, [900, 3000, 1, 2000], heads=8, kv=2, dim=128, seed=5,
                   k_at=[0, 3000, 6000, 9000], q_at=[0, 1, 2, 3], k_rows=12000)
    p.K.t.normal_()
    p.V.t.normal_()
    o = ah.Tensor3(4, 8, 128, "bf16")
    z = torch.empty(8, 4, device="cuda")
    ws = ah.space(tg.tg_attention_workspace_bytes(*p.sizes(), 1, 3000, "bf16"))
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        tg.check(tg.tg_attention(*p.sizes(), *p.Q.lay, *p.K.lay, *p.V.lay, *p.arrays(), 1, 3000, True, p.scale,
                                 *o.lay, z, "bf16", ws, s))
    for lens in ([900, 3000, 1, 2000], [1, 2, 3000, 0], [2500, 129, 128, 127]):
        p.dev[3].copy_(torch.tensor(lens))
        p.k_len = lens
        g.replay()
        torch.cuda.synchronize()
        want, eo, lse, el = ah.reference(p)
        ah.check(o.t, want, eo, f"replayed with {lens}")
        ah.check(z, lse, el, f"replayed with {lens} LSE")


def staircase(q_len, k_len, heads, dim, dtype, seed):
    """A problem whose rows outgrow their reference again and again: a warp's rows (32
    of a tile's 128) score the same for a key but for noise, and every warp has
    its own half blocks from which on its keys score `step` more, beyond what a reference
    may lag behind (2^30 BF16, 2^14 FP16).  So warps rescale O in different halves of
    successive blocks.  (Steps are whole numbers, exact in both types.)"""
    p = ah.Problem(q_len, k_len, heads=heads, kv=heads, dim=dim, dtype=dtype, causal=False, scale=1.0, sigma=0.25,
                   seed=seed)
    step = 24 if dtype == "bf16" else 12
    g = torch.Generator().manual_seed(seed)
    p.Q.t[:, :, :4] = 0.0
    for at, n in zip(p.q_at, q_len):
        i = torch.arange(n, device="cuda")
        p.Q.t[at + i, :, i % 128 // 32] = 4.0
    for at, n in zip(p.k_at, k_len):
        first = torch.randint(0, 64, (-(-n // 64), heads, 4), generator=g)  # where in the half block
        rise = torch.rand(-(-n // 64), heads, 4, generator=g) < 0.4
        rise[:2] = False  # (the first block's maximum is the first reference)
        where = torch.arange(n)[:, None, None]
        level = torch.zeros(n, heads, 4)
        for b in range(2, rise.shape[0]):
            level += (rise[b] & (where >= 64 * b + first[b])).float()
        p.K.t[at: at + n, :, :4] = (level * (step // 4)).to("cuda", p.K.t.dtype)
    p.Q.before, p.K.before = p.Q.buf.clone(), p.K.buf.clone()
    return p


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tiles,ranges", [(1, False), (1, True), (2, False), (2, True)])
def test_warps_outgrow_their_reference_in_different_halves(tg, tiles, ranges, dim, dtype):
    """Against FP64, and bit for bit the same again."""
    if tiles == 1:
        p = staircase([128, 100], [1500, 1300], 8, dim, dtype, 3) if ranges else \
            staircase([128] * 20, [1000] * 20, 16, dim, dtype, 4)
    elif ranges:
        p = staircase([300, 200], [3000, 2900], 16, dim, dtype, 5)
    else:
        p = staircase([1500, 900], [900, 1000], 16, dim, dtype, 6)
    got = plan(tg, p)
    assert got["tiles"] == tiles and (got["ranges"] > 1) == ranges, got
    o, z = ah.check_forward(tg, p)
    for _ in range(10):
        again, y = ah.run_forward(tg, p)
        assert torch.equal(again.t, o.t) and torch.equal(y, z)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_len,k_len,heads,kv", [
    ([1] * 6, [5000, 1, 0, 4097, 640, 700], 8, 2),  # single tokens, key ranges
    ([3, 40, 100], [400, 300, 700], 2, 2),          # a tile a sequence
    ([300, 700], [900, 700], 32, 16),               # two tiles a CTA
    ([1] * 300, [300] * 300, 4, 4),                 # whole key ranges
])
def test_queries_of_others_have_no_say(tg, q_len, k_len, heads, kv, dim, dtype):
    """Rows of Q between and behind the sequences, and the other sequences' own, lie in the
    same tiles: whatever they hold, a sequence's results are the same bits."""
    at, gap = [], 5
    for n in q_len:
        at.append((at[-1] + q_len[len(at) - 1] if at else 0) + gap)
    p = ah.Problem(q_len, k_len, heads=heads, kv=kv, dim=dim, dtype=dtype, causal=False, q_at=at,
                   q_rows=at[-1] + q_len[-1] + 130, seed=8)
    rows = p.rows()
    noise = torch.randn(p.Q.t.shape, generator=ah.gen(9), device="cuda").to(p.Q.t.dtype)
    p.Q.t[~rows] = 0
    want, z = ah.run_forward(tg, p)
    for f in (100.0, 10000.0, float("inf"), float("-inf"), float("nan")):
        p.Q.t[~rows] = noise[~rows].abs() * f if f != 100.0 else noise[~rows] * f
        got, y = ah.run_forward(tg, p)
        assert torch.equal(got.t[rows], want.t[rows]) and torch.equal(y[:, rows], z[:, rows]), f
    # every other sequence's queries changed
    p.Q.t[~rows] = 0
    kept = torch.zeros_like(rows)
    for a, n in zip(at[::2], q_len[::2]):
        kept[a: a + n] = True
    p.Q.t[rows & ~kept] = noise[rows & ~kept] * 100
    got, y = ah.run_forward(tg, p)
    assert torch.equal(got.t[kept], want.t[kept]) and torch.equal(y[:, kept], z[:, kept])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_len,heads,kv", [([100, 18], 7, 1), ([126], 12, 4), ([900, 1500], 28, 4), ([60], 48, 8)])
def test_groups_that_leave_rows_of_a_tile(tg, q_len, heads, kv, dim, dtype):
    """The same bits again, whatever an earlier call left in the rows that no load writes."""
    p = ah.Problem(q_len, [700] * len(q_len), heads=heads, kv=kv, dim=dim, dtype=dtype, causal=False, seed=8)
    outs = []
    for f in (0.0, 100.0, 0.01, float("inf"), 30000.0):
        # 128 rows a tile, of one value: one tile a CTA and two
        for fill in (ah.Problem([128] * 40, [64] * 40, heads=8, kv=8, dim=dim, dtype=dtype),
                     ah.Problem([2048], [64], heads=32, kv=32, dim=dim, dtype=dtype)):
            fill.Q.t.copy_(torch.randn(fill.Q.t.shape, generator=ah.gen(10), device="cuda") * f)
            ah.run_forward(tg, fill)
        outs.append(ah.run_forward(tg, p))
    for o, z in outs[1:]:
        assert torch.equal(o.t, outs[0][0].t) and torch.equal(z, outs[0][1])
