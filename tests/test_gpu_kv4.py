"""The 4-bit KV cache on the GPU against the float64 oracle: rows appended and read back bit
for bit, attention with accumulated weights, eviction, and their run together."""

import numpy as np
import pytest
import torch

import block_causal_streaming_sa_b200 as sa
from oracle import kv4
from sa_inputs import seed_of

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U32 = 2.0 ** -24                    # half a step of fp32, relative
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11}  # half a step of the output type


def normal(tag, shape, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed_of("kv4", tag) % (1 << 62))
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


class Pair:
    """A cache on the GPU and the oracle, given the same calls."""

    def __init__(self, B, H, D, N, dtype=BF):
        self.gpu = sa.QuantKVCache(B, H, D, N)
        # rows that were never written hold the worst bytes: NaN scales, NaN weights
        for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
            getattr(self.gpu, name).fill_(0xFF)
        self.gpu.weight.fill_(float("nan"))
        self.gpu.pos.fill_(-7)
        self.ref = kv4.Kv4Oracle(B, H, D, N)
        self.dtype, self.shape = dtype, (B, H, D, N)

    def append(self, tag, T, counts=None, replace=False, scale=1.0):
        B, H, D, _ = self.shape
        K = normal((tag, "k"), (B, T, H, D), self.dtype, scale)
        V = normal((tag, "v"), (B, T, H, D), self.dtype, 0.5)
        c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.gpu.append(K.cuda(), V.cuda(), counts=c, replace=replace)
        self.ref.append(f64(K), f64(V), counts, replace)

    def check_rows(self):
        """Every row held, its position, and the counters: equal."""
        B, H, D, N = self.shape
        g = self.gpu
        seq = g.seq.cpu().tolist()
        assert seq[0] == [self.ref.held(b) for b in range(B)]
        assert seq[1] == self.ref.total and seq[2] == self.ref.last
        kc, vc, ks, vs, pos = (t.cpu().numpy() for t in
                               (g.k_codes, g.v_codes, g.k_scales, g.v_scales, g.pos))
        for b in range(B):
            n = self.ref.held(b)
            for h in range(H):
                at = (b, h, slice(0, n))
                assert np.array_equal(kv4.dequantise(kc[at], ks[at]), self.ref.k[b][h])
                assert np.array_equal(kv4.dequantise(vc[at], vs[at]), self.ref.v[b][h])
                assert np.array_equal(pos[at], self.ref.pos[b][h])

    def check_weights(self, calls, e_max):
        """Weights of `calls` attentions. Each probability is off by a factor of e^err, err as
        in check_attend, the sums in fp32 by one rounding a term and call."""
        w = self.gpu.weight.cpu().double().numpy()
        for b in range(self.shape[0]):
            for h in range(self.shape[1]):
                ref = self.ref.weight[b][h]
                tol = (4 * score_error(self.shape[2], e_max) + 64 * calls * U32) * ref + 1e-30
                d = np.abs(w[b, h, :len(ref)] - ref)
                assert np.all(d <= tol), (b, h, float((d / (ref + 1e-30)).max()))

    def check_attend(self, tag, T, heads, counts=None, causal=False, scale=0.0,
                     add_weight=False, q_scale=1.0, view=None):
        B, H, D, _ = self.shape
        Q = normal((tag, "q"), (B, T, heads, D), self.dtype, q_scale)
        q = Q.cuda() if view is None else view(Q.cuda())
        c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        out = torch.full((B, T, heads, D), 7.0, dtype=self.dtype, device="cuda")
        lse = torch.full((B, heads, T), 7.0, device="cuda")
        self.gpu.attend(q, counts=c, causal=causal, scale=scale, out=out, lse=lse,
                        add_weight=add_weight)
        O, L, A, E = self.ref.attend(f64(Q), counts, causal, scale if scale > 0 else None,
                                     add_weight)
        return compare(f64(out), f64(lse), O, L, A, E, D, HALF[self.dtype])


def score_error(D, e):
    """A bound on the error of a scaled score, in natural units, for sum |q k| scale <= e: the
    products are exact, D additions in fp32 of at least 23 bits each and two scalings
    (2 half steps each), Q's row scaled by a power of two to fp16 (2^-25 of its largest
    value, D of them against sum |q k|, at most another step each); exp2's argument is
    rounded once more and its value is 2^-22 off."""
    return (3 * D + 8) * U32 * e + 2.0 ** -21


def compare(o, l, O, L, A, E, D, half):
    """GPU's O and lse against the oracle's; entries the oracle leaves NaN must be 7."""
    none = np.isnan(O)
    assert np.all(o[none] == 7.0), "rows behind the valid ones were written"
    assert np.all(l[np.isnan(L)] == 7.0)
    e_max = float(np.nanmax(E)) if not np.all(np.isnan(E)) else 0.0
    err = np.where(np.isnan(E), 0.0, score_error(D, np.nan_to_num(E)))
    err_o = np.transpose(err, (0, 2, 1))[..., None]
    # O = sum p v: p off by e^err and its own rounding to fp16 (half a step, 2^-11), p below
    # 2^-14 of the largest by 2^-25 of it instead, the normalisation by e^err again; then
    # the output's rounding.
    tol = (2 * err_o + 2.0 ** -11 + 2.0 ** -20) * A + half * np.abs(O) + 1e-7
    d = np.abs(o - O)
    assert np.all(d[~none] <= tol[~none]), \
        f"O off by {np.nanmax(d):.3e}, {np.nanmax(d / tol):.2f} of the tolerance"
    fin = np.isfinite(L)
    assert np.array_equal(l[np.isneginf(L)], L[np.isneginf(L)])
    dl = np.abs(l[fin] - L[fin])
    assert np.all(dl <= (err + 4 * U32 * np.abs(np.nan_to_num(L, neginf=0.0)))[fin]), \
        f"lse off by {dl.max():.3e}"
    return e_max


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T", [1, 17, 130])
def test_append_stores_the_format_bit_for_bit(D, dtype, T):
    p = Pair(2, 3, D, 384, dtype)
    p.append(("fmt", D, T, 0), T)
    p.check_rows()
    p.append(("fmt", D, T, 1), T, scale=300.0)
    p.append(("fmt", D, T, 2), 5, scale=2.0 ** -12)  # scales below fp16's normal range
    p.check_rows()
    assert p.gpu.check() == sa.SA_OK


def test_append_ties_zeros_and_scale_edges():
    """Values built on midpoints of every scale's codes, and blocks of zeros."""
    p = Pair(1, 1, 128, 1024, HF)
    mid = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = []
    for byte in range(8, 227):
        s = float(kv4.SCALES[byte])
        block = torch.cat((mid, -mid)) * s
        rows.append(torch.cat((block, torch.zeros(16), -torch.zeros(16), block[:8], block[:8],
                               torch.zeros(64))))
    K = torch.stack(rows).half()[None, :, None]
    p.gpu.append(K.cuda(), (-K).cuda())
    p.ref.append(f64(K), f64(-K))
    p.check_rows()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_out_of_range_values_saturate_and_are_reported(dtype):
    p = Pair(1, 2, 64, 128, dtype)
    p.append(("range", 0), 3)
    big = torch.zeros((1, 3, 2, 64), dtype=dtype)
    big[0, 0, 0, 0] = 65504 if dtype == HF else 1e30
    big[0, 1, 1, 5] = -float("inf")
    p.gpu.append(big.cuda(), torch.zeros_like(big).cuda())
    assert p.gpu.check() == sa.SA_ERR_RANGE
    k, v = torch.zeros_like(big).cuda(), torch.zeros_like(big).cuda()
    p.gpu.read_last(k, v)
    assert k[0, 0, 0, 0] == 61440 and k[0, 1, 1, 5] == -61440 and k.abs().sum() == 2 * 61440
    big[0, 2, 0, 7] = float("nan")
    p.gpu.append(big.cuda(), big.cuda(), replace=True)
    p.gpu.read_last(k, v)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
    p.gpu.reset()
    assert p.gpu.check() == sa.SA_OK and p.gpu.seq.abs().sum() == 0


def test_append_ragged_replace_and_strided():
    B, H, D = 4, 3, 64
    p = Pair(B, H, D, 256)
    p.append("r0", 40, counts=[40, 0, 7, 33])
    p.append("r1", 20, counts=[20, 20, 0, 1])
    p.append("r2", 9, counts=[3, 9, 9, 0], replace=True)
    p.check_rows()
    # more than T or less than 0 is clamped
    K = normal("clamp", (B, 4, H, D), BF)
    c = torch.tensor([99, -5, 4, 2], dtype=torch.int32, device="cuda")
    p.gpu.append(K.cuda(), K.cuda(), counts=c)
    p.ref.append(f64(K), f64(K), [4, 0, 4, 2])
    p.check_rows()
    # slices of a fused projection, and a broadcast token
    kv = normal("fused", (B, 6, 2 * H + 1, D), BF).cuda()
    p.gpu.append(kv[:, :, :H], kv[:, :, H:2 * H])
    p.ref.append(f64(kv[:, :, :H]), f64(kv[:, :, H:2 * H]))
    one = normal("one", (B, 1, H, D), BF).cuda().expand(B, 5, H, D)
    p.gpu.append(one, one)
    p.ref.append(f64(one), f64(one))
    p.check_rows()
    # T = 0 adds nothing; with replace it drops the last rows
    none = torch.empty((B, 0, H, D), dtype=BF, device="cuda")
    p.gpu.append(none, none, replace=True)
    p.ref.append(f64(none), f64(none), replace=True)
    p.check_rows()


def test_append_beyond_the_capacity_drops_rows_and_says_so():
    p = Pair(2, 2, 64, 128)
    p.append("c0", 120, counts=[120, 60])
    guard = [t.clone() for t in (p.gpu.k_codes, p.gpu.v_scales)]
    p.append("c1", 30)
    p.check_rows()
    assert p.gpu.seq[0].tolist() == [128, 90]
    assert p.gpu.check() == sa.SA_ERR_FULL
    assert torch.equal(guard[0][:, :, :60], p.gpu.k_codes[:, :, :60])
    p.check_attend("cq", 2, 2)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_read_leaves_rows_that_are_not_held(dtype):
    p = Pair(2, 2, 128, 128, BF)
    p.append("rd", 50, counts=[50, 20])
    k = torch.full((2, 40, 2, 128), 3.0, dtype=dtype, device="cuda")
    v = k.clone()
    p.gpu.read(15, k, v)
    for b, n in ((0, 35), (1, 5)):
        for h in range(2):
            assert np.array_equal(f64(k[b, :n, h]), p.ref.k[b][h][15:15 + n])
            assert np.array_equal(f64(v[b, :n, h]), p.ref.v[b][h][15:15 + n])
        assert (k[b, n:] == 3).all() and (v[b, n:] == 3).all()
    k.fill_(3)
    p.gpu.read(2 ** 31 - 1, k, v)
    assert (k == 3).all()


# ------------------------------------------------------------------ attention

SHAPES = [
    # B, Hk, group, D, T, rows of each sequence, causal
    (1, 1, 1, 64, 1, [1], False),
    (1, 2, 4, 128, 1, [700], False),
    (3, 2, 1, 128, 1, [129, 0, 64], False),
    (2, 1, 8, 64, 1, [2000, 31], True),
    (2, 3, 3, 128, 5, [333, 5], True),
    (1, 1, 5, 64, 7, [40], True),
    (2, 1, 16, 128, 2, [513, 900], False),
    (1, 2, 12, 64, 3, [257], True),
    (1, 2, 1, 128, 64, [64], True),
    (2, 2, 2, 64, 65, [200, 65], True),
    (1, 2, 1, 128, 127, [300], False),
    (1, 1, 1, 64, 128, [128], True),
    (1, 2, 4, 128, 129, [400], True),
    (2, 1, 3, 128, 100, [100, 385], True),
    (1, 3, 1, 64, 192, [576], False),
    (1, 1, 2, 128, 300, [1500], False),
    (1, 1, 7, 64, 97, [640], True),
    (1, 1, 1, 128, 513, [513], True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attend_matches_the_oracle(shape, dtype):
    B, H, G, D, T, rows, causal = shape
    p = Pair(B, H, D, -(-max(max(rows), T) // 128) * 128, dtype)
    p.append(("att", shape), max(rows), counts=rows)
    e = p.check_attend(("att", shape), T, H * G, counts=[min(T, n) if causal else T for n in rows],
                       causal=causal, add_weight=True)
    p.check_weights(1, e)
    e = max(e, p.check_attend(("att2", shape), T, H * G,
                              counts=[min(T, n) if causal else T for n in rows],
                              causal=causal, add_weight=True, scale=0.3, q_scale=0.5))
    p.check_weights(2, e)
    assert p.gpu.check() == sa.SA_OK


@pytest.mark.parametrize("G,T", [(1, 8), (3, 3), (2, 8), (1, 17), (8, 3), (5, 5), (4, 8), (11, 3),
                                 (8, 5), (7, 7), (16, 4), (5, 13)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_around_every_count_of_few_query_rows(G, T, D):
    """Query rows from one block of 8 to two of 32 and just beyond, masked inside a tile."""
    rows = [T + 3, 97, 161, 0, 64]
    p = Pair(5, 2, D, 256, HF)
    p.append(("few", G, T, D), 161, counts=rows)
    counts = [T, T - 1, T, 0, 1]
    e = p.check_attend(("few", G, T, D), T, 2 * G, counts=counts, causal=True, add_weight=True)
    e = max(e, p.check_attend(("few2", G, T, D), T, 2 * G, add_weight=True, q_scale=2.0))
    p.check_weights(2, e)


@pytest.mark.parametrize("T", [1, 5, 70])
def test_attend_many_sequences(T):
    """More sequences than a warp has lanes, of every length from none to several tiles."""
    B, H, G, D = 70, 2, 2, 64
    p = Pair(B, H, D, 256)
    lens = [(b * 37) % 200 for b in range(B)]
    p.append(("many", T), 200, counts=lens)
    counts = [min(T, n) if b % 3 else 0 for b, n in enumerate(lens)]
    e = p.check_attend(("many", T), T, H * G, counts=counts, causal=True, add_weight=True)
    p.check_weights(1, e)


def test_attend_items_split_over_many_blocks():
    """One head with a long cache: every block has a part of it, few and many query rows."""
    H, D, n = 1, 128, 40_000
    p = Pair(1, H, D, 40_064)
    for i in range(4):
        p.append(("split", i), n // 4)
    e = 0.0
    for T, G in ((1, 2), (6, 2), (40, 2), (300, 2)):
        e = max(e, p.check_attend(("split", T), T, G, add_weight=True))
    p.check_weights(4, e)


@pytest.mark.parametrize("T", [1, 4, 90, 200])
def test_attend_ragged_counts_leave_the_rest(T):
    B, H, G, D = 4, 2, 2, 128
    counts = [T, 0, max(1, T // 3), T - T // 4]
    p = Pair(B, H, D, 512)
    p.append(("rag", T), 450, counts=[450, 300, T + 5, T])
    for causal in (False, True):
        e = p.check_attend(("rag", T, causal), T, H * G, counts=counts, causal=causal,
                           add_weight=True)
    p.check_weights(2, e)


@pytest.mark.parametrize("T", [1, 3, 150])
def test_attend_without_rows_gives_zero_and_minus_infinity(T):
    p = Pair(2, 2, 64, 128)
    p.check_attend(("empty", T), T, 4, add_weight=True)
    p.append(("empty", T), 20, counts=[0, 20])
    p.check_attend(("empty1", T), T, 4, add_weight=True)
    assert torch.isnan(p.gpu.weight[0]).all()  # no row held: no weight touched


@pytest.mark.parametrize("T", [1, 6, 140])
def test_attend_large_and_sharp_scores(T):
    """Keys of very different size, so that maxima grow along the rows and most
    probabilities vanish; queries whose largest values are far from 1."""
    for D, dtype, qs in ((128, BF, 40.0), (64, HF, 20.0), (128, BF, 2.0 ** -30)):
        p = Pair(1, 2, D, 1024, dtype)
        for i in range(4):
            p.append(("sharp", T, i, D), 200, scale=0.3 * 3.0 ** i)
        p.check_attend(("sharp", T, D, qs), T, 4, q_scale=qs, add_weight=True)


@pytest.mark.parametrize("T", [1, 130])
def test_attend_with_infinite_or_nan_queries_spares_the_others(T):
    p = Pair(1, 1, 128, 256)
    p.append(("nan", T), 200)
    Q = normal(("nan", T), (1, T, 8, 128), BF).cuda()
    ref = p.gpu.attend(Q)
    Q[0, 0, 2, 5], Q[0, 0, 4, 9] = float("nan"), float("inf")
    out = p.gpu.attend(Q)
    assert torch.isnan(out[0, 0, 2].float()).all()
    keep = [0, 1, 3, 5, 6, 7]
    assert torch.equal(out[0, 0, keep], ref[0, 0, keep]) and torch.equal(out[0, 1:], ref[0, 1:])


@pytest.mark.parametrize("T", [1, 5, 133])
def test_attend_strided_queries_and_outputs(T):
    B, H, G, D = 2, 2, 2, 64
    p = Pair(B, H, D, 256)
    p.append(("str", T), 210)
    Q = normal(("strq", T), (B, T, H * G, D), BF).cuda()
    ref = p.gpu.attend(Q)
    fused = torch.zeros((B, T, H * G + 2 * H, D), dtype=BF, device="cuda")
    fused[:, :, :H * G] = Q
    out = torch.full((B, H * G, T, D + 8), 7.0, dtype=BF, device="cuda")
    p.gpu.attend(fused[:, :, :H * G], out=out[..., :D].transpose(1, 2))
    assert torch.equal(out[..., :D].transpose(1, 2), ref) and (out[..., D:] == 7).all()


@pytest.mark.parametrize("T", [1, 9, 200])
def test_attend_repeats_to_the_bit(T):
    p = Pair(3, 2, 128, 2048)
    p.append(("rep", T), 2000, counts=[2000, 777, 1300])
    Q = normal(("rep", T), (3, T, 8, 128), BF).cuda()
    got = []
    for _ in range(3):
        p.gpu.weight.zero_()
        lse = torch.empty((3, 8, T), device="cuda")
        out = p.gpu.attend(Q, lse=lse, add_weight=True)
        got.append((out, lse, p.gpu.weight.clone()))
    for x in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, got[0]))


def test_attend_two_halves_merge_by_lse():
    """Attention over two caches merged by lse equals attention over their rows."""
    H, D, n = 2, 128, 300
    whole, a, b = (Pair(1, H, D, 768) for _ in range(3))
    for tag, p in (("m0", a), ("m1", b)):
        p.append(tag, n)
        whole.append(tag, n)
    Q = normal("mq", (1, 3, H, D), BF)
    outs, lses = [], []
    for p in (a, b):
        lse = torch.empty((1, H, 3), device="cuda")
        outs.append(p.gpu.attend(Q.cuda(), lse=lse).double())
        lses.append(lse.double().transpose(1, 2)[..., None])
    w = torch.softmax(torch.stack(lses), 0)
    merged = (w * torch.stack(outs)).sum(0)
    O, _, A, E = whole.ref.attend(f64(Q))
    tol = (2 * score_error(D, E.max()) + 2.0 ** -11 + 2 * HALF[BF]) * A + 1e-6
    assert np.all(np.abs(f64(merged) - O) <= tol)


def test_attend_beyond_32_bit_offsets():
    """Planes of more than 2^32 bytes of codes: the last head's rows."""
    H, D, N = 72, 128, 1 << 20
    p = sa.QuantKVCache(1, H, D, N)
    ref = kv4.Kv4Oracle(1, H, D, N)
    K, V = normal("bigk", (1, 40, H, D), BF), normal("bigv", (1, 40, H, D), BF)
    p.append(K.cuda(), V.cuda())
    ref.append(f64(K), f64(V))
    assert p.k_codes.numel() > 1 << 32
    for T in (1, 130):
        Q = normal(("bigq", T), (1, T, H, D), BF)
        out = torch.full(Q.shape, 7.0, dtype=BF, device="cuda")
        lse = torch.full((1, H, T), 7.0, device="cuda")
        p.attend(Q.cuda(), out=out, lse=lse, add_weight=True)
        O, L, A, E = ref.attend(f64(Q), add_weight=True)
        compare(f64(out), f64(lse), O, L, A, E, D, HALF[BF])
    w = f64(p.weight[0, :, :40])
    want = np.stack(ref.weight[0])
    assert np.allclose(w, want, rtol=1e-3)
    p.evict(30, recent=4)
    ref.evict(30, recent=4)
    assert p.seq[0].tolist() == [30]
    k, v = (torch.zeros((1, 30, H, D), dtype=BF, device="cuda") for _ in range(2))
    p.read(0, k, v)
    assert np.array_equal(f64(k[0, :, H - 1]), ref.k[0][H - 1])


def test_causal_after_an_eviction_is_reported():
    p = Pair(1, 1, 64, 256)
    p.append("ord", 100)
    p.gpu.weight.zero_()
    p.gpu.evict(60)
    q = normal("ordq", (1, 4, 1, 64), BF).cuda()
    p.gpu.attend(q[:, :1], causal=True)
    assert p.gpu.check() == sa.SA_OK  # one token: every row is before it
    p.append("ord2", 4)
    p.gpu.attend(q, causal=True)
    assert p.gpu.check() == sa.SA_OK
    p.gpu.attend(torch.cat((q, q), 1), causal=True)
    assert p.gpu.check() == sa.SA_ERR_STATE


# ------------------------------------------------------------------ eviction

def evict_both(p, keep, first=0, recent=0):
    p.gpu.evict(keep, first=first, recent=recent)
    p.ref.evict(keep, first, recent)


def set_weights(p, tag, ties=False):
    B, H, D, N = p.shape
    g = torch.Generator().manual_seed(seed_of("kv4w", tag) % (1 << 62))
    w = torch.randint(0, 6, (B, H, N), generator=g).float() if ties else \
        torch.randn((B, H, N), generator=g)
    p.gpu.weight.copy_(w)
    for b in range(B):
        for h in range(H):
            p.ref.weight[b][h] = w[b, h, :p.ref.held(b)].double().numpy()


def check_evicted(p):
    p.check_rows()
    w = f64(p.gpu.weight)
    for b in range(p.shape[0]):
        for h in range(p.shape[1]):
            ref = p.ref.weight[b][h]
            assert np.array_equal(w[b, h, :len(ref)], ref, equal_nan=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("n,keep,first,recent", [
    (2, 1, 0, 0), (129, 128, 0, 0), (300, 299, 4, 16), (300, 1, 0, 0), (300, 1, 1, 0),
    (1000, 500, 0, 0), (1000, 500, 250, 250), (1500, 1100, 16, 64), (2100, 7, 3, 2),
])
def test_evict_matches_the_oracle(D, ties, n, keep, first, recent):
    p = Pair(2, 3, D, -(-n // 128) * 128)
    p.append(("ev", n), n, counts=[n, max(1, n - 40)])
    set_weights(p, (n, keep, ties), ties)
    evict_both(p, keep, first, recent)
    check_evicted(p)
    if keep > 1:  # again, with rows out of order
        p.append(("ev2", n), min(n - keep, 100))
        set_weights(p, (n, keep, ties, 2), ties)
        evict_both(p, keep - 1, min(first, 1), min(recent, keep - 2))
        check_evicted(p)


@pytest.mark.parametrize("n,keep", [(8200, 8000), (20_000, 9_001), (33_000, 32_999)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_over_several_blocks(n, keep, ties):
    """Heads shared by clusters of two to eight blocks, most weights equal or all distinct."""
    H, D = 3, 64
    c = sa.QuantKVCache(1, H, D, -(-n // 128) * 128)
    g = torch.Generator(device="cuda").manual_seed(n)
    K = torch.randn((1, n, H, D), generator=g, device="cuda").bfloat16()
    c.append(K, K)
    w = torch.randint(0, 2, c.weight.shape, generator=g, device="cuda").float() if ties else \
        torch.rand(c.weight.shape, generator=g, device="cuda")
    c.weight.copy_(w)
    vc = c.v_codes.clone()
    c.evict(keep, first=5, recent=100)
    for h in range(H):
        src = torch.tensor(kv4.rows_after_eviction(w[0, h, :n].cpu().numpy(), np.arange(n), n,
                                                   keep, 5, 100), device="cuda")
        assert torch.equal(c.weight[0, h, :keep], w[0, h, src])
        assert torch.equal(c.v_codes[0, h, :keep], vc[0, h, src])
        assert torch.equal(c.pos[0, h, :keep], src.int())


def test_evict_leaves_shorter_sequences_and_rows_behind():
    p = Pair(3, 2, 64, 512)
    p.append("sh", 400, counts=[400, 0, 150])
    set_weights(p, "sh")
    tail = [t[:, :, 200:].clone() for t in (p.gpu.k_codes, p.gpu.weight, p.gpu.pos)]
    evict_both(p, 200)
    check_evicted(p)
    for t, was in zip((p.gpu.k_codes, p.gpu.weight, p.gpu.pos), tail):
        now = t[:, :, 200:]
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8))
    assert p.gpu.seq[3].tolist() == [0, 0, 150]
    # nothing to evict: nothing changes
    before = p.gpu.seq.clone()
    evict_both(p, 200)
    evict_both(p, 512)
    evict_both(p, 100000)
    assert torch.equal(before, p.gpu.seq)
    check_evicted(p)


def test_evict_special_weights():
    """NaN below -inf, both zeros equal, +inf above every number but not above a protected
    row."""
    p = Pair(1, 1, 64, 128)
    p.append("sp", 12)
    inf, nan = float("inf"), float("nan")
    w = torch.tensor([nan, -0.0, 0.0, -inf, inf, 1e-45, -1e-45, 3e38, nan, -0.0, 0.0, -5.0])
    for keep in range(1, 12):
        q = Pair(1, 1, 64, 128)
        q.append("sp", 12)
        q.gpu.weight[0, 0, :12] = w.cuda()
        q.ref.weight[0][0] = w.double().numpy()
        evict_both(q, keep, recent=1)
        check_evicted(q)


def test_evict_long_rows():
    """More rows than any one block's registers or shared memory would hold."""
    H, D, n, keep = 2, 64, 150_000, 120_001
    c = sa.QuantKVCache(1, H, D, -(-n // 128) * 128)
    g = torch.Generator(device="cuda").manual_seed(5)
    K = torch.randn((1, n, H, D), generator=g, device="cuda").bfloat16()
    c.append(K, K)
    c.weight.copy_(torch.randint(0, 50_000, c.weight.shape, generator=g, device="cuda"))
    w, kc = c.weight.clone(), c.k_codes.clone()
    c.evict(keep, first=10, recent=1000)
    for h in range(H):
        src = torch.tensor(kv4.rows_after_eviction(w[0, h, :n].cpu().numpy(), np.arange(n), n,
                                                   keep, 10, 1000), device="cuda")
        assert torch.equal(c.weight[0, h, :keep], w[0, h, src])
        assert torch.equal(c.k_codes[0, h, :keep], kc[0, h, src])
        assert torch.equal(c.pos[0, h, :keep], src.int())


# ------------------------------------------------------------------ together

def test_a_stream_of_chunks_with_denoising_steps_and_eviction():
    """Each chunk: appended, re-appended at every step, attended with weights at the last,
    then the cache evicted to its bound. The weights pick the rows, so the oracle is given
    the GPU's weights before it evicts."""
    B, H, G, D, L, keep = 1, 2, 1, 64, 192, 400
    p = Pair(B, H, D, 640)
    for chunk in range(5):
        for step in range(3):
            p.append(("stream", chunk, step), L, replace=step > 0)
            p.check_attend(("stream", chunk, step), L, H * G, add_weight=step == 2)
        p.check_rows()
        w = f64(p.gpu.weight)
        for h in range(H):
            p.ref.weight[0][h] = w[0, h, :p.ref.held(0)]
        evict_both(p, keep, first=32, recent=64)
        check_evicted(p)
    assert p.gpu.check() == sa.SA_OK


def test_a_decoding_loop_captured_and_replayed():
    """append, attend with weights, evict as one graph: the rows' numbers live on the device,
    so one capture serves every step, growth and steady state alike."""
    B, H, G, D, keep, steps = 3, 2, 4, 128, 140, 30
    K = normal("gk", (steps, B, 1, H, D), BF).cuda()
    Q = normal("gq", (steps, B, 1, H * G, D), BF).cuda()

    def start():
        c = sa.QuantKVCache(B, H, D, 256)
        first = normal("g0", (B, 125, H, D), BF).cuda()
        c.append(first, first, counts=torch.tensor([125, 80, 0], dtype=torch.int32, device="cuda"))
        return c

    def step(c, k, q, out, lse):
        c.append(k, k)
        c.attend(q, out=out, lse=lse, add_weight=True, causal=True)
        c.evict(keep, first=4, recent=20)

    eager, want = start(), []
    for i in range(steps):
        out, lse = torch.empty_like(Q[0]), torch.empty((B, H * G, 1), device="cuda")
        step(eager, K[i], Q[i], out, lse)
        want.append((out, lse))

    c = start()
    k, q = K[0].clone(), Q[0].clone()
    out, lse = torch.empty_like(q), torch.empty((B, H * G, 1), device="cuda")
    warm = start()
    step(warm, k, q, out, lse)  # library loaded
    c._workspaces = warm._workspaces
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(c, k, q, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(steps):
        k.copy_(K[i])
        q.copy_(Q[i])
        graph.replay()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
    assert torch.equal(c.seq, eager.seq) and c.seq[0].tolist() == [140, 110, 30]
    for b in range(B):
        n = c.seq[0, b]
        assert torch.equal(c.weight[b, :, :n], eager.weight[b, :, :n])
        assert torch.equal(c.k_codes[b, :, :n], eager.k_codes[b, :, :n])
    assert c.check() == sa.SA_OK


def test_capture_needs_the_workspace_to_be_there():
    p = Pair(1, 1, 64, 128)
    p.append("cap", 10)
    q = normal("capq", (1, 1, 1, 64), BF).cuda()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before capturing"):
        with torch.cuda.graph(graph):
            p.gpu.attend(q)
    torch.cuda.synchronize()
    out = p.gpu.attend(q)  # and the cache still works
    assert torch.isfinite(out.float()).all()


def test_a_larger_workspace_leaves_captured_graphs_theirs():
    """A call that needs a larger workspace comes between a capture and its replay."""
    p = Pair(1, 2, 64, 512)
    p.append("wsp", 400)
    q = normal("wspq", (1, 1, 4, 64), BF).cuda()
    out = torch.empty_like(q)
    p.gpu.attend(q, out=out)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.gpu.attend(q, out=out)
    big = normal("wspb", (1, 300, 4, 64), BF).cuda()
    p.gpu.attend(big, add_weight=True)
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    out.zero_()
    graph.replay()
    assert torch.equal(out, want) and len(junk) == 8


def test_calls_on_another_stream():
    p = Pair(1, 2, 64, 256)
    side = torch.cuda.Stream()
    K = normal("sk", (1, 50, 2, 64), BF).cuda()
    torch.cuda.synchronize()
    p.gpu.append(K, K, stream=side)
    out = torch.empty((1, 50, 2, 64), dtype=BF, device="cuda")
    torch.cuda.synchronize()
    p.gpu.attend(K, out=out, stream=side, add_weight=True)
    p.gpu.evict(20, stream=side)
    assert p.gpu.check(side) == sa.SA_OK
    p.ref.append(f64(K), f64(K))
    O, _, A, _ = p.ref.attend(f64(K))
    assert np.all(np.abs(f64(out) - O) <= 2 * HALF[BF] * A + 1e-3 * A)
    assert p.gpu.seq[0].tolist() == [20]


def test_memory_comes_from_the_stream_that_writes_it():
    c = sa.QuantKVCache(1, 2, 64, 256)
    side = torch.cuda.Stream()
    K = normal("sm", (1, 50, 2, 64), BF).cuda()
    torch.cuda.synchronize()
    c.append(K, K, stream=side)
    out = c.attend(K, stream=side, add_weight=True)
    here = c.attend(K)
    assert c.check(side) == sa.SA_OK
    at = {t.data_ptr(): s["stream"] for t in (out, here, c._workspaces[-1])
          for s in torch.cuda.memory_snapshot()
          if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]}
    assert at == {out.data_ptr(): side.cuda_stream, c._workspaces[-1].data_ptr(): side.cuda_stream,
                  here.data_ptr(): torch.cuda.current_stream().cuda_stream}
    torch.cuda.synchronize()
    assert torch.equal(out, here)


@pytest.mark.parametrize("T", [1, 12, 200])
def test_lengths_are_those_behind_a_long_append(T):
    """Kernels may begin while the ones in front of them run: a sequence of calls without a
    pause gives the bits it gives with a wait after each."""
    H, D, rows = 12, 128, 9000
    g = torch.Generator(device="cuda").manual_seed(T)
    K = torch.randn((2, rows, H, D), generator=g, device="cuda").bfloat16()
    Q = torch.randn((2, T, H, D), generator=g, device="cuda").bfloat16()
    counts = torch.tensor([rows, 217], dtype=torch.int32, device="cuda")

    def run(pause):
        c = sa.QuantKVCache(2, H, D, 36096)
        results = []
        for i in range(4):
            c.append(K, K, counts=counts)
            pause()
            lse = torch.empty((2, H, T), device="cuda")
            results += [c.attend(Q, causal=True, lse=lse, add_weight=True), lse]
            pause()
        c.evict(11_000, 16, 500)
        pause()
        results.append(c.attend(Q, add_weight=True))
        assert c.check() == sa.SA_OK
        return results + [c.weight[1, :, :868], c.weight[0, :, :11_000], c.pos[0, :, :11_000]]

    run(torch.cuda.synchronize)  # workspaces and modules are there
    want = run(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))


# ------------------------------------------------------------------ refusals

def test_refusals_launch_nothing():
    p = Pair(2, 2, 64, 128)
    p.append("ref", 30)
    before = {n: getattr(p.gpu, n).clone() for n in ("seq", "k_codes", "weight", "status")}
    c, g = p.gpu._c, p.gpu
    x = torch.zeros((2, 3, 2, 64), dtype=BF, device="cuda")
    rows = sa.SaRows(x.data_ptr(), x.stride(0), x.stride(1), x.stride(2))
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(x)
    orow = sa.SaRows(o.data_ptr(), x.stride(0), x.stride(1), x.stride(2))

    def bad(status, call, *args, **kw):
        with pytest.raises(sa.SaError) as e:
            call(*args, **kw)
        assert e.value.status == status and "kv4: " in sa.last_error()

    inv = sa.SA_ERR_INVALID_ARG
    full = dict(workspace=ws.data_ptr(), workspace_bytes=ws.numel())
    bad(inv, sa.sa_kv4_append, c, rows, rows, 7, 3)
    bad(inv, sa.sa_kv4_append, c, rows, rows, 0, -1)
    bad(inv, sa.sa_kv4_append, c, rows, None, 0, 3)
    bad(inv, sa.sa_kv4_append, c, sa.SaRows(x.data_ptr() + 2, 384, 128, 64), rows, 0, 3)
    bad(inv, sa.sa_kv4_append, c, sa.SaRows(x.data_ptr(), 384, 124, 64), rows, 0, 3)
    bad(inv, sa.sa_kv4_append, c, sa.SaRows(x.data_ptr(), 384, -128, 64), rows, 0, 3)
    host = torch.zeros(4096, dtype=torch.uint8)
    hrow = sa.SaRows((host.data_ptr() + 15) & ~15, 384, 128, 64)
    bad(inv, sa.sa_kv4_append, c, hrow, rows, 0, 3)
    bad(inv, sa.sa_kv4_append, c, rows, rows, 0, 3, counts=host.data_ptr() & ~3)
    bad(inv, sa.sa_kv4_read, c, -2, rows, orow, 0, 3)
    bad(inv, sa.sa_kv4_read, c, 0, rows, rows, 0, 3)
    bad(inv, sa.sa_kv4_read, c, 0, sa.SaRows(x.data_ptr(), 384, 0, 64), orow, 0, 3)
    bad(inv, sa.sa_kv4_read, c, 0, sa.SaRows(x.data_ptr(), 384, 64, 64), orow, 0, 3)
    bad(inv, sa.sa_kv4_read, c, 0, sa.SaRows(x.data_ptr(), 320, 128, 64), orow, 0, 3)
    bad(inv, sa.sa_kv4_attend, c, rows, orow, 0, 3, 3, **full)   # heads % kv_heads
    bad(inv, sa.sa_kv4_attend, c, rows, rows, 0, 2, 3, **full)   # O aliases Q
    bad(inv, sa.sa_kv4_attend, c, rows, orow, 0, 2, 3, scale=float("nan"), **full)
    bad(inv, sa.sa_kv4_attend, c, rows, orow, 0, 2, 3, lse=ws.data_ptr() + 2, **full)
    need = sa.sa_kv4_attend_bytes(c, 2, 3, True)
    bad(inv, sa.sa_kv4_attend, c, rows, orow, 0, 2, 3, add_weight=True,
        workspace=ws.data_ptr(), workspace_bytes=need - 1)
    bad(inv, sa.sa_kv4_attend, c, rows, orow, 0, 2, 3, add_weight=True,
        workspace=ws.data_ptr() + 16, workspace_bytes=1 << 16)
    bad(inv, sa.sa_kv4_evict, c, 0, **full)
    bad(inv, sa.sa_kv4_evict, c, 5, first=3, recent=3, **full)
    bad(inv, sa.sa_kv4_evict, c, 5, first=-1, **full)
    bad(inv, sa.sa_kv4_evict, c, 5)
    bad(sa.SA_ERR_UNSUPPORTED, sa.sa_kv4_append, c, rows, rows, 0, 1 << 30)
    # the wrapper's own checks
    for call in (lambda: g.append(x.float(), x.float()), lambda: g.append(x, x[:, :2]),
                 lambda: g.append(x, x.half()), lambda: g.append(x.cpu(), x.cpu()),
                 lambda: g.attend(x[:, :, :1]), lambda: g.attend(x, out=o[:, :2]),
                 lambda: g.attend(x, lse=torch.zeros(5, device="cuda")),
                 lambda: g.append(x, x, counts=torch.zeros(2, dtype=torch.int64, device="cuda")),
                 lambda: g.append(x.transpose(2, 3)[:, :, :2], x),
                 lambda: sa.QuantKVCache(1, 1, 64, 100)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    for n, was in before.items():
        assert torch.equal(getattr(p.gpu, n).view(torch.uint8), was.view(torch.uint8)), n
    assert g.check() == sa.SA_OK


def test_from_tensors_checks_shapes():
    a = sa.QuantKVCache(1, 2, 64, 128)
    names = ("k_codes", "v_codes", "k_scales", "v_scales", "pos", "weight", "seq", "status")
    t = {n: getattr(a, n) for n in names}
    b = sa.QuantKVCache.from_tensors(**t)
    K = normal("ft", (1, 4, 2, 64), BF).cuda()
    b.append(K, K)
    assert a.seq[0].tolist() == [4]
    for n, wrong in (("pos", t["weight"]), ("k_scales", t["k_codes"]), ("seq", t["seq"][:3])):
        with pytest.raises(ValueError):
            sa.QuantKVCache.from_tensors(**dict(t, **{n: wrong}))
