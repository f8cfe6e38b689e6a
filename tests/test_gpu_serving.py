"""GPU: rotary positions, the nested cache's rows, attention over a shared
prefix, received weights and eviction against oracle/serving.py (fp64).

Tolerances are bounds of the arithmetic, stated where they are made: u = 2^-24
is a rounding to fp32, h = 2^-11 one to fp16 (relative)."""
import numpy as np
import pytest

import oracle
import w8_quantized_linear_b200 as bn
from oracle import serving as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

from test_gpu_parity import dev, host  # noqa: E402


@pytest.fixture(autouse=True)
def _no_wait_timeouts():
    bn.device_wait_timeout(reset=True)
    yield
    torch.cuda.synchronize()
    assert bn.device_wait_timeout(reset=True) == 0


U, HALF = 2.0 ** -24, 2.0 ** -11
LAYOUT = {"half": bn.ROPE_HALF, "pairs": bn.ROPE_PAIRS}
DTYPE = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ rotary
def _rope_bound(x, rot, layout, mag):
    """|a| + |b| of each value's pair, |x| of the others."""
    a = np.abs(np.asarray(x, np.float64))
    i = np.arange(rot // 2)
    p, q = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    s = a.copy()
    s[..., p] = s[..., q] = mag * (a[..., p] + a[..., q])
    return s


def _check_rope(y, x, w, rot, layout, mag, inverse):
    want = ref.rope(x, w, mag, layout, inverse)
    # a value is a c - b s: the angle is off by 9.4e-8 (24 of its bits), sincospif
    # by 2 ulp = 2 u of at most 1, and three fp32 roundings follow: < 4e-7 (|a| + |b|)
    tol = 4e-7 * _rope_bound(x, rot, layout, mag)
    if y.dtype == torch.float16:
        tol = tol * (1 + HALF) + HALF * np.abs(want) + 2.0 ** -25
    else:
        tol[..., rot:] = 0.0
    assert np.all(np.abs(host(y).astype(np.float64) - want) <= tol)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("src,dst", [("f16", "f16"), ("f16", "f32"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("M,heads,D,rot", [(1, 1, 2, 2), (3, 5, 128, 128), (7, 32, 128, 64),
                                           (2, 3, 80, 40), (5, 2, 96, 96), (4, 3, 65, 30),
                                           (1031, 9, 64, 16)])
def test_rope_matches_formula(M, heads, D, rot, layout, src, dst):
    rng = np.random.default_rng(M + D + rot)
    x = rng.standard_normal((M, heads, D)).astype(np.float16 if src == "f16" else np.float32)
    pos = rng.integers(0, 1 << 20, M).astype(np.int32)
    phases, mag = bn.rope_phases(rot, 1e4)
    y = bn.rope(dev(x), dev(pos), phases, mag, LAYOUT[layout], dtype=DTYPE[dst])
    assert y.dtype == DTYPE[dst] and y.is_contiguous()
    w = ref.angles(host(phases).view(np.uint64), pos)
    _check_rope(y, x, w, rot, layout, 1.0, False)


@pytest.mark.parametrize("name,kw", [("plain", {}), ("linear", dict(factor=4.0)),
                                     ("ntk", dict(factor=4.0)),
                                     ("bands", dict(factor=8.0, low=1.0, high=4.0, trained=8192)),
                                     ("yarn", dict(factor=16.0, low=1.0, high=32.0, trained=4096))])
def test_rope_far_and_negative_positions(name, kw):
    """The extreme int32 positions: the angle from 64-bit integers is exact."""
    rot, pos = 64, np.array([0, 1, -1, 131071, -131071, 2 ** 31 - 1, -2 ** 31], np.int32)
    kind = ["plain", "linear", "ntk", "bands", "yarn"].index(name)
    phases, mag = bn.rope_phases(rot, 5e5, kind, **kw)
    theta, want_mag = ref.rope_theta(rot, 5e5, name, **kw)
    # two evaluations of theta in fp64 (a power, a few products), 16 roundings at most, and
    # the phase's own rounding to a unit of 2^-64 turns: half of one is 2 pi 2^-65
    assert np.all(np.abs(host(phases).view(np.uint64) / 2.0 ** 64 * 2 * np.pi - theta)
                  <= 2.0 ** -49 * theta + np.pi * 2.0 ** -64)
    assert mag == np.float32(want_mag)
    x = np.random.default_rng(1).standard_normal((len(pos), 2, rot)).astype(np.float32)
    y = bn.rope(dev(x), dev(pos), phases, mag, dtype=torch.float32)
    _check_rope(y, x, ref.angles(host(phases).view(np.uint64), pos), rot, "half",
                float(np.float32(mag)), False)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_strides_and_in_place(layout):
    """Columns of a wider array, heads before tokens, odd strides and starts, in
    place and into a part of another array; what lies beside stays."""
    rng = np.random.default_rng(5)
    M, heads, D, rot = 6, 4, 128, 64
    phases, mag = bn.rope_phases(rot, 1e4)
    pos = rng.integers(0, 9000, M).astype(np.int32)
    w = ref.angles(host(phases).view(np.uint64), pos)
    wide = dev(rng.standard_normal((M, 48 * D + 1)).astype(np.float32))
    for first in (0, 8, 3):
        x = wide[:, first:first + heads * D].unflatten(1, (heads, D))
        _check_rope(bn.rope(x, dev(pos), phases, mag, LAYOUT[layout]), host(x), w, rot, layout, 1.0, False)
    x = dev(rng.standard_normal((heads, M, D)).astype(np.float16)).transpose(0, 1)
    out = torch.full((heads, M, D + 8), 7.0, dtype=torch.float16, device="cuda")
    y = out[..., :D].transpose(0, 1)
    bn.rope(x, dev(pos), phases, mag, LAYOUT[layout], out=y)
    _check_rope(y, host(x), w, rot, layout, 1.0, False)
    assert torch.all(out[..., D:] == 7.0)
    fresh = bn.rope(x, dev(pos), phases, mag, LAYOUT[layout])
    assert bn.rope(x, dev(pos), phases, mag, LAYOUT[layout], out=x) is x
    assert torch.equal(x, fresh)
    before = wide.clone()
    part = wide[:, 3:3 + heads * D].unflatten(1, (heads, D))
    bn.rope(part, dev(pos), phases, mag, LAYOUT[layout], out=part)
    _check_rope(part, host(before[:, 3:3 + heads * D].unflatten(1, (heads, D))), w, rot, layout, 1.0, False)
    assert torch.equal(wide[:, :3], before[:, :3]) and torch.equal(wide[:, 3 + heads * D:], before[:, 3 + heads * D:])


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_gradient(layout):
    """The inverse turn is the gradient: the formula's (the transpose), and central
    differences of a weighted sum of the outputs (linear in x, so only rounding counts)."""
    rng = np.random.default_rng(2)
    M, heads, D, rot, mag = 3, 2, 16, 12, 1.25
    phases, _ = bn.rope_phases(rot, 100.0)
    pos = dev(np.array([0, 5, 77], np.int32))
    x, g = (rng.standard_normal((M, heads, D)).astype(np.float32) for _ in range(2))
    gx = host(bn.rope(dev(g), pos, phases, mag, LAYOUT[layout], inverse=True, dtype=torch.float32))
    w = ref.angles(host(phases).view(np.uint64), host(pos))
    _check_rope(dev(gx), g, w, rot, layout, mag, True)
    for at in [(0, 0, 0), (1, 1, 3), (2, 0, 11), (2, 1, 15), (1, 0, 6)]:
        d = []
        for step in (1.0, -1.0):
            y = x.copy()
            y[at] += step
            d.append(host(bn.rope(dev(y), pos, phases, mag, LAYOUT[layout], dtype=torch.float32)).astype(np.float64))
        # two values of at most 2 mag (|x| + 1) each off by 4e-7 of it and the step's
        # own rounding, weighted by |g| of the pair
        got = float(((d[0] - d[1]) / 2 * g).sum())
        size = np.abs(g[at[0], at[1]]).sum() * 2 * mag * (np.abs(x).max() + 1)
        assert abs(got - gx[at]) <= 1e-6 * size


# -------------------------------------------------------------- cache rows
def _rows(rng, *shape):
    x = rng.standard_normal((*shape, 128)) * 0.8
    x[..., 5] += 2.0
    return x.astype(np.float16)


def _packed(x):
    """The oracle's packing of fp16 rows [..., 128]."""
    hi, lo, sc = oracle.kv_pack(x.reshape(-1, 128))
    return (hi.reshape(*x.shape[:-1], 64), lo.reshape(*x.shape[:-1], 64),
            sc.view(np.float16).reshape(x.shape[:-1]))


def _np(planes):
    return tuple(host(t) for t in planes)


@pytest.mark.parametrize("src", ["f16", "f32"])
@pytest.mark.parametrize("B,L,Hkv,cap", [(1, 1, 1, 1), (3, 4, 8, 11), (2, 300, 2, 301), (5, 7, 3, 40)])
def test_append_packs_bit_for_bit(B, L, Hkv, cap, src):
    """Without turning: the oracle's packing, bit for bit, at each start; nothing else is written."""
    rng = np.random.default_rng(B * L + cap)
    x = [_rows(rng, B, L, Hkv) for _ in range(2)]
    x[0][0, 0, 0] = 0.0                                     # an all-zero row
    x[1][0, 0, 0] = np.arange(128) * 2.0 ** -24             # subnormal: its scale is 18 2^-24
    ties = np.concatenate([np.arange(-112, 113, 2) / 16.0, np.arange(15) / 32.0 + 0.5])
    x[1][-1, -1, -1] = ties[:128]                           # max 7: scale 1, every value on the grid or a tie
    x[1][-1, -1, -1, 0] = 7.0
    start = rng.integers(0, cap - L + 1, B).astype(np.int32)
    k_pl, v_pl = bn.nested_cache(cap, Hkv, B)
    for p in k_pl + v_pl:
        p.view(torch.uint8).fill_(0x5a)
    typed = [dev(t if src == "f16" else t.astype(np.float32)) for t in x]
    bn.kv_append(*typed, dev(start), k_pl, v_pl)
    for pl, t in zip((k_pl, v_pl), x):
        want = _packed(t)
        for got, w in zip(_np(pl), want):
            full = np.full(got.shape, 0x5a, np.uint8) if got.dtype == np.uint8 else np.full(got.shape, 0x5a5a, np.uint16).view(np.float16)
            for b in range(B):
                full[b, start[b]:start[b] + L] = w[b]
            assert np.array_equal(got.view(np.uint8), full.view(np.uint8))


def test_append_near_ties_bit_for_bit():
    """Values next to the rounding borders of both nibbles, over many scales."""
    rng = np.random.default_rng(3)
    n = 4000
    s = np.exp(rng.uniform(-9, 8, n)).astype(np.float16).astype(np.float64)
    t = rng.integers(-224, 225, (n, 128)) / 32.0  # every border of 1/16 steps and of whole steps
    x = t * s[:, None]
    x[:, 0] = 7.0 * s
    x = np.clip(x, -65504, 65504).astype(np.float16)
    nudge = rng.integers(-1, 2, x.shape)  # the neighbours in fp16
    x = np.where(nudge == 0, x, np.nextafter(x, np.where(nudge > 0, np.float16(65504), np.float16(-65504))))
    x[:, 0] = np.max(np.abs(x), axis=1)
    x = x.reshape(1, n, 1, 128)
    k_pl, v_pl = bn.nested_cache(n, 1, 1)
    bn.kv_append(dev(x), dev(-x), dev(np.zeros(1, np.int32)), k_pl, v_pl)
    for pl, t in ((k_pl, x), (v_pl, -x)):
        for got, w in zip(_np(pl), _packed(t)):
            assert np.array_equal(got.view(np.uint8), w.view(np.uint8))


def test_append_clamps_rows_of_subnormal_scale():
    """max = 10 2^-24: the scale rounds down to 2^-24, 10 steps are clamped to 7 and 7/16."""
    x = np.zeros((1, 1, 1, 128), np.float16)
    x[..., :3] = np.array([10, -10, 3]) * 2.0 ** -24
    k_pl, v_pl = bn.nested_cache(1, 1, 1)
    bn.kv_append(dev(x), dev(x), dev(np.zeros(1, np.int32)), k_pl, v_pl)
    want = np.zeros(128)
    want[:3] = np.array([7 + 7 / 16, -8.5, 3]) * 2.0 ** -24
    assert np.array_equal(ref.values(1, _np(k_pl))[0, 0, 0], want)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("src", ["f16", "f32"])
def test_append_turns_as_rope_does(rot, layout, src):
    """Keys turned and packed: bit for bit rope and pack_weights in two calls; values as they are."""
    rng = np.random.default_rng(rot)
    B, L, Hkv, cap = 3, 37, 4, 50
    kv = rng.standard_normal((B, L, 2 * Hkv + 3, 128)).astype(np.float32)  # columns of a wider array
    kv = dev(kv).to(DTYPE[src])
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:2 * Hkv]
    pos = dev(rng.integers(-5, 1 << 20, (B, L)).astype(np.int32))
    start = dev(np.array([0, 13, 7], np.int32))
    phases, mag = bn.rope_phases(rot, 5e5, bn.ROPE_YARN, 8.0, 1.0, 32.0, 4096)
    k_pl, v_pl = bn.nested_cache(cap, Hkv, B)
    bn.kv_append(k, v, start, k_pl, v_pl, pos, phases, mag, LAYOUT[layout])
    turned = bn.rope(k.flatten(0, 1), pos.flatten(), phases, mag, LAYOUT[layout])
    for pl, x in ((k_pl, turned), (v_pl, v.half())):
        want = bn.pack_weights(x.reshape(-1, 128).contiguous())
        for got, w in zip(pl, want):
            w = w.reshape(B, L, Hkv, *got.shape[3:])
            for b, s in enumerate(host(start)):
                assert torch.equal(got[b, s:s + L].contiguous().view(torch.uint8), w[b].contiguous().view(torch.uint8))


def test_append_leaves_what_is_outside():
    """Counts below L, rows before 0 and past cap, a full and an empty count."""
    rng = np.random.default_rng(4)
    B, L, Hkv, cap = 5, 6, 2, 8
    x = dev(_rows(rng, B, L, Hkv))
    start, count = [0, 6, -3, 2, 8], [3, 6, 6, 0, 6]
    k_pl, v_pl = bn.nested_cache(cap, Hkv, B)
    for p in k_pl + v_pl:
        p.view(torch.uint8).fill_(0x5a)
    bn.kv_append(x, x, dev(np.array(start, np.int32)), k_pl, v_pl, count=dev(np.array(count, np.int32)))
    want = _packed(host(x))
    for got, w in zip(_np(k_pl) + _np(v_pl), want + want):
        for b in range(B):
            for t in range(cap):
                i = t - start[b]
                if 0 <= i < min(L, count[b]):
                    assert np.array_equal(got[b, t], w[b, i])
                else:
                    assert np.all(got[b, t:t + 1].view(np.uint8) == 0x5a)


@pytest.mark.parametrize("mode", [0, 1])
def test_read_gives_the_rows_values(mode):
    rng = np.random.default_rng(6)
    B, L, Hkv, cap = 3, 5, 3, 9
    planes = [_packed(_rows(rng, B, cap, Hkv)) for _ in range(2)]
    d = [tuple(dev(p) for p in x) for x in planes]
    start = np.array([0, 7, -2], np.int32)
    got = bn.kv_read(mode, dev(start), L, *d)
    for g, x in zip(got, planes):
        want = np.zeros((B, L, Hkv, 128))
        full = ref.values(mode, x)
        for b in range(B):
            for i in range(L):
                if 0 <= start[b] + i < cap:
                    want[b, i] = full[b, start[b] + i]
        assert np.array_equal(host(g), want.astype(np.float16))  # exact in fp32, rounded once
    whole = bn.kv_read(mode, None, cap, *d)
    assert np.array_equal(host(whole[1]), ref.values(mode, planes[1]).astype(np.float16))


# --------------------------------------------------------------- attention
class Attend:
    """A batch over a prefix of P tokens and own caches of `cap`."""

    def __init__(self, B, L, H, Hkv, P, cap, lens, seed=0, qscale=1.0):
        rng = np.random.default_rng(seed + B * L + P + cap)
        self.shape = (B, L, H, Hkv, P, cap)
        self.q = (rng.standard_normal((B, L, H, 128)) * qscale).astype(np.float16)
        self.prefix = [_packed(_rows(rng, P, Hkv)), _packed(rng.standard_normal((P, Hkv, 128)).astype(np.float16))] if P else None
        self.own = [_packed(_rows(rng, B, cap, Hkv)), _packed(rng.standard_normal((B, cap, Hkv, 128)).astype(np.float16))] if cap else None
        self.lens = np.array(lens, np.int32)
        self.upload()

    def upload(self):
        up = lambda c: None if c is None else tuple(tuple(dev(p) for p in x) for x in c)  # noqa: E731
        self.d = (dev(self.q), up(self.prefix), up(self.own), dev(self.lens))

    def bounds(self, mode, lse, size, out):
        """A score is a sum of 128 products in fp32, each addition off by at most
        2^-23 of the sum of magnitudes (truncation), times a scale and a rounding
        or two: ds <= 2^-16 max sum |q k| / sqrt(128) + 2^-22 max |s|.  Each weight
        and their sum are off by ds and exp2's 2^-22, so out by 2 (ds + 2^-21)
        sum p |v|; each p v_scale is rounded to fp16 (h), and so is out."""
        k = np.abs(np.concatenate([ref.values(mode, c[0]).reshape(-1, 128) for c in (self.prefix, self.own) if c]))
        ds = 2.0 ** -16 * float((np.abs(self.q.astype(np.float64)).max(axis=(0, 1, 2)) * k.max(axis=0)).sum()) / np.sqrt(128)
        fin = np.where(np.isfinite(lse), lse, 0.0)
        ds += 2.0 ** -21 * (1 + np.abs(fin).max())
        return (2 * (ds + 2.0 ** -21) + HALF) * size + HALF * np.abs(out) + 2.0 ** -24, 2 * ds + 2.0 ** -20 * (1 + np.abs(fin))

    def check(self, mode, got):
        out, lse, size = ref.attention(mode, self.q, self.prefix, self.own, self.lens)
        tol, tol_lse = self.bounds(mode, lse, size, out)
        go, gl = host(got[0]).astype(np.float64), host(got[1]).astype(np.float64)
        live = self.lens >= 0
        fin = np.isfinite(lse[live])
        assert np.array_equal(fin, np.isfinite(gl[live])) and np.all(gl[live][~fin] == -np.inf)
        assert np.all(np.abs(go - out)[live] <= tol[live])
        assert np.all(np.abs(gl[live][fin] - lse[live][fin]) <= tol_lse[live][fin])
        return go, gl


CASES = [  # B, L, H, Hkv, P, cap, lens
    (1, 1, 1, 1, 0, 1, [1]),
    (1, 1, 1, 1, 1, 0, [0]),
    (2, 1, 32, 8, 100, 20, [20, 3]),
    (3, 4, 8, 2, 129, 70, [70, 4, 2]),             # fewer own tokens than queries
    (4, 3, 4, 4, 0, 33, [33, 1, 0, 2]),            # no prefix: rows that see nothing
    (5, 1, 8, 1, 257, 300, [300, 0, 16, 17, 299]),
    (9, 5, 16, 2, 1000, 40, [40, 39, 5, 4, 1, 0, 33, 16, 40]),  # 360 rows a KV head: odd row tiles
    (33, 4, 4, 1, 515, 9, [i % 10 for i in range(33)]),         # 528 rows
    (2, 7, 24, 3, 4111, 1025, [1025, 700]),
    (2, 40, 8, 2, 300, 260, [260, 41]),            # more own rows than a tile
    (64, 2, 8, 8, 64, 3, [3] * 64),
]


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:6])))
def test_prefix_attention_matches_oracle(case, mode):
    a = Attend(*case)
    a.check(mode, bn.prefix_attention(mode, *a.d))


@pytest.mark.parametrize("mode", [0, 1])
def test_prefix_attention_large_scores_and_scales(mode):
    """Scores of hundreds (a softmax that is one token), value scales over twelve
    powers of two from token to token, and all-zero rows."""
    a = Attend(3, 2, 8, 2, 700, 90, [90, 50, 7], qscale=30.0)
    rng = np.random.default_rng(1)
    for c in (a.prefix, a.own):
        sc = c[1][2]
        sc *= np.exp2(rng.integers(-6, 7, sc.shape)).astype(np.float16)
        sc.reshape(-1)[::11] = 0.0
    a.upload()
    a.check(mode, bn.prefix_attention(mode, *a.d))


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("case", [
    (65, 4, 8, 2, 5000, 20, [i % 21 for i in range(65)]),      # 1040 rows: the last 16 alone, runs across heads
    (96, 1, 8, 2, 9001, 3, [3] * 96),                          # 384 rows, the last 128 alone
    (128, 2, 4, 4, 4097, 5, [5, 0, 2, 1] * 32),                # 256 rows, one token in the last tile
    (70, 1, 8, 1, 33000, 2, [2] * 70)],                        # a long prefix, 560 rows
    ids=lambda c: "x".join(map(str, c[:6])))
def test_prefix_attention_of_many_rows_matches_oracle(case, mode):
    """Runs of several units, of 256 rows, from one KV head and row group into the next."""
    a = Attend(*case)
    a.check(mode, bn.prefix_attention(mode, *a.d))


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("B,L,H,Hkv,P", [(40, 2, 8, 2, 1500), (300, 2, 8, 4, 3000), (3, 1, 8, 2, 700)])
def test_prefix_attention_growing_scores_and_scales(B, L, H, Hkv, P, mode):
    """Key and value scales that double every 100 tokens: each row's maximum and
    the greatest value scale grow from tile to tile, so the output is rescaled
    again and again; some tokens' values are all zero."""
    a = Attend(B, L, H, Hkv, P, 40, [40, 17, 0][:B] + [9] * (B - 3), qscale=3.0)
    for c, n in ((a.prefix, P), (a.own, 40)):
        for kv in c:
            up = np.exp2(np.minimum(np.arange(n) // 100, 9) - 6.0)[:, None]
            kv[2][...] = (kv[2].astype(np.float64) * up).astype(np.float16)
        c[1][2].reshape(-1)[::13] = 0.0
    a.upload()
    a.check(mode, bn.prefix_attention(mode, *a.d))


@pytest.mark.parametrize("B,L,H,Hkv,P", [(40, 2, 8, 2, 1500), (300, 2, 8, 4, 3000), (3, 1, 8, 2, 700)])
def test_prefix_attention_shows_nan(B, L, H, Hkv, P):
    """A query with a NaN gives NaN in its own row and nowhere else."""
    a = Attend(B, L, H, Hkv, P, 40, [40, 17, 0][:B] + [9] * (B - 3))
    want = bn.prefix_attention(1, *a.d)
    q = a.d[0].clone()
    q[1, 0, 3, 77] = float("nan")
    got = bn.prefix_attention(1, q, *a.d[1:])
    row = torch.zeros(B, L, H, dtype=torch.bool, device="cuda")
    row[1, 0, 3] = True
    assert torch.all(got[0][row].isnan()) and torch.all(got[1][row].isnan())
    assert torch.equal(got[0][~row], want[0][~row]) and torch.equal(got[1][~row], want[1][~row])


@pytest.mark.parametrize("mode", [0, 1])
def test_prefix_attention_hidden_rows_may_hold_anything(mode):
    """Rows behind a sequence's length with NaN and infinite scales, scratch full
    of NaN: the same bits; a sequence of negative length keeps its outputs."""
    a = Attend(4, 2, 8, 2, 90, 50, [50, 20, 0, 33], seed=3)
    want = bn.prefix_attention(mode, *a.d)
    for pl in a.own:
        for b, n in enumerate(a.lens):
            pl[2][b, n:] = np.array([np.nan, np.inf, -np.inf])[np.arange(50 - n) % 3][:, None]
            pl[0][b, n:] = 0xff
    a.lens[2] = -1
    a.upload()
    out, lse = torch.full_like(want[0], 3.0), torch.full_like(want[1], 5.0)
    ws = torch.full((bn.prefix_attention_ws_bytes(4, 2, 8, 2, 90, 50),), 0xff, dtype=torch.uint8, device="cuda")
    bn.prefix_attention(mode, *a.d, out=out, lse=lse, ws=ws)
    live = [0, 1, 3]
    assert torch.equal(out[live], want[0][live]) and torch.equal(lse[live], want[1][live])
    assert torch.all(out[2] == 3.0) and torch.all(lse[2] == 5.0)


def test_prefix_attention_longer_than_the_cache_is_the_whole_cache():
    a = Attend(2, 1, 4, 1, 30, 12, [12, 12])
    want = bn.prefix_attention(1, *a.d)
    got = bn.prefix_attention(1, *a.d[:3], dev(np.array([400, 13], np.int32)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_prefix_attention_agrees_with_single_sequence_attention():
    """One sequence, one query, all tokens in the prefix: bitnest_nested_attention."""
    a = Attend(1, 1, 32, 8, 777, 0, [0])
    out, _ = bn.prefix_attention(1, *a.d)
    kp, vp = (tuple(t.reshape(-1, *t.shape[2:]) if t.dim() > 2 else t.reshape(-1, 1) for t in x) for x in a.d[1])
    want = bn.nested_attention(1, a.d[0][0, 0], kp, vp, 8)
    # that one is within 1e-3 (|exact| + 1e-3 rms) of the exact value; this one within
    # Attend.bounds, whose h sum p |v| for the weights' fp16 is not small beside an
    # output that cancels to nearly zero, as the layer's measure asks
    exact, lse, size = ref.attention(1, a.q, a.prefix, None, a.lens)
    tol = a.bounds(1, lse, size, exact)[0] + 1e-3 * (np.abs(exact) + 1e-3 * np.sqrt(np.mean(exact ** 2)))
    assert np.all(np.abs(host(out).astype(np.float64) - host(want)) <= tol)


# ----------------------------------------------------- weights and eviction
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("B,L,H,Hkv,cap,lens", [(1, 1, 1, 1, 1, [1]), (3, 4, 8, 2, 70, [70, 2, 0]),
                                                (2, 1, 32, 8, 515, [515, 300]), (4, 9, 8, 1, 33, [33, 9, 40, -1]),
                                                (20, 3, 4, 4, 257, None), (1, 1, 8, 1, 9, None),
                                                (33, 5, 16, 2, 1000, None)])
def test_weights_match_oracle(B, L, H, Hkv, cap, lens, mode):
    rng = np.random.default_rng(B + cap)
    a = Attend(B, L, H, Hkv, cap if lens is None else 0, 0 if lens is None else cap, [0] * B if lens is None else lens)
    k = (a.prefix if lens is None else a.own)[0]
    d_k = (a.d[1] if lens is None else a.d[2])[0]
    lse = (rng.standard_normal((B, L, H)) + 6.0).astype(np.float32)
    lse[0, 0, 0] = -np.inf  # a query that saw nothing
    acc = rng.random((Hkv, cap) if lens is None else (B, Hkv, cap)).astype(np.float32)
    n = None if lens is None else np.maximum(a.lens, 0)
    want = ref.weights(mode, a.q, lse, k, acc, n)
    d_acc = dev(acc)
    assert bn.kv_weights(mode, a.d[0], dev(lse), d_k, d_acc, None if lens is None else a.d[3]) is d_acc
    # each weight exp(s - lse) is off by ds (Attend.bounds) and roundings of s - lse
    # and exp2; the sum of R rows by R u of itself, and one more with acc
    tol = a.bounds(mode, lse.astype(np.float64), 0.0, 0.0)[1]
    rel = tol[np.isfinite(lse)].max() if np.isfinite(lse).any() else 0.0
    rel += (B * L * H // Hkv + 2) * U
    assert np.all(np.abs(host(d_acc) - want) <= rel * (want - acc) + 2 * U * np.abs(want))


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("B,L,H,Hkv,P", [
    (32, 1, 16, 4, 128),       # 128 rows, one row tile; fewer token tiles than SMs
    (129, 1, 4, 4, 6000),      # 129 rows; 188 token tiles: one or two a CTA, runs across heads
    (16, 4, 32, 8, 9001),      # 256 rows; 568 token tiles, three or four a CTA
    (65, 2, 16, 2, 19000),     # 1040 rows; 298 tiles
    (150, 1, 2, 2, 38000)])    # one head a KV head; 594 tiles, four or five a CTA
def test_weights_of_many_rows_match_oracle(B, L, H, Hkv, P, mode):
    """The shared prefix's weights where a KV head has 128 rows or more, over the
    ways in which token tiles are dealt out; a few rows without weight."""
    rng = np.random.default_rng(P)
    q = (rng.standard_normal((B, L, H, 128)) * 1.2).astype(np.float16)
    k = tuple(rng.integers(0, 256, (P, Hkv, 64)).astype(np.uint8) for _ in range(2)) + (
        (rng.random((P, Hkv)) * 0.2).astype(np.float16),)
    lse = (rng.standard_normal((B, L, H)) + 20.0).astype(np.float32)
    lse[0, 0, 0] = lse[B // 2, 0, H - 1] = lse[B - 1, L - 1, H - 1] = -np.inf
    acc = rng.random((Hkv, P)).astype(np.float32)
    want = ref.weights(mode, q, lse, k, acc, None)
    got = host(bn.kv_weights(mode, dev(q), dev(lse), tuple(dev(x) for x in k), dev(acc)))
    # as in Attend.bounds and test_weights_match_oracle
    kv = np.abs(ref.values(mode, k).reshape(-1, 128)).max(0)
    ds = 2.0 ** -16 * float((np.abs(q.astype(np.float64)).max(axis=(0, 1, 2)) * kv).sum()) / np.sqrt(128)
    ds += 2.0 ** -21 * (1 + np.abs(lse[np.isfinite(lse)]).max())
    rel = 2 * ds + 2.0 ** -20 * (1 + np.abs(lse[np.isfinite(lse)]).max()) + (B * L * H // Hkv + 2) * U
    assert np.all(np.abs(got - want) <= rel * (want - acc) + 2 * U * np.abs(want))


def test_weights_of_a_softmax_sum_to_one():
    """Prefix and own weights with the attention's own lse: one for each row."""
    B, L, H, Hkv = 4, 3, 8, 2
    a = Attend(B, L, H, Hkv, 300, 60, [60, 3, 20, 0])
    _, lse = bn.prefix_attention(1, *a.d)
    shared = bn.kv_weights(1, a.d[0], lse, a.d[1][0], torch.zeros(Hkv, 300, device="cuda"))
    own = bn.kv_weights(1, a.d[0], lse, a.d[2][0], torch.zeros(B, Hkv, 60, device="cuda"), a.d[3])
    total = host(shared).astype(np.float64).sum(1) + host(own).astype(np.float64).sum((0, 2))
    rows = B * L * H // Hkv
    tol = a.bounds(1, host(lse).astype(np.float64), 0.0, 0.0)[1].max()
    assert np.all(np.abs(total - rows) <= 2 * rows * (tol + (rows + 2) * U))


@pytest.mark.parametrize("B,Hkv,cap,keep,sinks,recent,lens", [
    (1, 1, 1, 1, 0, 0, [1]), (2, 2, 50, 20, 4, 8, [50, 21]), (3, 3, 40, 40, 1, 1, [40, 39, 0]),
    (2, 8, 5000, 1000, 4, 200, [5000, 999]), (2, 1, 2500, 1, 0, 0, [2500, 1]),
    (2, 2, 300, 64, 64, 0, [300, 64]), (2, 2, 300, 64, 0, 64, [300, 65]), (2, 1, 1030, 1025, 0, 0, [1030, -1])])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict_matches_oracle(B, Hkv, cap, keep, sinks, recent, lens, kind):
    rng = np.random.default_rng(cap + keep)
    acc = np.exp(3 * rng.standard_normal((B, Hkv, cap))).astype(np.float32)
    if kind == "ties":
        acc = rng.integers(0, 3, acc.shape).astype(np.float32)
    elif kind == "odd":
        acc = rng.choice(np.array([0.0, -0.0, -1.0, np.nan, np.inf, -np.inf, 1e-45, 1.0], np.float32), acc.shape)
    pl = [[rng.integers(0, 256, (B, cap, Hkv, 64)).astype(np.uint8) for _ in range(2)]
          + [rng.integers(0, 1 << 16, (B, cap, Hkv)).astype(np.uint16).view(np.float16)] for _ in range(2)]
    d = [tuple(dev(p) for p in x) for x in pl]
    cap_out = keep + 3
    out = bn.nested_cache(cap_out, Hkv, B)
    for p in out[0] + out[1]:
        p.view(torch.uint8).fill_(0x5a)
    acc_out = torch.full((B, Hkv, cap_out), 9.0, device="cuda")
    kept, n = bn.kv_evict(dev(acc), dev(np.array(lens, np.int32)), keep, sinks, recent, *d, *out, acc_out)
    kept, n, acc_out = host(kept), host(n), host(acc_out)
    got = [_np(x) for x in out]
    for b in range(B):
        assert n[b] == min(lens[b], keep)
        for j in range(Hkv):
            if lens[b] < 0:
                assert np.all(kept[b, j] == -1) and np.all(acc_out[b, j] == 9.0)
                continue
            want = ref.evict(acc[b, j], lens[b], keep, sinks, recent)
            assert kept[b, j].tolist() == want + [-1] * (keep - len(want))
            assert np.array_equal(acc_out[b, j, :len(want)].view(np.uint32), acc[b, j, want].view(np.uint32))
            assert np.all(acc_out[b, j, len(want):] == 0.0)
            for x, y in zip(pl, got):
                for p, q in zip(x, y):
                    assert np.array_equal(q[b, :len(want), j].copy().view(np.uint8), p[b, want, j].copy().view(np.uint8))
                    assert np.all(q[b, len(want):, j].copy().view(np.uint8) == 0x5a)


# ----------------------------------------------------------- calls together
def test_serving_run():
    """A prompt into the shared prefix, then verify passes of a batch: queries
    turned, keys and values appended, attention, weights, eviction when the
    caches fill; each attention against the oracle on the caches as they are,
    each eviction against the oracle's choice."""
    rng = np.random.default_rng(11)
    B, L, H, Hkv, P, cap, keep = 3, 4, 8, 2, 150, 24, 12
    phases, mag = bn.rope_phases(128, 5e5)
    prefix = bn.nested_cache(P, Hkv, 1)
    kv = dev(rng.standard_normal((1, P, 2 * Hkv, 128)).astype(np.float32))
    bn.kv_append(kv[:, :, :Hkv], kv[:, :, Hkv:], dev(np.zeros(1, np.int32)), *prefix,
                 pos=torch.arange(P, dtype=torch.int32, device="cuda")[None], phases=phases)
    prefix = tuple(tuple(t[0] for t in x) for x in prefix)
    own, spare = bn.nested_cache(cap, Hkv, B), bn.nested_cache(cap, Hkv, B)
    acc, acc2 = (torch.zeros(B, Hkv, cap, device="cuda") for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    pos0, evictions = P, 0
    for step in range(9):
        qkv = dev(rng.standard_normal((B * L, (H + 2 * Hkv) * 128)).astype(np.float32))  # the layer's fp32 output
        heads = qkv.view(B * L, H + 2 * Hkv, 128)
        pos = (pos0 + torch.arange(L, dtype=torch.int32, device="cuda")).repeat(B, 1).contiguous()
        q = bn.rope(heads[:, :H], pos.flatten(), phases, mag).view(B, L, H, 128)
        if int(lens.max()) + L > cap:
            before, n0 = host(acc), host(lens)
            kept, new = bn.kv_evict(acc, lens, keep, 2, 4, *own, *spare, acc2)
            for b in range(B):
                for j in range(Hkv):
                    want = ref.evict(before[b, j], int(n0[b]), keep, 2, 4)
                    assert host(kept)[b, j, :len(want)].tolist() == want
            own, spare, acc, acc2, lens = spare, own, acc2, acc, new
            evictions += 1
        kv = heads.view(B, L, H + 2 * Hkv, 128)
        bn.kv_append(kv[:, :, H:H + Hkv], kv[:, :, H + Hkv:], lens, *own, pos=pos, phases=phases, magnitude=mag)
        lens = lens + L
        got = bn.prefix_attention(bn.TARGET, q, prefix, own, lens)
        a = Attend.__new__(Attend)
        a.q, a.lens = host(q), host(lens)
        a.prefix, a.own = [_np(x) for x in prefix], [_np(x) for x in own]
        a.check(1, got)
        old = host(acc)
        bn.kv_weights(bn.TARGET, q, got[1], own[0], acc, lens)
        want = ref.weights(1, a.q, host(got[1]), a.own[0], old, a.lens)
        rel = a.bounds(1, host(got[1]).astype(np.float64), 0.0, 0.0)[1].max() + 20 * U
        assert np.all(np.abs(host(acc) - want) <= rel * (want - old) + 2 * U * np.abs(want))
        pos0 += L
    assert evictions >= 1


def _step(a, mode, phases, pos, x, planes, acc, out_cache, acc_out):
    q = bn.rope(x.flatten(0, 1), pos.flatten(), phases).view(x.shape)
    bn.kv_append(x[:, :, :planes[0][0].shape[2]], x[:, :, :planes[0][0].shape[2]], a.d[3], *planes, pos=pos, phases=phases)
    out, lse = bn.prefix_attention(mode, q, a.d[1], planes, a.d[3] + x.shape[1])
    bn.kv_weights(mode, q, lse, planes[0], acc, a.d[3] + x.shape[1])
    kept, n = bn.kv_evict(acc, a.d[3] + x.shape[1], 10, 1, 2, *planes, *out_cache, acc_out)
    return out, lse, kept, n


def test_captured_and_on_another_stream():
    """A step on a side stream, and captured in a graph and replayed on new
    inputs: the same bits as on the default stream."""
    B, L, H, Hkv, P, cap = 3, 2, 8, 2, 200, 40
    a = Attend(B, L, H, Hkv, P, cap, [30, 0, 13])
    phases, _ = bn.rope_phases(128, 1e4)
    pos = (a.d[3][:, None] + torch.arange(L, dtype=torch.int32, device="cuda")).contiguous()
    rng = np.random.default_rng(0)
    xs = [dev(rng.standard_normal((B, L, H, 128)).astype(np.float32)) for _ in range(3)]

    def state():
        return (tuple(tuple(t.clone() for t in pl) for pl in a.d[2]), torch.zeros(B, Hkv, cap, device="cuda"),
                bn.nested_cache(16, Hkv, B), torch.zeros(B, Hkv, 16, device="cuda"))

    def flat(r, st):
        return [*r, *st[0][0], *st[0][1], st[1], *st[2][0], *st[2][1], st[3]]

    want = []
    for x in xs:
        st = state()
        want.append([t.clone() for t in flat(_step(a, 1, phases, pos, x, *st), st)])
    side = torch.cuda.Stream()
    for x, w in zip(xs, want):
        st = state()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = flat(_step(a, 1, phases, pos, x, *st), st)
        side.synchronize()
        assert all(torch.equal(g.view(torch.uint8) if g.is_floating_point() else g,
                               t.view(torch.uint8) if t.is_floating_point() else t) for g, t in zip(got, w))
    st, x = state(), xs[0].clone()
    fresh = state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = _step(a, 1, phases, pos, x, *st)
    for new, w in zip(xs, want):
        for old, t in zip(flat((), st), flat((), fresh)):
            old.copy_(t)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g.view(torch.uint8) if g.is_floating_point() else g,
                               t.view(torch.uint8) if t.is_floating_point() else t)
                   for g, t in zip(flat(r, st), w))


def test_captured_attention_and_weights_of_many_rows():
    """The tcgen05 kernels, own tokens beside them, captured once and replayed on
    new inputs, and on a side stream: the same bits as on the default stream."""
    cases = [Attend(70, 2, 8, 2, 6000, 50, [(7 * i + s) % 51 for i in range(70)], seed=s) for s in range(3)]

    def step(q, prefix, own, lens, acc):
        out, lse = bn.prefix_attention(1, q, prefix, own, lens)
        bn.kv_weights(1, q, lse, prefix[0], acc)
        return out, lse

    want = []
    for a in cases:
        acc = torch.zeros(2, 6000, device="cuda")
        want.append((*step(*a.d, acc), acc))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, w in zip(cases, want):
            acc = torch.zeros(2, 6000, device="cuda")
            got = (*step(*a.d, acc), acc)
            side.synchronize()
            assert all(torch.equal(g, t) for g, t in zip(got, w))
    flat = lambda d: [d[0], *(t for c in d[1:3] for pl in c for t in pl), d[3]]  # noqa: E731
    held = Attend(70, 2, 8, 2, 6000, 50, [0] * 70, seed=9)
    acc = torch.zeros(2, 6000, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        acc.zero_()
        r = step(*held.d, acc)
    for a, w in zip(cases, want):
        for old, new in zip(flat(held.d), flat(a.d)):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, t) for g, t in zip((*r, acc), w))


@pytest.mark.parametrize("mode", [0, 1])
def test_weights_of_many_own_rows(mode):
    """More than 128 rows of one sequence's KV head."""
    a = Attend(3, 40, 8, 2, 0, 300, [300, 41, 7])
    lse = (np.random.default_rng(1).standard_normal((3, 40, 8)) + 6.0).astype(np.float32)
    acc = torch.zeros(3, 2, 300, device="cuda")
    got = host(bn.kv_weights(mode, a.d[0], dev(lse), a.d[2][0], acc, a.d[3]))
    want = ref.weights(mode, a.q, lse, a.own[0], np.zeros((3, 2, 300)), a.lens)
    rel = a.bounds(mode, lse.astype(np.float64), 0.0, 0.0)[1].max() + (160 + 2) * U
    assert np.all(np.abs(got - want) <= rel * want)


def test_attention_of_nothing():
    """A prefix of no tokens and an empty cache: zeros and -inf."""
    q = torch.randn(2, 1, 4, 128, device="cuda").half()
    own = bn.nested_cache(0, 2, 2)
    out, lse = bn.prefix_attention(1, q, bn.nested_cache(0, 2), own, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert torch.all(out == 0) and torch.all(lse == -torch.inf)


def test_two_calls_at_once():
    """Two attentions at the same time on two streams, each with scratch of its own."""
    cases = [Attend(8, 4, 16, 2, 2000, 100, [i * 12 for i in range(8)], seed=s) for s in range(2)]
    want = [bn.prefix_attention(1, *a.d) for a in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(10):
        for i, (a, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(bn.prefix_attention(1, *a.d))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for r in g:
            assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])


def test_cache_past_32_bits():
    """A cache whose byte offsets pass 2^32: its last rows are appended, read,
    attended, weighed and kept."""
    Hkv, cap, B = 8, 4_300_000, 2  # 2 * 4.3e6 * 8 * 64 bytes = 4.4e9 a plane
    planes = tuple((torch.zeros((B, cap, Hkv, 64), dtype=torch.uint8, device="cuda"),) * 2
                   + (torch.zeros((B, cap, Hkv), dtype=torch.float16, device="cuda"),) for _ in range(2))
    planes = tuple((p[0], torch.zeros_like(p[0]), p[2]) for p in planes)
    rng = np.random.default_rng(9)
    x = _rows(rng, B, 5, Hkv)
    start = dev(np.array([0, cap - 5], np.int32))
    bn.kv_append(dev(x), dev(x), start, *planes)
    k, v = bn.kv_read(1, start, 5, *planes)
    want = ref.values(1, _packed(x)).astype(np.float16)
    assert np.array_equal(host(k), want) and np.array_equal(host(v), want)
    # the zero rows before them are 4.3e6 equal weights: attention of the last sequence is
    # sum_t e^{s_t} v_t / (n + sum e^{s_t}), the first's is its five rows alone
    q = (rng.standard_normal((B, 1, Hkv, 128)) * 2).astype(np.float16)
    lens = dev(np.array([5, cap], np.int32))
    out, lse = bn.prefix_attention(1, dev(q), None, planes, lens)
    s = np.einsum("bhd,bthd->bht", q[:, 0].astype(np.float64), ref.values(1, _packed(x))) / np.sqrt(128)
    total = np.exp(s).sum(-1) + np.array([0, cap - 5])[:, None]
    o = np.einsum("bht,bthd->bhd", np.exp(s) / total[..., None], ref.values(1, _packed(x)))
    # the sum over 4.3e6 tokens: in each lane's running sum at most 4.3e6 / 64 additions of u;
    # scores and roundings as in Attend.bounds, below 1e-3 here
    assert np.all(np.abs(host(lse)[:, 0] - np.log(total)) <= 1e-3 + 4.3e6 / 64 * U)
    # out: the last sequence's values are below 2^-14, where fp16 steps by 2^-24
    assert np.all(np.abs(host(out)[:, 0] - o) <= 8e-3 * np.abs(o).max(-1, keepdims=True) + 2.0 ** -25)
    acc = torch.zeros(B, Hkv, cap, device="cuda")
    bn.kv_weights(1, dev(q), lse, planes[0], acc, lens)
    w = np.exp(s - host(lse)[:, 0].astype(np.float64)[..., None])
    assert np.all(np.abs(host(acc[1, :, -5:]) - w[1]) <= 1e-3 * w[1])
    small = bn.nested_cache(9, Hkv, B)
    kept, n = bn.kv_evict(acc, lens, 9, 4, 5, *planes, *small, torch.zeros(B, Hkv, 9, device="cuda"))
    assert host(kept)[1, 3].tolist() == [0, 1, 2, 3] + list(range(cap - 5, cap)) and host(n).tolist() == [5, 9]
    assert np.array_equal(host(small[1][0])[1, 4:], host(planes[1][0][1, -5:]))
