"""GPU: the serving calls at the borders of their kernels: alignments, runs that
end inside a row group, long caches, rounding, and no bounded wait that gives up.
The checks and their bounds are test_gpu_serving's."""
import os
import subprocess
import sys

import numpy as np
import pytest

import w8_quantized_linear_b200 as bn
from oracle import serving as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import test_gpu_serving  # noqa: E402
from test_gpu_parity import dev, host  # noqa: E402
from test_gpu_serving import Attend  # noqa: E402


@pytest.fixture(autouse=True)
def _no_wait_timeouts():
    bn.device_wait_timeout(reset=True)
    yield
    torch.cuda.synchronize()
    assert bn.device_wait_timeout(reset=True) == 0


# ------------------------------------------------------------------ rotary
@pytest.mark.parametrize("layout", [bn.ROPE_HALF, bn.ROPE_PAIRS])
@pytest.mark.parametrize("src,dst", [("f16", "f16"), ("f16", "f32"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("D,rot", [(128, 64), (80, 32), (128, 8), (24, 16), (96, 96)])
def test_rope_at_any_element(D, rot, src, dst, layout):
    """x and y at any element of a wider array, heads that turn in part: only the
    element type's alignment is asked for.  The same bits as from an aligned array,
    which test_gpu_serving holds against the oracle; what lies beside stays."""
    types = {"f16": torch.float16, "f32": torch.float32}
    M, heads = 5, 3
    rng = np.random.default_rng(D + rot)
    row = heads * D + 16
    base = dev(rng.standard_normal((M, row)).astype(np.float32)).to(types[src])
    pos = dev(rng.integers(0, 9000, M).astype(np.int32))
    phases, mag = bn.rope_phases(rot, 1e4)

    def view(wide, first):
        return wide[:, first:first + heads * D].unflatten(1, (heads, D))

    for first in (0, 1, 2, 4, 6, 8, 12):
        x = view(base, first)
        want = bn.rope(x.contiguous(), pos, phases, mag, layout, dtype=types[dst])
        assert torch.equal(bn.rope(x, pos, phases, mag, layout, dtype=types[dst]), want)
        for to in (0, 1, 2, 4, 6):
            wide = torch.full((M, row), 7.0, dtype=types[dst], device="cuda")
            bn.rope(x, pos, phases, mag, layout, out=view(wide, to))
            assert torch.equal(view(wide, to), want)
            assert torch.all(wide[:, :to] == 7.0) and torch.all(wide[:, to + heads * D:] == 7.0)
        if src == dst:
            wide = base.clone()
            bn.rope(view(wide, first), pos, phases, mag, layout, out=view(wide, first))
            assert torch.equal(view(wide, first), want)
            assert torch.equal(wide[:, :first], base[:, :first])
            assert torch.equal(wide[:, first + heads * D:], base[:, first + heads * D:])


@pytest.mark.parametrize("layout", [bn.ROPE_HALF, bn.ROPE_PAIRS])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (80, 40)])
def test_rope_in_place_of_many_tokens(D, rot, dtype, layout):
    """Several heads a thread, x and y the same array: the bits of another array."""
    M, heads = 3001, 32
    x = torch.randn((M, heads, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(dtype)
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    phases, mag = bn.rope_phases(rot, 1e4)
    want = bn.rope(x, pos, phases, mag, layout, dtype=dtype)
    assert bn.rope(x, pos, phases, mag, layout, out=x) is x
    assert torch.equal(x, want)


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("B,L,H,Hkv,P", [
    (65, 4, 32, 8, 130),    # 5 row groups a head (the last of 16 rows), two token tiles each
    (128, 2, 64, 8, 100),   # one token tile a row group: a group begins as the one before ends
    (33, 4, 32, 8, 1290)])  # runs of 6: from one row group into the next at any tile
def test_prefix_attention_of_many_row_groups(B, L, H, Hkv, P, mode):
    """Several row groups a CTA, each of one or a few token tiles: what a group's
    last product leaves is complete before it is read, call after call."""
    a = Attend(B, L, H, Hkv, P, 3, [i % 4 for i in range(B)])
    first = bn.prefix_attention(mode, *a.d)
    a.check(mode, first)
    for _ in range(50):
        got = bn.prefix_attention(mode, *a.d)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("B,L,H,Hkv,P,cap", [
    (1, 2, 8, 1, 700, 0), (2, 2, 8, 1, 700, 0), (8, 1, 8, 1, 700, 0),  # eight, four and two warps a row
    (8, 2, 8, 1, 900, 0), (8, 2, 8, 1, 0, 900)])                       # one; own tokens: eight
def test_prefix_attention_joins_a_ctas_warps(B, L, H, Hkv, P, cap, mode):
    """The states of a CTA's warps that share rows, call after call."""
    a = Attend(B, L, H, Hkv, P, cap, [cap - 100 * i * (cap > 0) for i in range(B)])
    first = bn.prefix_attention(mode, *a.d)
    a.check(mode, first)
    for _ in range(50):
        got = bn.prefix_attention(mode, *a.d)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def _two_kinds(c):
    """Tokens of two kinds in turn: the first's score is q k = c / sqrt(128) above
    the second's, their values are 4 and -7 (all codes are the draft's and the
    target's alike)."""
    B, L, H, Hkv, P, cap = c.shape
    q = np.zeros((B, L, H, 128), np.float16)
    # the second kind's weight e^-x is just above 4 / 7, so outputs nearly cancel, and as
    # far from a value of 11 bits as one can be there
    x = np.arange(5.0, 7.5, 2.0 ** -8).astype(np.float16).astype(np.float64)
    w = np.exp(-x / np.sqrt(128.0))
    off = np.abs(w.astype(np.float16).astype(np.float64) / w - 1)
    off[np.abs(7 * w - 4) > 0.1] = 0.0
    assert off.max() > 0.8 * 2.0 ** -11
    q[..., 0] = x[off.argmax()]
    c.q = q
    first = np.arange(max(P, cap)) % 2 == 0

    def planes(n, rows, value):
        hi = np.full((n, 64), 0x88, np.uint8)
        hi[:] = value(first[:n])
        hi = np.broadcast_to(hi.reshape((1,) * (len(rows) - 2) + (n, 1, 64)), (*rows, 64)).copy()
        return hi, np.full_like(hi, 0x88), np.ones(rows, np.float16)

    def key(f):
        out = np.full((len(f), 64), 0x88, np.uint8)
        out[:, 0] = np.where(f, 0x89, 0x88)  # 1 or 0 in column 0
        return out

    def val(f):
        return np.where(f, 0xcc, 0x11).astype(np.uint8)[:, None]

    c.prefix = [planes(P, (P, Hkv), key), planes(P, (P, Hkv), val)] if P else None
    c.own = [planes(cap, (B, cap, Hkv), key), planes(cap, (B, cap, Hkv), val)] if cap else None
    c.upload()
    return c


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("shape", [(64, 1, 8, 1, 512, 0), (1, 1, 8, 1, 512, 0), (2, 1, 8, 1, 512, 0),
                                   (2, 4, 8, 1, 0, 512), (1, 2, 4, 1, 0, 512)],
                         ids=lambda c: "x".join(map(str, c)))
def test_prefix_attention_keeps_the_weights_bits(shape, mode):
    """Outputs that nearly cancel show what the weights p v_scale lose on their way
    into the product: 2^-11 of them would be 2^-12 of sum p |v| here."""
    a = _two_kinds(Attend(*shape, [shape[5]] * shape[0]))
    out, _, size = ref.attention(mode, a.q, a.prefix, a.own, a.lens)
    got = host(bn.prefix_attention(mode, *a.d)[0]).astype(np.float64)
    # scores below 1: their roundings and exp2's are below 2^-20 of a weight, two fp16
    # terms hold it to 2^-22; up to 512 additions off by 2^-23 of the sum of magnitudes;
    # parts join with a few roundings more; the output's own rounding
    tol = (512 * 2.0 ** -23 + 2.0 ** -18) * size + 2.0 ** -11 * np.abs(out) + 2.0 ** -25
    assert np.all(2.0 ** -12.6 * size > 2 * (tol - 2.0 ** -11 * np.abs(out)))  # the loss would show
    assert np.all(np.abs(got - out) <= tol)


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("shape", [(64, 1, 8, 1, 700, 0), (1, 1, 8, 1, 700, 0), (2, 4, 8, 1, 0, 700)],
                         ids=lambda c: "x".join(map(str, c)))
def test_prefix_attention_of_the_greatest_scores(shape, mode):
    """Scores just below 2^22, where fp32 steps by 1/4 and 1/2: finite outputs, to
    which only the tokens of the greatest score add."""
    B, L, H, Hkv, P, cap = shape
    a = Attend(*shape, [cap] * B)
    rng = np.random.default_rng(0)
    n = P or cap
    a.q = np.zeros((B, L, H, 128), np.float16)
    a.q[..., 0] = 60000.0
    rows = (P, Hkv) if P else (B, cap, Hkv)
    code = rng.integers(1, 8, n)
    code[[0, n // 2]] = 7
    hi = np.full((n, 64), 0x88, np.uint8)
    hi[:, 0] = 0x80 | (8 + code)
    hi = np.broadcast_to(hi.reshape((1,) * (len(rows) - 2) + (n, 1, 64)), (*rows, 64)).copy()
    scale = np.float16(112.5)  # 60000 * 7 * 112.5 / sqrt(128) = 4.18e6
    k = hi, np.full_like(hi, 0x88), np.full(rows, scale, np.float16)
    if P:
        a.prefix[0] = k
    else:
        a.own[0] = k
    a.upload()
    out, lse, size = ref.attention(mode, a.q, a.prefix, a.own, a.lens)
    assert 2.0 ** 21.9 < lse.max() < 2.0 ** 22
    got = bn.prefix_attention(mode, *a.d)
    # Equal scores have equal roundings and the next is 6e5 below, so within a part of the
    # tokens weights are exact but for their two terms' 2^-22 and a few roundings.  Parts
    # join by their lse in fp32 (log 2): half a step is 2^-24 of it, so a part's weight is
    # off by a factor of at most exp(2^-24 lse), two parts' ratio by its square (1.65 here).
    # lse: three roundings of the score.
    part = np.expm1(2 * 2.0 ** -24 * lse)[..., None]
    assert np.all(np.abs(host(got[0]).astype(np.float64) - out)
                  <= (part + 2.0 ** -18) * size + 2.0 ** -11 * np.abs(out) + 2.0 ** -25)
    assert np.all(np.abs(host(got[1]) - lse) <= 2.0 ** -21 * np.abs(lse))


def test_lengths_past_the_cache_count_as_the_whole_cache():
    """Several queries a sequence: attention, weights and eviction alike."""
    B, L, H, Hkv, cap = 2, 3, 8, 2, 20
    a = Attend(B, L, H, Hkv, 30, cap, [cap, cap])
    longer = dev(np.array([cap + 5, 2 ** 31 - 1], np.int32))
    want = bn.prefix_attention(1, *a.d)
    got = bn.prefix_attention(1, *a.d[:3], longer)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    acc = [bn.kv_weights(1, a.d[0], want[1], a.d[2][0], torch.zeros(B, Hkv, cap, device="cuda"), n)
           for n in (a.d[3], longer)]
    assert torch.equal(*acc)
    kept = [bn.kv_evict(acc[0], n, 7, 2, 2, *a.d[2], *bn.nested_cache(7, Hkv, B),
                        torch.zeros(B, Hkv, 7, device="cuda")) for n in (a.d[3], longer)]
    assert torch.equal(kept[0][0], kept[1][0]) and torch.equal(kept[0][1], kept[1][1])


# ----------------------------------------------------------------- weights
def _check_weights(mode, q, lse, k, acc, lens, got):
    """test_gpu_serving's bound: each weight off by the score's error and roundings
    of s - lse and exp2, the sum of R rows by R u of itself."""
    want = ref.weights(mode, q, lse, k, acc, lens)
    kv = np.abs(ref.values(mode, k).reshape(-1, 128)).max(0)
    ds = 2.0 ** -16 * float((np.abs(q.astype(np.float64)).max(axis=(0, 1, 2)) * kv).sum()) / np.sqrt(128)
    size = 1 + np.abs(lse[np.isfinite(lse)]).max()
    ds += 2.0 ** -21 * size
    B, L, H, _ = q.shape
    rel = 2 * ds + 2.0 ** -20 * size + (B * L * H // k[0].shape[-2] + 2) * 2.0 ** -24
    assert np.all(np.abs(got - want) <= rel * (want - acc) + 2.0 ** -23 * np.abs(want))


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("B,L,H,Hkv,P", [
    (224, 4, 8, 8, 2400),   # 7 row tiles; 152 token tiles, 19 a head: runs of one and two, across heads
    (100, 1, 64, 8, 5003),  # 7 row tiles; 320 token tiles, 40 a head: two or three a CTA
    (170, 1, 64, 8, 4800),  # 11 row tiles; 304 token tiles, 38 a head
    (48, 1, 64, 8, 9600)])  # 3 row tiles: one slot is left out of segments of one tile
def test_weights_of_odd_row_tiles(B, L, H, Hkv, P, mode):
    """Row tiles that leave a slot out at a segment's end, segments of one token
    tile in a row: each row's lse is there until the last slot has read it."""
    rng = np.random.default_rng(P)
    q = (rng.standard_normal((B, L, H, 128)) * 1.2).astype(np.float16)
    k = tuple(rng.integers(0, 256, (P, Hkv, 64)).astype(np.uint8) for _ in range(2)) + (
        (rng.random((P, Hkv)) * 0.2).astype(np.float16),)
    lse = (rng.standard_normal((B, L, H)) + 20.0).astype(np.float32)
    acc = rng.random((Hkv, P)).astype(np.float32)
    d = dev(q), dev(lse), tuple(dev(x) for x in k)
    first = bn.kv_weights(mode, *d, dev(acc))
    _check_weights(mode, q, lse, k, acc, None, host(first))
    for _ in range(20):
        assert torch.equal(bn.kv_weights(mode, *d, dev(acc)), first)


# ---------------------------------------------------------------- eviction
@pytest.mark.parametrize("B,Hkv,cap,keep,sinks,recent,lens", [
    (2, 2, 8193, 4000, 4, 64, [8193, 8000]),            # rows of 8 spans, held
    (2, 2, 32768, 18000, 4, 1024, [32768, 20001]),      # ... all of them full
    (2, 2, 32769, 18000, 0, 0, [32769, 32768]),         # two chunks, the second of one token
    (1, 2, 70001, 10000, 4, 100, [70001]),              # three chunks, the choice in the top third
    (2, 2, 70001, 38500, 4, 100, [70001, 65537]),       # of three weights: ties run out in the second chunk
    (1, 2, 70001, 45800, 4, 100, [70001]),              # ... in the third
    (1, 1, 70001, 66000, 0, 0, [70001])])               # ... among the least
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict_of_long_rows_matches_oracle(B, Hkv, cap, keep, sinks, recent, lens, kind):
    """Rows of one chunk that stay in registers, and of several that are read again
    in each round, with ties carried from chunk to chunk; row addresses that are
    not 16-byte aligned."""
    test_gpu_serving.test_evict_matches_oracle(B, Hkv, cap, keep, sinks, recent, lens, kind)


def test_evict_ties_run_out_in_each_chunk():
    """Equal weights but for a few: the first of them are kept, up to any place."""
    n, rng = 70001, np.random.default_rng(0)
    acc = np.full((1, 1, n), 2.0, np.float32)
    acc[0, 0, rng.integers(0, n, 500)] = 3.0
    acc[0, 0, rng.integers(0, n, 500)] = 1.0
    src, lens = bn.nested_cache(n, 1, 1), dev(np.array([n], np.int32))
    for keep in (700, 32000, 33000, 65400, 66100, 69900):
        kept, _ = bn.kv_evict(dev(acc), lens, keep, 2, 3, *src, *bn.nested_cache(keep, 1, 1),
                              torch.zeros(1, 1, keep, device="cuda"))
        assert host(kept)[0, 0].tolist() == ref.evict(acc[0, 0], n, keep, 2, 3)


# ----------------------------------------------------------------- capture
_FIRST = """
import torch, w8_quantized_linear_b200 as bn
B, L, H, Hkv, P, cap = 70, 2, 8, 2, 3000, 40
d = dict(device="cuda")
x = torch.randn(B * L, H + 2 * Hkv, 128, **d)
pos = torch.arange(B * L, dtype=torch.int32, **d)
phases, mag = bn.rope_phases(128, 1e4)
prefix, own, out = bn.nested_cache(P, Hkv), bn.nested_cache(cap, Hkv, B), bn.nested_cache(16, Hkv, B)
fill = torch.randn(1, P, 2 * Hkv, 128, **d)
zero, lens = torch.zeros(B, dtype=torch.int32, **d), torch.full((B,), 30, dtype=torch.int32, **d)
accs = lambda: (torch.zeros(Hkv, P, **d), torch.zeros(B, Hkv, cap, **d), torch.zeros(B, Hkv, 16, **d))
acc = accs()

def step():
    q = bn.rope(x[:, :H], pos, phases, mag).view(B, L, H, 128)
    kv = x.view(B, L, -1, 128)
    bn.kv_append(kv[:, :, H:H + Hkv], kv[:, :, H + Hkv:], zero, *own, pos=pos.view(B, L), phases=phases)
    one = tuple(tuple(t[None] for t in c) for c in prefix)
    bn.kv_append(fill[:, :, :Hkv], fill[:, :, Hkv:], zero[:1], *one)
    o, lse = bn.prefix_attention(bn.TARGET, q, prefix, own, lens)
    bn.kv_weights(bn.TARGET, q, lse, prefix[0], acc[0])
    bn.kv_weights(bn.TARGET, q, lse, own[0], acc[1], lens)
    kept, n = bn.kv_evict(acc[1], lens, 10, 1, 2, *own, *out, acc[2])
    return (o, lse, kept, n, *acc, *bn.kv_read(bn.TARGET, None, cap, *own))

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    r = step()
graph.replay()
got = [t.clone() for t in r]
acc = accs()
assert all(torch.equal(a, b) for a, b in zip(got, step())) and bool(got[0].abs().max() > 0)
torch.cuda.synchronize()
assert bn.device_wait_timeout() == 0
print("same")
"""


def test_first_calls_of_a_process_may_be_captured():
    """A graph that holds the first calls a process makes, replayed: the bits of plain calls."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
