"""Rotary positions and the nested cache's serving entry points on the host (no
GPU): every refusal comes before anything is launched, and empty problems
succeed.  Addresses are fake and never read."""
import ctypes

import numpy as np
import pytest

import w8_quantized_linear_b200 as bn
from oracle import serving as ref
from w8_quantized_linear_b200 import build

A, B2 = 0x10000, 0x20000
MIS = A + 2


@pytest.fixture(scope="module")
def L():
    build.build()
    return bn.lib()


def cache(base=A, **kw):
    c = bn._KvCacheC(*(base + 0x100 * i for i in range(6)))
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_rope_phases(L):
    ph = (ctypes.c_uint64 * 64)()
    m = ctypes.c_float()

    def call(rot=128, base=1e4, scaling=0, factor=1.0, low=1.0, high=4.0, trained=8192, p=ph):
        return L.bitnest_rope_phases(rot, base, scaling, factor, low, high, trained, p, ctypes.byref(m))

    assert call(rot=0) == 2 and call(rot=3) == 2 and call(rot=1 << 20) == 2
    assert call(rot=2, scaling=2, factor=2.0) == 2  # rot / (rot - 2)
    assert call(base=1.0) == 1 and call(base=float("nan")) == 1 and call(base=float("inf")) == 1
    assert call(scaling=5) == 1 and call(scaling=-1) == 1 and call(p=None) == 1
    assert call(scaling=1, factor=0.5) == 1 and call(scaling=1, factor=float("inf")) == 1
    assert call(scaling=3, factor=2.0, low=0.0) == 1 and call(scaling=3, factor=2.0, high=1.0) == 1
    assert call(scaling=4, factor=2.0, trained=0) == 1
    names = ["plain", "linear", "ntk", "bands", "yarn"]
    for kind, name in enumerate(names):
        assert call(scaling=kind, factor=8.0) == 0
        theta, mag = ref.rope_theta(128, 1e4, name, 8.0, 1.0, 4.0, 8192)
        got = np.array(ph[:], dtype=np.uint64)
        # two evaluations in fp64 (a power, a few products), 16 roundings at most, and the
        # phase's own rounding to a unit of 2^-64 turns: half of one is 2 pi 2^-65
        assert np.all(np.abs(got / 2.0 ** 64 * 2 * np.pi - theta) <= 2.0 ** -49 * theta + np.pi * 2.0 ** -64)
        assert m.value == np.float32(mag)
    assert call() == 0 and ph[0] == round(2.0 ** 64 / (2 * np.pi))


def test_rope_refusals(L):
    def call(x=A, xt=0, x_tok=512, x_head=128, pos=A, ph=A, M=2, heads=4, D=128, rot=64, layout=0,
             y=B2, yt=0, y_tok=512, y_head=128):
        return L.bitnest_rope(x, xt, x_tok, x_head, pos, ph, 1.0, M, heads, D, rot, layout, 0, y, yt,
                              y_tok, y_head, None)

    assert call(xt=2) == 1 and call(yt=-1) == 1 and call(layout=2) == 1
    assert call(x=None) == 1 and call(y=None) == 1 and call(pos=None) == 1 and call(ph=None) == 1
    assert call(rot=0) == 2 and call(rot=63) == 2 and call(rot=130) == 2 and call(D=1, rot=0) == 2
    assert call(M=-1) == 2 and call(heads=-1) == 2 and call(heads=70000) == 2
    assert call(M=1 << 31) == 2 and call(D=1 << 17) == 2
    assert call(y_head=127) == 2 and call(y_tok=511) == 2 and call(x_tok=-1) == 2 and call(y_head=-128) == 2
    assert call(y=A, yt=1) == 1 and call(y=A, y_tok=640) == 1  # in place, not onto itself
    assert call(x=A + 1) == 3 and call(y=B2 + 2, yt=1) == 3 and call(pos=MIS) == 3 and call(ph=A + 4) == 3
    assert call(M=0, x=None) == 0 and call(heads=0, y=None) == 0


def test_append_and_read_refusals(L):
    def app(k=A, kt=1024, v=A, vt=1024, type=0, B=2, n=3, Hkv=8, start=A, count=None, pos=A, ph=A,
            rot=128, layout=0, c=cache(), cap=16):
        return L.bitnest_kv_append(k, kt, v, vt, type, B, n, Hkv, start, count, pos, ph, 1.0, rot,
                                   layout, c, cap, None)

    assert app(type=2) == 1 and app(layout=3) == 1 and app(k=None) == 1 and app(v=None) == 1
    assert app(start=None) == 1 and app(pos=None) == 1 and app(c=None) == 1
    assert app(c=cache(v_lo=None)) == 1 and app(c=cache(k_scale=A + 8)) == 3
    assert app(rot=8) == 2 and app(rot=24) == 2 and app(rot=144) == 2
    assert app(kt=1023) == 2 and app(kt=1028) == 3 and app(vt=1026, type=1) == 3
    assert app(B=-1) == 2 and app(n=-1) == 2 and app(Hkv=0) == 2 and app(cap=-1) == 2 and app(n=1 << 31) == 2
    assert app(k=MIS) == 3 and app(start=A + 1) == 3 and app(count=A + 1) == 3 and app(ph=A + 4) == 3
    assert app(B=0, k=None) == 0 and app(n=0) == 0 and app(cap=0) == 0

    def read(mode=1, c=cache(), B=2, cap=16, Hkv=8, start=A, n=3, k=A, v=A):
        return L.bitnest_kv_read(mode, c, B, cap, Hkv, start, n, k, v, None)

    assert read(mode=2) == 1 and read(c=None) == 1 and read(k=None) == 1 and read(c=cache(v_lo=None)) == 1
    assert read(n=-1) == 2 and read(Hkv=0) == 2 and read(v=MIS) == 3 and read(start=A + 1) == 3
    assert read(mode=0, c=cache(v_lo=None, k_lo=MIS), v=MIS) == 3  # the draft does not look at lo planes
    assert read(B=0) == 0 and read(n=0) == 0


def test_prefix_attention_refusals(L):
    need = L.bitnest_prefix_attention_ws_bytes(4, 2, 8, 2, 100, 20)
    assert need > 0 and need % 16 == 0
    assert L.bitnest_prefix_attention_ws_bytes(4, 2, 6, 2, 100, 20) == -2  # 3 heads a KV head
    assert L.bitnest_prefix_attention_ws_bytes(0, 2, 8, 2, 100, 20) == 0

    def call(mode=1, q=A, B=4, n=2, H=8, Hkv=2, D=128, pc=cache(), P=100, oc=cache(), cap=20, lens=A,
             out=A, lse=A, ws=A, nb=need):
        return L.bitnest_prefix_attention(mode, q, B, n, H, Hkv, D, pc, P, oc, cap, lens, out, lse, ws,
                                          nb, None)

    assert call(mode=2) == 1 and call(q=None) == 1 and call(out=None) == 1 and call(lens=None) == 1
    assert call(pc=None) == 1 and call(oc=None) == 1 and call(oc=cache(v_lo=None)) == 1
    assert call(ws=None) == 1 and call(nb=need - 1) == 1
    assert call(D=64) == 2 and call(H=6) == 2 and call(H=32) == 2 and call(n=0) == 2 and call(P=-1) == 2
    assert call(B=-1) == 2 and call(cap=-1) == 2 and call(P=1 << 31) == 2
    assert call(q=MIS) == 3 and call(out=MIS) == 3 and call(ws=MIS) == 3 and call(lens=A + 1) == 3
    assert call(lse=A + 1) == 3 and call(pc=cache(k_hi=MIS)) == 3
    assert call(B=0, q=None) == 0


def test_weights_refusals(L):
    def call(mode=1, q=A, lse=A, B=4, n=2, H=8, Hkv=2, D=128, hi=A, lo=A, sc=A, cap=20, lens=A, acc=A):
        return L.bitnest_kv_weights(mode, q, lse, B, n, H, Hkv, D, hi, lo, sc, cap, lens, acc, None)

    assert call(mode=-1) == 1 and call(q=None) == 1 and call(lse=None) == 1 and call(lo=None) == 1
    assert call(acc=None) == 1 and call(D=127) == 2 and call(H=10) == 2 and call(n=0) == 2
    assert call(B=40000) == 2 and call(cap=-1) == 2 and call(hi=MIS) == 3 and call(acc=A + 1) == 3
    assert call(mode=0, lo=None, acc=A + 1) == 3
    assert call(B=0) == 0 and call(cap=0) == 0


def test_evict_refusals(L):
    def call(acc=A, lens=A, B=2, Hkv=2, cap=30, keep=10, sinks=2, recent=3, src=cache(), dst=cache(B2),
             dcap=12, dacc=B2, kept=B2, dlen=B2 + 64):
        return L.bitnest_kv_evict(acc, lens, B, Hkv, cap, keep, sinks, recent, src, dst, dcap, dacc, kept,
                                  dlen, None)

    assert call(keep=0) == 1 and call(keep=13) == 1 and call(sinks=-1) == 1 and call(recent=9) == 1
    assert call(sinks=11) == 1 and call(acc=None) == 1 and call(lens=None) == 1 and call(kept=None) == 1
    assert call(dst=cache()) == 1 and call(dacc=A) == 1 and call(dlen=A) == 1  # onto themselves
    assert call(src=None) == 1 and call(dst=cache(B2, v_hi=None)) == 1
    assert call(Hkv=0) == 2 and call(B=-1) == 2 and call(cap=-1) == 2
    assert call(dst=cache(B2, k_hi=B2 + 2)) == 3 and call(kept=B2 + 1) == 3
    assert call(B=0) == 0


def test_python_refusals():
    """Wrong types, shapes and devices are refused before the library is called."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(ValueError):
        bn.rope(z(2, 3, 128), z(2, dtype=torch.int32), z(64, dtype=torch.int64))  # on the CPU
    with pytest.raises(ValueError):
        bn.rope(z(2, 3, 128, dtype=torch.float64), z(2, dtype=torch.int32), z(64, dtype=torch.int64))
    k_pl, v_pl = bn.nested_cache(8, 2, 1, device="cpu")
    assert k_pl[0].shape == (1, 8, 2, 64) and v_pl[2].shape == (1, 8, 2)
    with pytest.raises(ValueError):
        bn.kv_append(z(1, 2, 2, 128), z(1, 2, 2, 128), z(1, dtype=torch.int32), k_pl, v_pl)
    with pytest.raises(ValueError):
        bn.kv_read(1, None, 2, k_pl, v_pl)
    with pytest.raises(ValueError):
        bn.prefix_attention(1, z(1, 1, 4, 128, dtype=torch.float16), None, (k_pl, v_pl), z(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        bn.prefix_attention(1, z(1, 1, 4, 128, dtype=torch.float16), None, None, z(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        bn.kv_evict(z(1, 2, 8), z(1, dtype=torch.int32), 2, 0, 0, k_pl, v_pl, k_pl, v_pl, z(1, 2, 8))


def test_oracle_attention_against_a_dense_softmax():
    """The oracle on unit-scale codes against numpy's dense softmax, with the causal edge."""
    rng = np.random.default_rng(0)
    B, n, H, Hkv, P, cap = 2, 2, 4, 2, 5, 4
    mk = lambda *s: (rng.integers(0, 256, (*s, 64)).astype(np.uint8), rng.integers(0, 256, (*s, 64)).astype(np.uint8), np.full(s, 0.25, np.float16))  # noqa: E731
    prefix, own = [mk(P, Hkv) for _ in range(2)], [mk(B, cap, Hkv) for _ in range(2)]
    q = rng.standard_normal((B, n, H, 128)).astype(np.float16)
    lens = np.array([4, 1])
    out, lse, _ = ref.attention(1, q, prefix, own, lens)
    for b in range(B):
        k, v = (np.concatenate([ref.values(1, prefix[i]), ref.values(1, own[i])[b]]) for i in range(2))
        for i in range(n):
            seen = np.r_[np.ones(P, bool), np.arange(cap) <= lens[b] - n + i]
            s = np.einsum("hd,thd->ht", q[b, i].astype(float), np.repeat(k, 2, 1)) / np.sqrt(128)
            e = np.exp(s) * seen
            assert np.allclose(lse[b, i], np.log(e.sum(1)), rtol=1e-12)
            assert np.allclose(out[b, i], np.einsum("ht,thd->hd", e / e.sum(1, keepdims=True), np.repeat(v, 2, 1)), rtol=1e-10, atol=1e-12)
    # the weights of every row sum to one
    a = ref.weights(1, q, lse, prefix[0], np.zeros((Hkv, P)))
    o = ref.weights(1, q, lse, own[0], np.zeros((B, Hkv, cap)), lens)
    assert np.allclose(a.sum(1) + o.sum((0, 2)), B * n * H / Hkv, rtol=1e-12)


def test_oracle_evict_by_hand():
    acc = np.array([9, 1, 5, 5, 0, 5, 2, 3], np.float32)
    assert ref.evict(acc, 8, 8, 0, 0) == list(range(8))
    assert ref.evict(acc, 8, 4, 0, 0) == [0, 2, 3, 5]
    assert ref.evict(acc, 8, 4, 2, 1) == [0, 1, 2, 7]  # of the three fives the first
    acc[2] = np.nan
    assert ref.evict(acc, 8, 3, 0, 0) == [0, 3, 5] and ref.evict(acc, 7, 6, 1, 0) == [0, 1, 3, 4, 5, 6]


def test_weights_refuses_more_tiles_of_a_shared_cache_than_it_counts(L):
    def call(Hkv, cap, lens=None):
        return L.bitnest_kv_weights(1, A, A, 1, 1, Hkv, Hkv, 128, A, A, A, cap, lens, A + 1, None)

    # (the misaligned acc ends the calls whose shape is taken)
    assert call(128, 1 << 30) == 2 and call(129, 1 << 30) == 2 and call(127, 1 << 30) == 3
    assert call(65535, 16384 * 128) == 3 and call(65535, 16385 * 128) == 2  # 2^30 - 2^14 tiles, and 65535 more
    assert call(128, 1 << 30, lens=A) == 3  # own tokens: another kernel
