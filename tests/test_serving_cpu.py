"""Host-side checks of the serving operators (rotary, chunk store, chunk
attention, accumulated weights, eviction): bad arguments are refused before
anything is launched, by the C entry points and by the Python wrappers, and the
rotary frequencies equal their formulas.  None of it needs a GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_jl_key_b200 as jl

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)          # 16-byte aligned, never dereferenced
FAKE2, FAKE3 = ctypes.c_void_p(1 << 21), ctypes.c_void_p(3 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)

INVALID, UNSUPPORTED, OK, WORKSPACE = (jl.JL_ERR_INVALID_ARG, jl.JL_ERR_UNSUPPORTED, jl.JL_OK,
                                       jl.JL_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    from bit_jl_key_b200 import build
    build.build()
    return jl.load()


def caller(f, **defaults):
    def call(**kw):
        assert set(kw) <= set(defaults), kw
        return f(*dict(defaults, **kw).values())
    return call


# --------------------------------------------------------------------------

@pytest.mark.parametrize("rot", [2, 20, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(lib, rot, base):
    j = np.arange(rot // 2)
    plain = base ** (-2.0 * j / rot)
    get = lambda *a, **k: jl.jl_rotary_frequencies(rot, base, *a, device="cpu", **k).double().numpy()
    # each is rounded to float once: half a step, 2^-24 of the value (and the
    # float64 pow's own error, far below)
    close = lambda a, b: np.all(np.abs(a - b) <= 2.0 ** -23 * np.abs(b))
    assert close(get(), plain)
    assert close(get("linear", factor=4.0), plain / 4.0)
    ntk = get("ntk", factor=8.0)
    if rot > 2:
        assert close(ntk, (base * 8.0 ** (rot / (rot - 2))) ** (-2.0 * j / rot))
        assert close(ntk[-1:], plain[-1:] / 8.0) and ntk[0] == 1.0
    band = get("banded", factor=8.0, original_len=8192, low=1.0, high=4.0)
    turns = 8192 * plain / (2 * math.pi)
    assert close(band[turns >= 4.0], plain[turns >= 4.0])
    assert close(band[turns <= 1.0], plain[turns <= 1.0] / 8.0)
    mid = (turns > 1.0) & (turns < 4.0)
    x = (turns[mid] - 1.0) / 3.0
    assert close(band[mid], plain[mid] * (x + (1 - x) / 8.0))


def test_frequencies_refused(lib):
    buf = (ctypes.c_float * 64)()
    call = caller(lib.jl_rotary_frequencies, r=64, base=1e4, sc=0, factor=2.0, L=10, low=1.0,
                  high=4.0, out=ctypes.cast(buf, ctypes.c_void_p))
    assert call() == OK
    for bad in (dict(r=63), dict(r=0), dict(r=2048), dict(base=1.0), dict(base=math.nan),
                dict(base=math.inf), dict(sc=4), dict(sc=-1), dict(out=NULL),
                dict(sc=1, factor=0.0), dict(sc=2, factor=math.nan), dict(sc=3, L=0),
                dict(sc=3, low=4.0), dict(sc=3, high=math.nan)):
        assert call(**bad) == INVALID, bad
    with pytest.raises(ValueError):
        jl.jl_rotary_frequencies(64, scaling="other", device="cpu")


def test_rotary_refused(lib):
    call = caller(lib.jl_rotary, Q=FAKE, K=FAKE, dt=jl.JL_BF16, n=4, Hq=8, Hkv=2, d=128, rot=128,
                  qt=1024, qh=128, kt=256, kh=128, pos=FAKE, freq=FAKE, inter=0, inv=0, scale=1.0,
                  oq=FAKE2, oqt=1024, oqh=128, ok=FAKE2, okt=256, okh=128, stream=NULL)
    assert call(n=0) == OK
    for bad in (dict(dt=2), dict(n=-1), dict(Hq=0), dict(Hkv=0), dict(rot=127), dict(rot=0),
                dict(rot=130), dict(Q=NULL), dict(oq=NULL), dict(ok=NULL), dict(pos=NULL),
                dict(freq=NULL), dict(Q=ctypes.c_void_p((1 << 20) + 1)), dict(pos=ODD),
                dict(dt=jl.JL_F32, Q=ODD), dict(inter=2), dict(inv=-1), dict(scale=math.nan),
                dict(scale=math.inf), dict(qt=-1), dict(oqh=64), dict(oqt=0), dict(oqt=512),
                dict(okt=128, okh=128)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=129, rot=2, qh=129, oqh=129, oqt=2000, kh=129, okh=129, okt=400),
                dict(d=2048, qh=2048, oqh=2048, oqt=1 << 20), dict(n=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad


POOLS = dict(codes=FAKE, norms=FAKE, values=FAKE, pages=10, P=64)


def test_store_refused(lib):
    call = caller(lib.jl_store_paged, c=FAKE, n=FAKE, V=FAKE, vt=256, vh=128, N=10, Hkv=2, words=8,
                  cn=1, d=128, cu=FAKE, B=2, **POOLS, table=FAKE, mp=4, lens=FAKE, stream=NULL)
    assert call(N=0) == OK and call(B=0) == OK
    for bad in (dict(N=-1), dict(B=-1), dict(mp=0), dict(Hkv=0), dict(pages=0), dict(P=48),
                dict(P=0), dict(codes=NULL), dict(norms=ODD), dict(values=ODD), dict(c=NULL),
                dict(c=ODD), dict(n=NULL), dict(V=NULL), dict(V=ODD), dict(vt=4), dict(vh=-8),
                dict(cu=NULL), dict(cu=ODD), dict(table=NULL), dict(lens=NULL)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(words=0), dict(words=65), dict(cn=0), dict(cn=3), dict(N=1 << 31),
                dict(Hkv=1 << 16)):
        assert call(**bad) == UNSUPPORTED, bad


def test_chunk_refused(lib):
    need = lib.jl_chunk_attention_workspace_bytes(10, 2, 8, 2, 200, 256, 128)
    assert need > 10 * 8 * 256 * 2
    f = lib.jl_chunk_attention_workspace_bytes
    assert f(0, 2, 8, 2, 200, 256, 128) == 0 and f(10, 0, 8, 2, 200, 256, 128) == 0
    assert f(10, 2, 8, 3, 200, 256, 128) == 0 and f(10, 2, 8, 2, 200, 96, 128) == 0
    assert f(10, 2, 8, 2, 200, 256, 96) == 0 and f(1 << 30, 2, 8, 2, 200, 256, 128) == 0
    call = caller(lib.jl_chunk_attention_paged, Q=FAKE, dt=jl.JL_BF16, qt=1024, qh=128, N=10,
                  S=FAKE, **POOLS, table=FAKE, mp=4, lens=FAKE, cu=FAKE, B=2, Hq=8, Hkv=2,
                  max_len=200, m=256, d=128, scale=0.1, out=FAKE, ws=FAKE, wsb=need, stream=NULL)
    assert call(N=0) == OK and call(B=0) == OK
    for bad in (dict(dt=3), dict(N=-1), dict(B=-1), dict(Hq=9), dict(Hkv=0), dict(max_len=0),
                dict(pages=0), dict(mp=0), dict(P=40), dict(max_len=257), dict(scale=math.nan),
                dict(scale=math.inf), dict(Q=NULL), dict(S=NULL), dict(S=ODD), dict(codes=NULL),
                dict(norms=ODD), dict(values=NULL), dict(table=NULL), dict(lens=NULL),
                dict(cu=NULL), dict(out=NULL), dict(out=ODD), dict(qt=-1),
                dict(dt=jl.JL_F32, Q=ODD)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(m=96), dict(d=96), dict(N=1 << 29), dict(pages=1 << 26, P=64)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=NULL), dict(ws=ODD), dict(wsb=need - 1)):
        assert call(**bad) == WORKSPACE, bad


def test_chunk_workspace_for_a_range_of_shapes(lib):
    """The bytes of a call do not grow with its shapes (few and many rows have
    kernels of their own); the bound for the largest shapes holds all smaller ones."""
    import random
    need = lib.jl_chunk_attention_workspace_bytes
    bound = lib.jl_chunk_attention_workspace_bound
    assert jl.jl_chunk_attention_workspace_bound(2048, 64, 32, 8, 32768, 256, 128) == bound(
        2048, 64, 32, 8, 32768, 256, 128)
    # fewer sequences, or a shorter cache, of as many rows: the kernel for many rows
    for big, small in (((2048, 64, 32768), (2048, 32, 32768)), ((8192, 16, 524288), (8192, 16, 131072))):
        a, b = need(*big[:2], 32, 8, big[2], 256, 128), need(*small[:2], 32, 8, small[2], 256, 128)
        assert 0 < a < b <= bound(*big[:2], 32, 8, big[2], 256, 128)
    rng = random.Random(4)
    log = lambda hi: int(math.exp(rng.uniform(0, math.log(hi))))
    reached = 0
    for _ in range(300):
        N, B, L = log(20000), log(64), log(300000)
        Hkv, G = rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 8])
        m, d = rng.choice([64, 128, 256, 512]), rng.choice([64, 128])
        top = bound(N, B, Hkv * G, Hkv, L, m, d)
        most = 0
        for _ in range(60):
            n, b, t = (x if rng.random() < 0.3 else log(x) for x in (N, B, L))
            most = max(most, need(n, b, Hkv * G, Hkv, t, m, d))
            assert most <= top, (N, B, Hkv, G, L, m, d, n, b, t)
        reached += most > top / 2
        # and it is no more than the largest keys that the rule admits, beside the rest
        assert top <= 8 * 2 ** 30 + 2 * N * Hkv * G * (max(m, d) + 8) + 2 ** 26
    assert reached > 150                        # not a bound for its own sake
    assert bound(0, 2, 8, 2, 200, 256, 128) == 0 and bound(10, 0, 8, 2, 200, 256, 128) == 0
    assert bound(10, 2, 8, 3, 200, 256, 128) == 0 and bound(10, 2, 8, 2, 200, 96, 128) == 0


def test_chunk_largest_sizes(lib):
    """Keys of a tile past the last one, and the units (row tile, key tile) of a
    head, are counted in 32 bits: what would pass them is refused."""
    f = lib.jl_chunk_attention_workspace_bytes
    call = caller(lib.jl_chunk_attention_paged, Q=FAKE, dt=jl.JL_BF16, qt=1024, qh=128, N=10,
                  S=FAKE, codes=FAKE, norms=FAKE, values=FAKE, pages=10, P=64, table=FAKE,
                  mp=2 ** 26, lens=FAKE, cu=FAKE, B=2, Hq=8, Hkv=2, max_len=200, m=256, d=128,
                  scale=0.1, out=FAKE, ws=NULL, wsb=0, stream=NULL)
    for N, B, Hq, Hkv, max_len, fits in (
            (10, 2, 8, 2, 2 ** 31 - 128, True), (10, 2, 8, 2, 2 ** 31 - 127, False),
            (10, 2, 8, 2, 2 ** 31 - 1, False),
            (2 ** 11, 1, 32, 8, 2 ** 20, True),            # a long prompt over a million keys
            (2 ** 17, 1, 32, 8, 2 ** 20, True),
            (2 ** 20, 1, 8, 8, 2 ** 20, True),             # and a million tokens over them
            (2 ** 11, 1, 64, 8, 2 ** 30, False)):          # 256 row tiles of 2^23 key tiles
        assert (f(N, B, Hq, Hkv, max_len, 256, 128) > 0) == fits, (N, max_len)
        got = call(N=N, B=B, Hq=Hq, Hkv=Hkv, max_len=max_len)
        assert got == (WORKSPACE if fits else UNSUPPORTED), (N, max_len)


def test_accumulate_refused(lib):
    call = caller(lib.jl_accumulate_attention, s=FAKE, m=FAKE, lens=FAKE, B=2, Hq=8, Hkv=2,
                  max_len=100, scale=0.1, decay=1.0, out=FAKE, stream=NULL)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(Hq=7), dict(Hkv=0), dict(max_len=0), dict(scale=math.nan),
                dict(decay=math.inf), dict(s=NULL), dict(m=NULL), dict(lens=NULL), dict(out=NULL),
                dict(s=ODD), dict(out=ODD)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(Hq=1026, Hkv=2), dict(max_len=1 << 31), dict(B=1 << 23)):
        assert call(**bad) == UNSUPPORTED, bad


def test_accumulate_refuses_an_output_over_what_it_reads(lib):
    """Blocks write while others read, so only the mass itself may be written."""
    B, Hq, Hkv, T = 2, 8, 2, 100
    s, m, out, lens = (ctypes.c_void_p(i << 24) for i in (1, 2, 3, 4))
    at = lambda p, off: ctypes.c_void_p(p.value + off)
    call = caller(lib.jl_accumulate_attention, s=s, m=m, lens=lens, B=B, Hq=Hq, Hkv=Hkv, max_len=T,
                  scale=0.1, decay=1.0, out=out, stream=NULL)
    mass, all_scores = B * Hkv * T * 4, B * Hq * T * 4
    for bad in (dict(out=s), dict(out=at(s, all_scores - 4)), dict(out=at(s, 4 - mass)),
                dict(out=at(m, 16)), dict(out=at(m, -16)), dict(out=at(m, mass - 4)),
                dict(out=at(lens, 4)), dict(out=at(lens, 4 - mass))):
        assert call(**bad) == INVALID, bad
    # beside them, over the mass itself, and over a mass that is not read: past the checks
    # (there is no GPU here to launch on, or the launch is the caller's to make)
    if not torch.cuda.is_available():
        for good in (dict(), dict(out=m), dict(out=at(s, all_scores)), dict(out=at(m, mass)),
                     dict(out=at(m, 16), decay=0.0), dict(m=NULL, decay=0.0)):
            assert call(**good) not in (INVALID, UNSUPPORTED, OK), good


def test_evict_refused(lib):
    call = caller(lib.jl_evict_paged, m=FAKE, lens=FAKE, B=2, Hkv=2, max_len=200, keep=100,
                  recent=10, sink=4, words=8, cn=1, d=128, **POOLS, src=FAKE, sp=4, dst=FAKE2,
                  dp=2, oi=FAKE, om=FAKE2, ol=FAKE3, stream=NULL)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(Hkv=0), dict(max_len=0), dict(keep=0), dict(recent=-1),
                dict(sink=-1), dict(recent=97), dict(recent=2 ** 31 - 1, sink=2 ** 31 - 1),
                dict(sp=0), dict(dp=0), dict(dp=1), dict(sp=3), dict(P=48), dict(codes=NULL),
                dict(m=NULL), dict(lens=NULL), dict(src=NULL), dict(dst=NULL), dict(oi=NULL),
                dict(om=NULL), dict(ol=NULL), dict(om=FAKE), dict(om=ODD)):
        assert call(**bad) == INVALID, bad
    # written and still read: the mass, in part too; the lengths; a cache shrunk in place
    at = lambda p, off: ctypes.c_void_p(p.value + off)
    for bad in (dict(om=at(FAKE, 2 * 2 * 200 * 4 - 4)), dict(om=at(FAKE, 4 - 2 * 2 * 100 * 4)),
                dict(ol=FAKE), dict(ol=at(FAKE, 4)), dict(dst=FAKE)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=80), dict(words=99), dict(cn=4)):
        assert call(**bad) == UNSUPPORTED, bad


def test_evict_refuses_outputs_over_what_it_reads_or_writes(lib):
    B, Hkv, T, keep, P, pages, words, d = 2, 2, 200, 100, 64, 10, 8, 128
    ptr = {k: ctypes.c_void_p((i + 1) << 26) for i, k in enumerate(
        ("m", "lens", "codes", "norms", "values", "src", "dst", "oi", "om", "ol"))}
    rows = pages * Hkv * P
    size = dict(m=B * Hkv * T * 4, lens=B * 4, codes=rows * words * 4, norms=rows * 2,
                values=rows * d * 2, src=B * 4 * 4, dst=B * 2 * 4, oi=B * Hkv * keep * 4,
                om=B * Hkv * keep * 4, ol=B * 4)
    call = caller(lib.jl_evict_paged, m=ptr["m"], lens=ptr["lens"], B=B, Hkv=Hkv, max_len=T,
                  keep=keep, recent=10, sink=4, words=words, cn=1, d=d, codes=ptr["codes"],
                  norms=ptr["norms"], values=ptr["values"], pages=pages, P=P, src=ptr["src"], sp=4,
                  dst=ptr["dst"], dp=2, oi=ptr["oi"], om=ptr["om"], ol=ptr["ol"], stream=NULL)
    for out in ("oi", "om", "ol"):
        for other in ptr:
            if other != out:
                for at in (ptr[other].value + size[other] - 4, ptr[other].value + 4 - size[out]):
                    assert call(**{out: ctypes.c_void_p(at)}) == INVALID, (out, other)
    if not torch.cuda.is_available():          # side by side: past the checks
        assert call() not in (INVALID, UNSUPPORTED, OK)
        assert call(om=ctypes.c_void_p(ptr["oi"].value + size["oi"])) not in (INVALID, UNSUPPORTED)


def test_evict_largest_sizes(lib):
    """The grid of moved keys is counted in blocks of 128 keys, in 64 bits."""
    ptr = [ctypes.c_void_p((i + 1) << 50) for i in range(10)]
    call = caller(lib.jl_evict_paged, m=ptr[0], lens=ptr[1], B=1, Hkv=1, max_len=200, keep=100,
                  recent=0, sink=0, words=8, cn=1, d=128, codes=ptr[2], norms=ptr[3],
                  values=ptr[4], pages=10, P=64, src=ptr[5], sp=4, dst=ptr[6], dp=2, oi=ptr[7],
                  om=ptr[8], ol=ptr[9], stream=NULL)
    most = 2 ** 31 - 1
    wide = dict(dp=2 ** 25)                     # destination pages for any keep
    for keep, B, Hkv, fits in ((most, 1, 1, True), (most - 126, 1, 1, True), (most, 15, 8, True),
                               (most, 16, 8, False), (2 ** 20, 2 ** 10, 2 ** 8, False),
                               (2 ** 20, 2 ** 10, 2 ** 8 - 1, True), (1, 2 ** 12, 2 ** 12, False),
                               (1, 2 ** 12, 2 ** 12 - 1, True)):
        got = call(keep=keep, B=B, Hkv=Hkv, **wide)
        if not fits:
            assert got == UNSUPPORTED, (keep, B, Hkv)
        elif not torch.cuda.is_available():     # (nothing to launch on: past the checks)
            assert got not in (INVALID, UNSUPPORTED, OK), (keep, B, Hkv)


# --------------------------------------------------------------------------
# the wrappers' own checks, on CPU tensors (which they refuse last)

def _cache(B=2, Hkv=2, d=64, W=4, P=32, pages=6):
    return (torch.zeros(pages, Hkv, P, W, dtype=torch.int32),
            torch.zeros(pages, Hkv, P, dtype=torch.float16),
            torch.zeros(pages, Hkv, P, d, dtype=torch.bfloat16),
            torch.zeros(B, 3, dtype=torch.int32), torch.zeros(B, dtype=torch.int32))


def test_wrappers_refuse():
    cp, npg, vp, table, lens = _cache()
    cu = torch.zeros(3, dtype=torch.int32)
    Q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    S = torch.zeros(128, 64, dtype=torch.bfloat16)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.zeros(32)
    bad = (ValueError, TypeError)

    def refused(f, *a, **k):
        with pytest.raises(bad):
            f(*a, **k)

    # rotary
    refused(jl.jl_rotary, Q.half(), pos, freq)
    refused(jl.jl_rotary, Q[0], pos, freq)
    refused(jl.jl_rotary, Q, pos.long(), freq)
    refused(jl.jl_rotary, Q, pos[:3], freq)
    refused(jl.jl_rotary, Q, pos, freq.double())
    refused(jl.jl_rotary, Q, pos, freq, K=Q.float())
    refused(jl.jl_rotary, Q, pos, freq, K=Q[:3])
    refused(jl.jl_rotary, Q, pos, freq, out_q=Q[:, :2])
    refused(jl.jl_rotary, Q, pos, freq, out_k=Q)
    refused(jl.jl_rotary, Q.transpose(1, 2), pos, freq)
    refused(jl.jl_rotary, Q, pos, freq)                       # not on a GPU
    # store
    codes, norms = torch.zeros(5, 2, 4, dtype=torch.int32), torch.zeros(5, 2, dtype=torch.float16)
    V = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    ok = [codes, norms, V, cu, cp, npg, vp, table, lens]
    for i, t in ((0, codes[:4]), (0, codes.long()), (0, codes[..., :2]), (1, norms.float()),
                 (1, norms[:, :1]), (2, V.float()), (2, V[..., :32]), (2, V.transpose(1, 2)),
                 (3, cu[:2]), (3, cu.long()), (4, cp.long()), (4, cp[0]), (5, npg.float()),
                 (6, vp.half()), (7, table[0]), (7, table.long()), (8, lens.long())):
        refused(jl.jl_store_paged, *ok[:i], t, *ok[i + 1:])
    refused(jl.jl_store_paged, *ok)                           # not on a GPU
    # chunk attention
    ok = [Q, S, cp, npg, vp, table, lens, cu]
    for i, t in ((0, Q.half()), (0, Q[0]), (0, Q[..., :32]), (1, S.float()), (1, S[:64]),
                 (2, cp[..., :2]), (3, torch.zeros(*npg.shape, 2, dtype=torch.float16)),
                 (4, vp.float()), (5, table.long()), (6, lens.long()), (7, cu[:2])):
        refused(jl.jl_chunk_attention_paged, *ok[:i], t, *ok[i + 1:], 90)
    refused(jl.jl_chunk_attention_paged, *ok, 90, out=Q.float())
    refused(jl.jl_chunk_attention_paged, *ok, 90)             # not on a GPU
    # weights
    sc, mass = torch.zeros(2, 4, 50), torch.zeros(2, 2, 50)
    for a in ((sc.half(), mass, lens), (sc[0], mass, lens), (sc, mass[..., :40], lens),
              (sc, mass.double(), lens), (sc, mass, lens.long()), (sc, mass, lens[:1])):
        refused(jl.jl_accumulate_attention, *a, 0.1)
    refused(jl.jl_accumulate_attention, sc, mass, lens, 0.1, out=sc)
    refused(jl.jl_accumulate_attention, sc, mass, lens, 0.1)  # not on a GPU
    # eviction
    ok = [mass, lens, 20, cp, npg, vp, table, table]
    for i, t in ((0, mass.double()), (0, mass[:, :1]), (1, lens.long()), (2, 0), (6, table[0]),
                 (7, table.long())):
        refused(jl.jl_evict_paged, *ok[:i], t, *ok[i + 1:])
    refused(jl.jl_evict_paged, *ok, out_index=torch.zeros(2, 2, 19, dtype=torch.int32))
    refused(jl.jl_evict_paged, *ok)                           # not on a GPU


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Launched there, the kernels would read this device's memory from the other."""
    class On:
        def __init__(self, index):
            self.device = torch.device("cuda", index)
            self.cuda_stream = 0

        def get_device(self):
            return self.device.index

    def no_entry(*a):
        raise AssertionError("the call went on")

    monkeypatch.setattr(torch.cuda, "device", no_entry)
    monkeypatch.setattr(torch.cuda, "stream", no_entry)
    for stream, tensor in ((On(1), On(0)), (On(0), On(1))):
        with pytest.raises(ValueError, match="device"):
            jl._on(stream, (tensor,), no_entry)
