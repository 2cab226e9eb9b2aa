"""The serving operators against plain float64 implementations: rotary
positions, a chunk into the pages, attention of a chunk, accumulated weights,
eviction, and a run of them together.

Tolerances are sums of the roundings on the way, written where they are used;
a bf16 rounding is half a step, 2^-8 of the value, a binary16 one 2^-11, an
fp32 one 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import bit_jl_key_b200 as jl
import oracle
from tests import helpers as H

pytestmark = pytest.mark.gpu

U32, U16, UB = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8
DEV = "cuda"


def _rng(seed):
    return np.random.default_rng(seed)


def _randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, torch.int32)


# --------------------------------------------------------------------------
# rotary

def rotary64(x, pos, freq, inter, inverse, scale):
    """float64 numpy; also the sum |a| + |b| of each entry's pair."""
    x = np.array(x, dtype=np.float64)
    h = len(freq)
    e, o = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if inter else (slice(0, h), slice(h, 2 * h))
    ang = (np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64))[:, None]
    ang = -ang if inverse else ang
    a, b = x[..., e].copy(), x[..., o].copy()
    mag = np.zeros_like(x)
    mag[..., e] = mag[..., o] = np.abs(a) + np.abs(b)
    x[..., e] = scale * (a * np.cos(ang) - b * np.sin(ang))
    x[..., o] = scale * (a * np.sin(ang) + b * np.cos(ang))
    return x, mag * abs(scale)


def check_rotary(got, x, pos, freq, inter, inverse, scale):
    want, mag = rotary64(H.f64(x), pos.cpu().numpy(), freq.cpu().numpy(), inter, inverse, scale)
    # fp32: sin and cos are off by 2 ulp (2^-23 at most), times scale, one
    # product and one fma: 6 roundings of |a| + |b|; then the output's own
    tol = 6 * U32 * mag + (UB if x.dtype == torch.bfloat16 else U32) * np.abs(want)
    err = np.abs(H.f64(got) - want)
    assert np.all(err <= tol + 1e-38), (err - tol).max()
    r = 2 * len(freq)
    assert torch.equal(got[..., r:], x[..., r:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot", [(1, 8, 2, 128, 128), (77, 6, 3, 64, 32),
                                            (5, 1, 1, 128, 20), (300, 4, 4, 64, 64),
                                            (2500, 2, 1, 128, 64), (3, 2, 2, 6, 2)])
def test_rotary(dtype, inter, n, Hq, Hkv, d, rot):
    qkv = _randn(1, n, Hq + 2 * Hkv, d, dtype=dtype)
    Q, K = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    rng = _rng(n)
    pos = _i32(rng.integers(-5, 1 << 20, size=n))
    freq = jl.jl_rotary_frequencies(rot, scaling="banded", factor=8.0, original_len=8192)
    for inverse, scale in ((False, 1.0), (True, 1.0), (False, -1.3)):
        oq, ok = jl.jl_rotary(Q, pos, freq, K=K, interleaved=inter, inverse=inverse, scale=scale)
        check_rotary(oq, Q, pos, freq, inter, inverse, scale)
        check_rotary(ok, K, pos, freq, inter, inverse, scale)
    # queries alone; in place; into other strides; heads ahead of tokens
    assert torch.equal(jl.jl_rotary(Q, pos, freq, interleaved=inter),
                       jl.jl_rotary(Q, pos, freq, K=K, interleaved=inter)[0])
    want = jl.jl_rotary(Q, pos, freq, K=K, interleaved=inter)
    out = torch.full((Hq + 1, n, d + 8), 7.0, dtype=dtype, device=DEV)
    view = out[:Hq, :, :d].transpose(0, 1)
    jl.jl_rotary(Q.transpose(0, 1).contiguous().transpose(0, 1), pos, freq, interleaved=inter,
                 out_q=view)
    assert torch.equal(view, want[0])
    assert torch.all(out[Hq] == 7.0) and torch.all(out[:, :, d:] == 7.0)
    v_part = qkv[:, Hq + Hkv:].clone()
    jl.jl_rotary(Q, pos, freq, K=K, interleaved=inter, out_q=Q, out_k=K)
    assert torch.equal(Q, want[0]) and torch.equal(K, want[1])
    assert torch.equal(qkv[:, Hq + Hkv:], v_part)


def test_rotary_unaligned_rows_and_extremes():
    d, n = 64, 9
    flat = _randn(2, n * 3 * (d + 1) + 1)
    Q = flat[1:].view(n, 3, d + 1)[..., :d]                    # rows at odd 4-byte offsets
    pos = _i32([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, 12345678, 3, 4])
    freq = torch.tensor([1.0, 0.7, 1e-3, 0.0] + [0.1] * 28, device=DEV)
    got = jl.jl_rotary(Q, pos, freq)
    check_rotary(got, Q, pos, freq, False, False, 1.0)
    assert jl.jl_rotary(Q[:0], pos[:0], freq).shape == (0, 3, d)
    x = Q.clone()
    x[0, 0, 0], x[1, 0, 1] = math.inf, math.nan                # stay in their own pairs
    y = jl.jl_rotary(x, pos, freq)
    bad = ~torch.isfinite(y)
    assert {tuple(i) for i in bad.nonzero().tolist()} <= {(0, 0, 0), (0, 0, 32), (1, 0, 1),
                                                          (1, 0, 33)}
    with pytest.raises(jl.JLError):
        jl.jl_rotary(Q, pos, torch.zeros(33, device=DEV))      # rot_dim above d


def test_rotary_inverse_is_the_gradient():
    n, Hq, d = 13, 3, 64
    x, gy = _randn(3, n, Hq, d), _randn(4, n, Hq, d)
    pos = _i32(_rng(0).integers(0, 5000, size=n))
    freq = jl.jl_rotary_frequencies(48)
    gx = jl.jl_rotary(gy, pos, freq, inverse=True, scale=1.5)
    # the formula's gradient by autograd in float64 (the copied entries are not scaled)
    xx = x.double().requires_grad_()
    ang = pos.double()[:, None, None] * freq.double()
    a, b = xx[..., :24], xx[..., 24:48]
    y = torch.cat([1.5 * (a * ang.cos() - b * ang.sin()), 1.5 * (a * ang.sin() + b * ang.cos()),
                   xx[..., 48:]], -1)
    y.backward(gy.double())
    assert torch.all((gx.double() - xx.grad).abs() <= 8 * U32 * 1.5 * 2 * gy.abs().max())
    # and by differences: the rotation is linear, so any step serves
    e = _randn(5, n, Hq, d)
    f = lambda t: (jl.jl_rotary(t, pos, freq, scale=1.5).double() * gy.double()).sum()
    diff = f(x + e) - f(x - e)
    exact = 2 * (gx.double() * e.double()).sum()
    # each of the sum's terms carries the roundings of an fp32 rotation
    bound = 16 * U32 * 1.5 * 2 * ((x.abs() + e.abs()).double() * 2 * gy.abs().double().max()).sum()
    assert abs(diff - exact) <= bound


# --------------------------------------------------------------------------
# a paged cache made from keys with the oracle's codes

def table_for(lens, P, pages, rng, width=None):
    width = width or max(1, max(-(-int(L) // P) for L in lens))
    perm = rng.permutation(pages)
    tab = np.full((len(lens), width), -1, dtype=np.int32)
    k = 0
    for b, L in enumerate(lens):
        p = -(-int(L) // P)
        tab[b, :p] = perm[k:k + p]
        k += p
    assert k <= pages
    return tab


class Cache:
    """Pools full of garbage (random codes, NaN norms and values) apart from the
    sequences' keys, whose code bits and norms are random too."""

    def __init__(self, lens, Hkv, d, m, P, seed, norm_scale=None, extra=3):
        rng = _rng(seed)
        self.lens, self.Hkv, self.d, self.m, self.P = list(lens), Hkv, d, m, P
        pages = sum(-(-int(L) // P) for L in lens) + extra
        self.table = table_for(lens, P, pages, rng)
        self.codes = rng.integers(0, 2 ** 32, size=(pages, Hkv, P, m // 32), dtype=np.uint64
                                  ).astype(np.uint32)
        self.norms = np.full((pages, Hkv, P), np.nan, np.float16)
        self.values = torch.full((pages, Hkv, P, d), math.nan, dtype=torch.bfloat16)
        scale = math.sqrt(d) if norm_scale is None else norm_scale
        for b, L in enumerate(lens):
            t = np.arange(L)
            pg, sl = self.table[b, t // P], t % P
            self.norms[pg, :, sl] = (scale * np.exp(0.3 * rng.standard_normal((L, Hkv)))
                                     ).astype(np.float16)
            self.values[pg, :, sl] = torch.from_numpy(rng.standard_normal((L, Hkv, d))
                                                      ).to(torch.bfloat16)
        self.S = jl.jl_sketch_init(m, d, 0)

    def dev(self):
        return (torch.from_numpy(self.codes.view(np.int32)).to(DEV),
                torch.from_numpy(self.norms).to(DEV), self.values.to(DEV), _i32(self.table))

    def keys(self, b, h):
        """(khat [L, d] and its sketch form [L, m], values [L, d]) in float64."""
        t = np.arange(self.lens[b])
        pg, sl = self.table[b, t // self.P], t % self.P
        z = H.code_bits(self.codes[pg, h, sl], self.m).astype(np.float64) * 2 - 1
        zn = z * (self.norms[pg, h, sl].astype(np.float64) * math.sqrt(math.pi / 2) / self.m)[:, None]
        return zn @ H.f64(self.S), zn, H.f64(self.values[pg, h, sl])


def chunk64(c, Q, counts, scale, first=0):
    """Attention of the chunk in float64 with the tolerance of each output:
    {(row, head): (out, tol)}."""
    S = H.f64(c.S)
    Hq = Q.shape[1]
    G = Hq // c.Hkv
    out, row = {}, first
    for b, n in enumerate(counts):
        for h in range(c.Hkv):
            khat, zn, v = c.keys(b, h)
            for i in range(n):
                seen = max(0, c.lens[b] - n + i + 1)
                for g in range(G):
                    q = H.f64(Q[row + i, h * G + g])
                    if seen == 0:
                        out[row + i, h * G + g] = (np.zeros(c.d), np.zeros(c.d))
                        continue
                    s = scale * (khat[:seen] @ q)
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    o = w @ v[:seen]
                    A = w @ np.abs(v[:seen])
                    # a logit's error: the projection u = S q, or q and khat, as
                    # binary16, and the fp32 sums of m or d products
                    by_u = np.abs(zn[:seen]) @ np.abs(S @ q) * (U16 + (c.m + c.d) * U32)
                    by_k = np.abs(khat[:seen]) @ np.abs(q) * 2 * (U16 + c.d * U32)
                    delta = abs(scale) * np.maximum(by_u, by_k).max()
                    # plus the fp32 exponent's own rounding, relative to its size
                    delta += 4 * U32 * (np.abs(s).max() + 8)
                    # weights: bf16 and the exponential's 2^-13; output: bf16
                    tol = (UB + 2.0 ** -13 + 2 * delta * math.exp(2 * delta)) * 1.01 * A
                    tol += UB * (np.abs(o) + tol) + 1e-30
                    out[row + i, h * G + g] = (o, tol)
        row += n
    return out


def run_chunk(c, Q, counts, lens=None, pad=(0, 0), scale=None, **kw):
    """The call on a batch with pad[0] rows before and pad[1] behind."""
    cu = pad[0] + np.concatenate([[0], np.cumsum(counts)])
    codes, norms, values, table = c.dev()
    lens = c.lens if lens is None else lens
    out = torch.full((Q.shape[0], Q.shape[1], c.d), 7.0, dtype=torch.bfloat16, device=DEV)
    return jl.jl_chunk_attention_paged(Q, c.S, codes, norms, values, table, _i32(lens), _i32(cu),
                                       max(max(lens), 1), softmax_scale=scale, out=out, **kw)


def check_chunk(c, Q, counts, got, scale, first=0):
    g = H.f64(got)
    for (r, h), (o, tol) in chunk64(c, Q, counts, scale, first).items():
        if np.isnan(o).all():                                   # infinite norms: no answer
            assert np.isnan(g[r, h]).all(), (r, h)
            continue
        err = np.abs(g[r, h] - o)
        assert np.all(err <= tol), (r, h, (err / np.maximum(tol, 1e-30)).max())


CHUNKS = [
    # lens, counts, Hq, Hkv, d, m, P, dtype
    ([1], [1], 1, 1, 64, 64, 32, torch.bfloat16),
    ([130, 1, 64], [3, 1, 2], 8, 2, 128, 256, 32, torch.bfloat16),      # few rows, granule 32
    ([257, 100], [5, 8], 8, 1, 128, 128, 64, torch.float32),             # 64-row tiles
    ([300, 129, 128], [9, 2, 0], 6, 2, 64, 512, 96, torch.bfloat16),     # G = 3, no row of b = 2
    ([40, 700], [12, 3], 10, 2, 128, 512, 128, torch.float32),           # G = 5, granule 128
    ([200, 33], [200, 33], 4, 2, 128, 256, 64, torch.bfloat16),          # whole prompts: many rows
    ([310], [310], 3, 3, 64, 128, 32, torch.float32),
    ([129, 260], [129, 131], 2, 1, 64, 64, 96, torch.bfloat16),
    ([500], [170], 16, 1, 128, 512, 128, torch.bfloat16),                # long row tiles, causal
    ([5, 3, 140], [9, 3, 141], 4, 2, 128, 128, 32, torch.bfloat16),      # n > L: rows that see nothing
    ([2, 0, 3], [5, 2, 1], 4, 2, 64, 64, 64, torch.bfloat16),            # and an empty cache
]


@pytest.mark.parametrize("lens,counts,Hq,Hkv,d,m,P,dtype", CHUNKS)
def test_chunk_attention(lens, counts, Hq, Hkv, d, m, P, dtype):
    c = Cache(lens, Hkv, d, m, P, seed=len(lens) + d + m)
    N, pad = sum(counts), (2, 3)
    Q = _randn(7, N + 5, Hq, d, dtype=dtype)
    got = run_chunk(c, Q, counts, pad=pad)
    check_chunk(c, Q, counts, got, d ** -0.5, first=2)
    # rows of no sequence stay as they were
    assert torch.all(got[:2] == 7.0) and torch.all(got[2 + N:] == 7.0)
    # the same again, bit for bit
    assert torch.equal(got, run_chunk(c, Q, counts, pad=pad))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [64, 128, 256, 512])
@pytest.mark.parametrize("n,n2,G", [(3, 7, 4), (11, 23, 3), (97, 5, 4)])
def test_chunk_attention_every_kernel(d, m, n, n2, G):
    """Each sketch size and head size on 32-row tiles, on 64-row tiles (more than
    32 rows a sequence on average, ends inside a tile) and on expanded keys."""
    c = Cache([n + 130, 290], 2, d, m, 32 if d == 64 else 64, seed=d + m + n)
    dtype = torch.float32 if m in (64, 256) else torch.bfloat16
    Q = _randn(21, n + n2 + 1, 2 * G, d, dtype=dtype)
    got = run_chunk(c, Q, [n, n2], pad=(1, 0))
    check_chunk(c, Q, [n, n2], got, d ** -0.5, first=1)
    assert torch.all(got[0] == 7.0)
    assert torch.equal(got, run_chunk(c, Q, [n, n2], pad=(1, 0)))


@pytest.mark.parametrize("counts,G", [([1], 100), ([1, 0, 0, 0], 100), ([2, 1], 71), ([3], 97)])
def test_chunk_attention_more_heads_than_rows_of_a_tile(counts, G):
    """A token's heads over several row tiles, of each height."""
    lens = [150 + 20 * i for i in range(len(counts))]
    c = Cache(lens, 2, 64, 64, 32, seed=24)
    Q = _randn(25, sum(counts), 2 * G, 64, dtype=torch.bfloat16)
    check_chunk(c, Q, counts, run_chunk(c, Q, counts), 64 ** -0.5)


@pytest.mark.parametrize("longest,others,G", [(1, 1, 2), (900, 1, 4), (40, 12, 16)])
def test_chunk_attention_more_sequences_than_the_plan_takes_at_once(longest, others, G):
    """300 sequences: of single tokens, with a long chunk among them (more row
    tiles than are counted one by one), and with many rows each; some empty."""
    B, d, m = 300, 64, 64
    rng = _rng(26)
    counts = rng.integers(0, others + 1, size=B) if others > 1 else (rng.random(B) < 0.8) * 1
    counts = counts + (others if others > 1 else 0)
    counts[[0, 7, 299]] = 0, 0, others
    counts[260] = longest
    lens = (counts + rng.integers(0, 40, size=B)).tolist()
    counts = counts.tolist()
    c = Cache(lens, 1, d, m, 32, seed=27)
    N = sum(counts)
    assert (N * G >= 160 * B) == (others > 1)
    Q = _randn(28, N, G, d, dtype=torch.bfloat16)
    got = run_chunk(c, Q, counts)
    first = np.concatenate([[0], np.cumsum(counts)])
    for b in (1, 100, 255, 256, 257, 259, 260, 261, 298, 299):
        sub = Cache.__new__(Cache)
        sub.__dict__ = dict(c.__dict__, lens=[lens[b]], table=c.table[b:b + 1])
        part = slice(int(first[b]), int(first[b + 1]))
        if counts[b] > 50:                                      # its last rows stand for it
            part = slice(part.stop - 20, part.stop)
        check_chunk(sub, Q[part], [part.stop - part.start], got[part], d ** -0.5)
    assert torch.isfinite(got.float()).all() and torch.equal(got, run_chunk(c, Q, counts))


@pytest.mark.parametrize("n", [60, 700])
def test_chunk_attention_prompt_beside_single_tokens(n):
    """A prompt's chunk and decode steps in one batch: whichever kernel its rows
    choose, in one workspace that serves every smaller batch too."""
    lens, counts, Hq, Hkv, d, m = [n + 40, 300, 1, 129, 500, 33], [n, 1, 1, 1, 0, 1], 8, 2, 128, 256
    c = Cache(lens, Hkv, d, m, 64, seed=22)
    N, most = sum(counts), max(lens)
    ws = torch.full((jl.jl_chunk_attention_workspace_bound(N, 6, Hq, Hkv, most, m, d),), 255,
                    dtype=torch.uint8, device=DEV)
    Q = _randn(23, N, Hq, d, dtype=torch.bfloat16)
    check_chunk(c, Q, counts, run_chunk(c, Q, counts, workspace=ws), d ** -0.5)
    for k in (1, 3, 6):                                         # the first k sequences alone
        sub = Cache.__new__(Cache)
        sub.__dict__ = dict(c.__dict__, lens=lens[:k], table=c.table[:k])
        few = counts[:k]
        for part in (few, [min(x, 2) for x in few], [min(x, 45) for x in few]):
            q = Q[:sum(part)]
            check_chunk(sub, q, part, run_chunk(sub, q, part, workspace=ws), d ** -0.5)


@pytest.mark.parametrize("rows", [4, 400])
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_chunk_attention_scales_and_strides(rows, scale):
    c = Cache([rows + 150], 2, 64, 128, 64, seed=3)
    qkv = _randn(8, rows, 8, 64 + 16, dtype=torch.bfloat16)
    Q = qkv[:, 2:6, 8:72]                                       # strided heads and tokens
    got = run_chunk(c, Q, [rows], scale=scale)
    check_chunk(c, Q, [rows], got, scale)
    Qt = Q.transpose(0, 1).contiguous().transpose(0, 1)         # heads ahead of tokens
    assert torch.equal(got, run_chunk(c, Qt, [rows], scale=scale))
    odd = torch.zeros(rows * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(rows, 4, 64)
    odd.copy_(Q)                                                # rows at odd 2-byte offsets
    assert torch.equal(got, run_chunk(c, odd, [rows], scale=scale))


@pytest.mark.parametrize("n", [6, 300])
def test_chunk_attention_large_and_small_magnitudes(n):
    """Norms and queries far from 1: peaked rows, nearly uniform ones, zeros;
    the last scale passes binary16 for some keys, whose norms are infinite."""
    for norm_scale, q_scale in ((300.0, 1.0), (1e-3, 1e-3), (0.05, 2e4), (6e4, 1e-4)):
        c = Cache([n + 200], 1, 64, 128, 64, seed=5, norm_scale=norm_scale)
        Q = _randn(9, n, 2, 64) * q_scale
        Q[1] = 0.0
        check_chunk(c, Q, [n], run_chunk(c, Q, [n]), 64 ** -0.5)


@pytest.mark.parametrize("n,L", [(5, 20000), (300, 20000), (5, 60001)])
def test_chunk_attention_long_split_context(n, L):
    """One sequence over every block of the grid, each with a state to join."""
    c = Cache([L], 1, 64, 64, 64, seed=6)
    Q = _randn(10, n, 2, 64, dtype=torch.bfloat16)
    got = run_chunk(c, Q, [n])
    for i in (0, 1, n // 2, n - 1):                             # some rows, the last ones
        sub = Cache.__new__(Cache)
        sub.__dict__ = dict(c.__dict__, lens=[L - n + i + 1])
        check_chunk(sub, Q[i:i + 1], [1], got[i:i + 1], 64 ** -0.5)


def test_chunk_attention_equals_decode_steps():
    """Row i of a chunk is a decode step over the keys it sees."""
    Hq, Hkv, d, m, P, n, L = 8, 2, 128, 256, 64, 5, 333
    c = Cache([L], Hkv, d, m, P, seed=11)
    Q = _randn(12, n, Hq, d, dtype=torch.bfloat16)
    got = run_chunk(c, Q, [n]).float()
    codes, norms, values, table = c.dev()
    for i in range(n):
        step = jl.jl_decode_attention_paged(Q[i:i + 1].contiguous(), c.S, codes, norms, values,
                                            table, _i32([L - n + i + 1]), L).float()[0]
        # both round weights and outputs to bf16, and values are N(0, 1)
        assert (got[i] - step).abs().max() <= 4 * UB


def test_chunk_attention_nan_and_inf_stay_in_their_rows():
    c = Cache([150], 1, 64, 128, 32, seed=13)
    for n in (4, 320):
        c.lens[0] = 150
        Q = _randn(14, n, 2, 64)
        ref = run_chunk(c, Q, [n])
        Q[1, 0, 3], Q[2, 1, 5] = math.nan, math.inf
        got = run_chunk(c, Q, [n])
        same = torch.ones(n, 2, dtype=torch.bool)
        same[1, 0] = same[2, 1] = False
        assert torch.equal(got[same.to(DEV)], ref[same.to(DEV)])
        seen = [150 - n + i + 1 > 0 for i in (1, 2)]
        if seen[0]:
            assert torch.isnan(got[1, 0]).all()
        if seen[1]:
            assert not torch.isfinite(got[2, 1].float()).any()
    # a masked key's norm may be anything: the last key is seen by the last row alone
    n = 4
    pg, sl = c.table[0, 149 // 32], 149 % 32
    for x in (math.nan, math.inf):
        Q = _randn(15, n, 2, 64)
        ref = run_chunk(c, Q, [n])
        old = c.norms[pg, 0, sl]
        c.norms[pg, 0, sl] = x
        got = run_chunk(c, Q, [n])
        c.norms[pg, 0, sl] = old
        assert torch.equal(got[:n - 1], ref[:n - 1])


@pytest.mark.parametrize("n", [4, 320])
@pytest.mark.parametrize("x", [math.nan, math.inf])
def test_chunk_attention_a_key_that_is_not_finite_shows_in_every_row_that_sees_it(n, x):
    """One key whose norm is not finite, at each place of a group of eight, in
    the first tile, in inner ones, where some rows see it and others do not, and
    last: rows that see it are NaN in all dims, the others as without it."""
    L, P = 600, 32
    c = Cache([L], 1, 64, 128, P, seed=13)
    Q = _randn(15, n, 2, 64)
    ref = run_chunk(c, Q, [n])
    assert torch.isfinite(ref.float()).all()
    for t in (*range(8), 130, 206, 207, L - n, L - n + 1, L - n // 2, L - 1):
        at = c.table[0, t // P], 0, t % P
        old = c.norms[at]
        c.norms[at] = x
        got = run_chunk(c, Q, [n])
        c.norms[at] = old
        sees = torch.arange(n) + L - n + 1 > t
        assert sees.any()
        assert torch.isnan(got[sees.to(DEV)].float()).all(), t
        assert torch.equal(got[~sees.to(DEV)], ref[~sees.to(DEV)]), t


def test_chunk_attention_many_rows_with_queries_that_are_not_finite():
    """NaN and infinite queries among many rows, each over keys that it sees."""
    n, L = 320, 600
    c = Cache([L], 1, 64, 128, 32, seed=13)
    Q = _randn(14, n, 2, 64)
    ref = run_chunk(c, Q, [n])
    Q[1, 0, 3], Q[2, 1, 5] = math.nan, math.inf
    got = run_chunk(c, Q, [n])
    same = torch.ones(n, 2, dtype=torch.bool)
    same[1, 0] = same[2, 1] = False
    assert torch.equal(got[same.to(DEV)], ref[same.to(DEV)])
    assert torch.isnan(got[~same.to(DEV)].float()).all()
    # a row whose only key scores -inf
    c.lens[0] = n
    khat = c.keys(0, 0)[0][0]
    j = int(np.argmin(khat))
    assert khat[j] < 0
    Q[:] = 1.0
    Q[0, :, j] = math.inf
    got = run_chunk(c, Q, [n])
    assert torch.isnan(got[0].float()).all() and torch.isfinite(got[1:].float()).all()


def test_chunk_attention_bad_lengths_and_pages_are_reported():
    c = Cache([100, 70], 1, 64, 64, 32, seed=16)
    Q = _randn(17, 8, 1, 64)
    codes, norms, values, table = c.dev()
    ref = run_chunk(c, Q, [4, 4])
    call = lambda lens, cu, tab=table, max_len=100: jl.jl_chunk_attention_paged(
        Q, c.S, codes, norms, values, tab, _i32(lens), _i32(cu), max_len,
        out=torch.zeros(8, 1, 64, dtype=torch.bfloat16, device=DEV))
    for lens, cu in (([100, 101], [0, 4, 8]), ([100, -1], [0, 4, 8]), ([100, 70], [0, 4, 9]),
                     ([100, 70], [0, 4, 3]), ([100, 70], [-1, 4, 8])):
        got = call(lens, cu)
        assert jl.jl_device_error() == jl.JL_DERR_DECODE_PLAN, (lens, cu)
        if cu[:2] == [0, 4]:
            assert torch.equal(got[:4], ref[:4])                # the other sequence is served
    # rows given to two sequences: the later one is dropped
    bad3 = jl.jl_chunk_attention_paged(Q, c.S, codes, norms, values, table[[0, 1, 0]].contiguous(),
                                       _i32([100, 70, 100]), _i32([0, 8, 2, 8]), 100)
    torch.cuda.synchronize()
    assert bad3.shape == Q.shape and jl.jl_device_error() == jl.JL_DERR_DECODE_PLAN
    for entry in (-1, codes.shape[0], 2 ** 31 - 1):
        tab = table.clone()
        tab[1, 1] = entry
        got = call([100, 70], [0, 4, 8], tab)
        assert jl.jl_device_error() == jl.JL_DERR_PAGE
        assert torch.equal(got[:4], ref[:4])
    assert torch.equal(call([100, 70], [0, 4, 8]), ref) and jl.jl_device_error() == 0


@pytest.mark.parametrize("n", [7, 200])
def test_chunk_attention_graphs_streams_and_workspaces(n):
    c = Cache([400, 350], 2, 128, 128, 64, seed=18)
    counts = [n, n]
    Qs = [_randn(20 + i, 2 * n, 4, 128, dtype=torch.bfloat16) for i in range(3)]
    refs = [run_chunk(c, q, counts) for q in Qs]
    codes, norms, values, table = c.dev()
    lens, cu = _i32(c.lens), _i32([0, n, 2 * n])
    need = jl.jl_chunk_attention_workspace_bytes(2 * n, 2, 4, 2, 400, 128, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)    # contents do not matter
    call = lambda q, out=None, **k: jl.jl_chunk_attention_paged(q, c.S, codes, norms, values, table,
                                                                lens, cu, 400, out=out, **k)
    assert torch.equal(call(Qs[0], workspace=ws), refs[0])
    with pytest.raises(jl.JLError) as e:
        call(Qs[0], workspace=ws[:-256])
    assert e.value.status == jl.JL_ERR_WORKSPACE
    # two graphs over one workspace, replayed in turn with other queries
    q_in, outs, graphs = [q.clone() for q in Qs[:2]], [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for q in q_in:
        g, out = torch.cuda.CUDAGraph(), torch.zeros_like(refs[0])
        with torch.cuda.graph(g, stream=side):
            call(q, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for order in ((0, 1), (1, 0)):
        for i in order:
            graphs[i].replay()
    q_in[0].copy_(Qs[2])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], refs[2]) and torch.equal(outs[1], refs[1])
    # calls side by side on two streams, each with a workspace of its own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((call(Qs[0], stream=s1), call(Qs[1], stream=s2)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, refs[0]) and torch.equal(b, refs[1])
    raw = call(Qs[0], stream=s1.cuda_stream)                    # a stream as its handle
    torch.cuda.synchronize()
    assert torch.equal(raw, refs[0])


# --------------------------------------------------------------------------
# store

@pytest.mark.parametrize("W,cn,d", [(8, 1, 128), (2, 1, 64), (12, 2, 128), (3, 2, 64)])
def test_store(W, cn, d):
    Hkv, P, counts, before = 3, 32, [5, 0, 40, 1], [0, 10, 60, 31]
    N, pad = sum(counts), 2
    rng = _rng(1)
    tab = table_for([a + b for a, b in zip(before, counts)], P, 12, rng)
    one = () if cn == 1 else (2,)
    make = lambda lead, s: (_i32(rng.integers(-2 ** 31, 2 ** 31, size=(*lead, W))),
                            _randn(s, *lead, *one).half(),
                            _randn(s + 1, *lead, d, dtype=torch.bfloat16))
    pools = make((12, Hkv, P), 2)
    codes, norms, _ = make((N + pad, Hkv), 4)
    V = _randn(6, N + pad, 2 * Hkv + 1, d, dtype=torch.bfloat16)[:, Hkv:2 * Hkv]
    want = [t.clone() for t in pools]
    r = 1
    for b, n in enumerate(counts):
        for i in range(n):
            pg, sl = tab[b, (before[b] + i) // P], (before[b] + i) % P
            for w, x in zip(want, (codes, norms, V)):
                w[pg, :, sl] = x[r]
            r += 1
    cu = 1 + np.concatenate([[0], np.cumsum(counts)])
    jl.jl_store_paged(codes, norms, V, _i32(cu), *pools, _i32(tab), _i32(before))
    for w, p in zip(want, pools):
        assert torch.equal(w, p)
    # no row, no sequence
    jl.jl_store_paged(codes[:0], norms[:0], V[:0], _i32([0] * 5), *pools, _i32(tab), _i32(before))
    for w, p in zip(want, pools):
        assert torch.equal(w, p)


def test_store_bad_pages_skip_and_report():
    Hkv, P, d = 2, 32, 64
    pools = (torch.zeros(4, Hkv, P, 2, dtype=torch.int32, device=DEV),
             torch.zeros(4, Hkv, P, dtype=torch.float16, device=DEV),
             torch.zeros(4, Hkv, P, d, dtype=torch.bfloat16, device=DEV))
    codes = torch.ones(6, Hkv, 2, dtype=torch.int32, device=DEV)
    norms = torch.ones(6, Hkv, dtype=torch.float16, device=DEV)
    V = torch.ones(6, Hkv, d, dtype=torch.bfloat16, device=DEV)
    for tab, before in (([[0, 4]], [29]), ([[0, -1]], [29]), ([[0]], [29]), ([[0, 1]], [-3]),
                        ([[0, 1]], [61])):
        for p in pools:
            p.zero_()
        jl.jl_store_paged(codes, norms, V, _i32([0, 6]), *pools, _i32(tab), _i32(before))
        assert jl.jl_device_error() == jl.JL_DERR_PAGE
        assert pools[0].sum() == 3 * Hkv * 2 and pools[2].float().sum() == 3 * Hkv * d


# --------------------------------------------------------------------------
# accumulated weights

@pytest.mark.parametrize("B,Hq,Hkv,T", [(1, 1, 1, 1), (3, 6, 2, 77), (2, 8, 8, 4096),
                                        (2, 16, 1, 9000), (1, 4, 2, 70001)])
@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
def test_accumulate(B, Hq, Hkv, T, decay):
    rng = _rng(T)
    lens = rng.integers(0, T + 1, size=B)
    lens[0] = T
    scores = _randn(1, B, Hq, T) * 20
    for b in range(B):
        scores[b, :, lens[b]:] = math.nan                       # never read into a result
    mass = _randn(2, B, Hkv, T).abs()
    scale = 0.11
    out = torch.full_like(mass, 5.0)
    m_in = torch.full_like(mass, math.nan) if decay == 0.0 else mass
    got = jl.jl_accumulate_attention(scores, m_in, _i32(lens), scale, decay=decay, out=out)
    assert got is out
    for b, L in enumerate(lens):
        assert torch.all(out[b, :, L:] == 5.0)
        if L == 0:
            continue
        x = H.f64(scores[b, :, :L]) * scale
        w = np.exp(x - x.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        W = w.reshape(Hkv, Hq // Hkv, L).sum(1)
        old = decay * H.f64(mass[b, :, :L])
        # exponents in fp32 (four roundings of their size, in the statistics
        # and in the weight), exp2's 2 ulp each, sums of up to T / 2048 + 64
        tol = W * U32 * (8 * (np.abs(x).max() * 1.5 + 1) + 80 + T / 1024) + 2 * U32 * (old + W)
        assert np.all(np.abs(H.f64(out[b, :, :L]) - (old + W)) <= tol + 1e-37)
    if decay:
        again = jl.jl_accumulate_attention(scores, mass, _i32(lens), scale, decay=decay)
        assert again is mass                                     # in place
        for b, L in enumerate(lens):
            assert torch.equal(mass[b, :, :L], out[b, :, :L])


def test_accumulate_masked_rows_and_lengths():
    B, Hq, Hkv, T = 2, 4, 2, 100
    scores = _randn(3, B, Hq, T)
    scores[0, 0] = -math.inf                                     # a head with nothing
    scores[0, 1, ::2] = -math.inf
    scores[1, 3] = torch.finfo(torch.float32).min                # the lowest value, everywhere
    out = jl.jl_accumulate_attention(scores, torch.zeros(B, Hkv, T, device=DEV), _i32([T, T]), 1.0)
    assert torch.isfinite(out).all()
    assert abs(out[0, 0].sum().item() - 1) < 1e-5 and torch.all(out[0, 0, ::2] == 0)
    assert abs(out[1, 1].sum().item() - 2) < 1e-5
    out = jl.jl_accumulate_attention(scores, torch.zeros(B, Hkv, T, device=DEV), _i32([-1, T + 1]),
                                     1.0)
    assert jl.jl_device_error() == jl.JL_DERR_DECODE_PLAN
    assert torch.all(out[0] == 0) and abs(out[1, 0].sum().item() - 2) < 1e-5


@pytest.mark.parametrize("T", [1, 5, 77, 2000, 2001, 70001])
@pytest.mark.parametrize("x", [math.nan, math.inf])
def test_accumulate_scores_that_are_not_finite_show_in_the_whole_row(T, x):
    """As a softmax has it: one such score, and none of its head's weights is a
    number, however few keys the thread that meets it has besides."""
    for t in {0, T // 2, T - 1}:
        scores = _randn(5, 1, 4, T)
        ref = jl.jl_accumulate_attention(scores, torch.zeros(1, 2, T, device=DEV), _i32([T]), 1.0)
        scores[0, 1, t] = x
        out = jl.jl_accumulate_attention(scores, torch.zeros(1, 2, T, device=DEV), _i32([T]), 1.0)
        assert torch.isnan(out[0, 0]).all(), t
        assert torch.equal(out[0, 1], ref[0, 1])


@pytest.mark.parametrize("scale,values", [
    (0.0, (0.0, torch.finfo(torch.float32).min)),               # uniform, whatever the scores
    (0.0, (3e38, -3e38)),
    (1e-38, (3e38, -3e38)),                                     # logits 3 and -3
    (-1e-38, (3.4e38, -3.4e38, 1e38)),
    (1.0, (1.0, torch.finfo(torch.float32).min)),               # an additive mask
    (3e38, (1.0, 0.0)),                                         # the larger ones alone
])
def test_accumulate_scales_and_scores_of_any_size(scale, values):
    T = 600
    scores = torch.tensor(values, device=DEV).repeat(T)[:T].view(1, 1, T).contiguous()
    out = jl.jl_accumulate_attention(scores, torch.zeros(1, 1, T, device=DEV), _i32([T]), scale)
    x = H.f64(scores[0, 0]) * float(np.float32(scale))
    w = np.exp(x - x.max())
    w /= w.sum()
    # as in test_accumulate; a scale of 0 counts as 2^-149, which makes a
    # difference of at most 2^129 logits of 2^-20
    tol = w * (U32 * (8 * (min(np.abs(x).max(), 100.0) * 1.5 + 1) + 80) +
               (2 * 2.0 ** -20 if scale == 0 else 0))
    assert np.all(np.abs(H.f64(out[0, 0]) - w) <= tol + 1e-37)


# --------------------------------------------------------------------------
# eviction

def evict64(mass, L, keep, recent, sink):
    if L <= keep:
        return np.arange(L)
    cand = np.arange(sink, L - recent)
    rank = np.where(np.isnan(mass[cand]), -np.inf, mass[cand])
    nan_last = np.isnan(mass[cand])
    order = sorted(range(len(cand)), key=lambda i: (nan_last[i], -rank[i], i))
    best = cand[order[:keep - recent - sink]]
    return np.sort(np.concatenate([np.arange(sink), best, np.arange(L - recent, L)]))


@pytest.mark.parametrize("lens,keep,recent,sink,W,cn,d,P", [
    ([100, 33, 0, 64], 40, 8, 4, 8, 1, 128, 32),
    ([1], 1, 0, 0, 2, 1, 64, 32),
    ([5000, 4999], 777, 100, 3, 12, 2, 64, 64),
    ([20000], 9001, 0, 0, 4, 1, 64, 128),
    ([90, 91], 90, 40, 50, 3, 2, 128, 96),                       # nothing is chosen by mass
    ([50, 60], 100, 10, 2, 4, 1, 64, 32),                        # everything stays
])
def test_evict(lens, keep, recent, sink, W, cn, d, P):
    B, Hkv, T = len(lens), 2, max(lens) + 3
    rng = _rng(keep)
    new = [min(L, keep) for L in lens]
    need = [sum(-(-x // P) for x in v) for v in (lens, new)]
    pages = sum(need) + 2
    both = table_for(lens + new, P, pages, rng, width=-(-max(T, keep) // P))
    src, dst = both[:B], both[B:]
    one = () if cn == 1 else (2,)
    pools = (_i32(rng.integers(-2 ** 31, 2 ** 31, size=(pages, Hkv, P, W))),
             _randn(1, pages, Hkv, P, *one).half(), _randn(2, pages, Hkv, P, d,
                                                           dtype=torch.bfloat16))
    mass = rng.standard_normal((B, Hkv, T)).astype(np.float32)
    mass[mass < -0.5] = 0.0                                      # ties, and both zeros
    mass[:, 1, ::7] = -0.0
    mass[:, 0, 5::11] = 0.25
    mass[:, 0, 1::50], mass[:, 1, 2::60], mass[:, 1, 3::70] = np.nan, np.inf, -np.inf
    want = [t.clone() for t in pools]
    m = torch.from_numpy(mass).to(DEV)
    idx, om, ol = jl.jl_evict_paged(m, _i32(lens), keep, *pools, _i32(src), _i32(dst),
                                    recent=recent, sink=sink)
    assert ol.tolist() == new
    for b, L in enumerate(lens):
        for h in range(Hkv):
            t = evict64(mass[b, h], L, keep, recent, sink)
            assert np.array_equal(idx[b, h, :len(t)].cpu().numpy(), t)
            assert torch.all(idx[b, h, len(t):] == -1) and torch.all(om[b, h, len(t):] == 0)
            assert np.array_equal(om[b, h, :len(t)].cpu().numpy(), mass[b, h, t], equal_nan=True)
            j = np.arange(len(t))
            for w in want:
                w[dst[b, j // P], h, j % P] = w[src[b, t // P], h, t % P]
    for w, p in zip(want, pools):
        assert torch.equal(w, p)                                 # all other rows as they were


def test_evict_long_rows_read_from_memory():
    """More keys than the blocks of a cluster can hold in shared memory."""
    L, keep, P = 420000, 1000, 128
    mass = _randn(3, 1, 1, L)
    pages = -(-L // P) + -(-keep // P)
    pools = (torch.arange(pages * P, dtype=torch.int32, device=DEV).view(pages, 1, P, 1),
             torch.zeros(pages, 1, P, dtype=torch.float16, device=DEV),
             torch.zeros(pages, 1, P, 64, dtype=torch.bfloat16, device=DEV))
    tab = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    src, dst = tab[:, :-(-L // P)].contiguous(), tab[:, -(-L // P):].contiguous()
    idx, om, _ = jl.jl_evict_paged(mass, _i32([L]), keep, *pools, src, dst, recent=10, sink=1)
    want = evict64(mass[0, 0].cpu().numpy(), L, keep, 10, 1)
    assert np.array_equal(idx[0, 0].cpu().numpy(), want)
    assert np.array_equal(pools[0].view(-1)[-(-L // P) * P:][:keep].cpu().numpy(), want)


def test_evict_bad_lengths_and_pages_are_reported():
    P, d, keep = 32, 64, 20
    pools = (torch.ones(6, 1, P, 2, dtype=torch.int32, device=DEV),
             torch.ones(6, 1, P, dtype=torch.float16, device=DEV),
             torch.ones(6, 1, P, d, dtype=torch.bfloat16, device=DEV))
    mass = _randn(4, 1, 1, 50)
    for lens, src, dst, code in (([51], [[0, 1]], [[2]], jl.JL_DERR_DECODE_PLAN),
                                 ([-1], [[0, 1]], [[2]], jl.JL_DERR_DECODE_PLAN),
                                 ([50], [[0, 6]], [[2]], jl.JL_DERR_PAGE),
                                 ([50], [[0, 1]], [[-1]], jl.JL_DERR_PAGE)):
        _, _, ol = jl.jl_evict_paged(mass, _i32(lens), keep, *pools, _i32(src), _i32(dst))
        assert jl.jl_device_error() == code
        assert ol.item() == max(0, min(lens[0], keep))


# --------------------------------------------------------------------------
# where they can go wrong

@pytest.mark.parametrize("n", [1, 5, 300])
def test_chunk_attention_of_one_key_is_its_value(n):
    """A sequence of one key, and the last of n rows that alone sees it: the
    weight cancels in full, so the value comes out as it went in."""
    c = Cache([1, 1], 2, 128, 256, 32, seed=13)
    Q = _randn(14, n + 1, 8, 128, dtype=torch.bfloat16)
    got = run_chunk(c, Q, [n, 1])
    for b, row in ((0, n - 1), (1, n)):
        want = c.values[c.table[b, 0], :, 0].to(DEV).repeat_interleave(4, 0)
        assert torch.equal(got[row], want)
    assert torch.all(got[:n - 1] == 0)


@pytest.mark.parametrize("n", [5, 200])
def test_offsets_beyond_32_bits(n):
    """The last pages of pools whose values pass 2^32 entries: stored, attended
    over, evicted."""
    P, d, m, L, keep = 128, 128, 64, 700, 200
    c = Cache([L], 1, d, m, P, seed=15, extra=2)
    used = c.codes.shape[0]
    first = 2 ** 32 // (P * d) + 5 - used
    pools = [torch.empty(first + used, *x.shape[1:], dtype=x.dtype, device=DEV)
             for x in c.dev()[:3]]
    for p, x in zip(pools, c.dev()[:3]):
        p[first:] = x
    assert pools[2].numel() > 2 ** 32
    table = np.where(c.table >= 0, c.table + first, -1)
    free = first + np.setdiff1d(np.arange(used), c.table)
    # the last n keys are taken out and stored anew
    t = np.arange(L - n, L)
    at = torch.from_numpy(table[0, t // P]).long(), slice(None), torch.from_numpy(t % P)
    new = [p[at[0].to(DEV), 0, at[2].to(DEV)].unsqueeze(1).contiguous() for p in pools]
    for p in pools:
        p[at[0].to(DEV), 0, at[2].to(DEV)] = 0
    jl.jl_store_paged(*new, _i32([0, n]), *pools, _i32(table), _i32([L - n]))
    for p, x in zip(pools, c.dev()[:3]):
        assert torch.equal(p[first:].view(torch.uint8), x.view(torch.uint8))
    Q = _randn(16, n, 2, d, dtype=torch.bfloat16)
    got = jl.jl_chunk_attention_paged(Q, c.S, *pools, _i32(table), _i32([L]), _i32([0, n]), L)
    assert torch.equal(got, run_chunk(c, Q, [n]))
    mass = _randn(17, 1, 1, L)
    idx, _, _ = jl.jl_evict_paged(mass, _i32([L]), keep, *pools, _i32(table), _i32(free[None]),
                                  recent=7, sink=3)
    kept = evict64(mass[0, 0].cpu().numpy(), L, keep, 7, 3)
    assert np.array_equal(idx[0, 0].cpu().numpy(), kept)
    j = np.arange(keep)
    for p in pools:
        a = p[torch.from_numpy(free[j // P]).to(DEV), 0, torch.from_numpy(j % P).to(DEV)]
        b = p[torch.from_numpy(table[0, kept // P]).long().to(DEV), 0,
              torch.from_numpy(kept % P).to(DEV)]
        assert torch.equal(a, b)


def test_rotary_and_weights_beyond_32_bits():
    """Strides and tensors past 2^31 entries."""
    tok, n, H_, d = 2 ** 30 + 64, 4, 2, 64
    big = torch.empty(3 * tok + H_ * d, dtype=torch.bfloat16, device=DEV)
    Q = big.as_strided((n, H_, d), (tok, d, 1))
    Q.copy_(_randn(1, n, H_, d, dtype=torch.bfloat16))
    f = jl.jl_rotary_frequencies(d)
    pos = _i32([0, 7, 2 ** 31 - 1, -5])
    want = jl.jl_rotary(Q.contiguous(), pos, f)
    assert torch.equal(jl.jl_rotary(Q, pos, f), want)
    assert jl.jl_rotary(Q, pos, f, out_q=Q) is Q and torch.equal(Q, want)
    del big, Q
    Hq, T = 9, 2 ** 28
    scores = torch.empty(1, Hq, T, device=DEV)
    scores.normal_(generator=torch.Generator(DEV).manual_seed(2))
    mass = torch.zeros(1, Hq, T, device=DEV)
    jl.jl_accumulate_attention(scores, mass, _i32([T]), 0.5)
    alone = torch.zeros(1, 1, T, device=DEV)
    jl.jl_accumulate_attention(scores[:, -1:].contiguous(), alone, _i32([T]), 0.5)
    # both rows are split over as many blocks, so the sums have one order
    assert torch.equal(mass[:, -1:], alone)
    # a thread sums 2^16 of the weights, each step rounded by 2^-24 of the sum
    assert abs(mass[0, -1].double().sum().item() - 1) < 2.0 ** -8


def test_strides_along_a_single_token_or_head_are_not_read():
    Hkv, P, d = 1, 32, 64
    pools = (torch.zeros(2, Hkv, P, 2, dtype=torch.int32, device=DEV),
             torch.zeros(2, Hkv, P, dtype=torch.float16, device=DEV),
             torch.zeros(2, Hkv, P, d, dtype=torch.bfloat16, device=DEV))
    V = _randn(1, 1, Hkv, d, dtype=torch.bfloat16).as_strided((1, Hkv, d), (3, 5, 1))
    codes, norms = torch.ones(1, 1, 2, dtype=torch.int32, device=DEV), torch.ones(
        1, 1, dtype=torch.float16, device=DEV)
    jl.jl_store_paged(codes, norms, V, _i32([0, 1]), *pools, _i32([[1]]), _i32([3]))
    assert torch.equal(pools[2][1, 0, 3], V[0, 0]) and pools[0].sum() == 2
    f = jl.jl_rotary_frequencies(d)
    assert torch.equal(jl.jl_rotary(V, _i32([9]), f), jl.jl_rotary(V.contiguous(), _i32([9]), f))


@pytest.mark.parametrize("n,Hq,Hkv,d,rot", [(1, 65536, 0, 2, 2), (2, 2500, 1700, 6, 4),
                                            (1300, 70, 3, 1024, 1024)])
def test_rotary_of_many_heads(n, Hq, Hkv, d, rot):
    """More heads than a block takes at once, and the widest head."""
    Q = _randn(2, n, Hq, d, dtype=torch.bfloat16)
    K = _randn(3, n, Hkv, d, dtype=torch.bfloat16) if Hkv else None
    pos, freq = _i32(np.arange(n) * 1000 + 7), jl.jl_rotary_frequencies(rot)
    got = jl.jl_rotary(Q, pos, freq, K=K)
    for y, x in ((got[0], Q), (got[1], K)) if Hkv else ((got, Q),):
        some = sorted({0, n // 2, n - 1})                       # (in float64, not all of them)
        check_rotary(y[some], x[some], pos[some], freq, False, False, 1.0)
        assert torch.equal(y[:, -1:], jl.jl_rotary(x[:, -1:], pos, freq))


@pytest.mark.parametrize("G", [1, 2, 3, 511, 512])
def test_accumulate_heads_of_a_group(G):
    T, Hkv = 130, 2
    scores = _randn(6, 1, G * Hkv, T)
    out = jl.jl_accumulate_attention(scores, torch.zeros(1, Hkv, T, device=DEV), _i32([T]), 0.7)
    x = H.f64(scores[0]) * float(np.float32(0.7))
    w = np.exp(x - x.max(-1, keepdims=True))
    w = (w / w.sum(-1, keepdims=True)).reshape(Hkv, G, T).sum(1)
    # as in test_accumulate, with a sum over the group's heads
    tol = w * U32 * (8 * (np.abs(x).max() * 1.5 + 1) + 80 + G)
    assert np.all(np.abs(H.f64(out[0]) - w) <= tol)


@pytest.mark.parametrize("W", [64, 33, 17])
@pytest.mark.parametrize("d", [64, 128])
def test_store_and_evict_codes_of_more_words_than_a_key_has_lanes(W, d):
    Hkv, P, n, keep = 2, 32, 75, 41
    rng = _rng(W)
    pools = (torch.zeros(6, Hkv, P, W, dtype=torch.int32, device=DEV),
             torch.zeros(6, Hkv, P, 2, dtype=torch.float16, device=DEV),
             torch.zeros(6, Hkv, P, d, dtype=torch.bfloat16, device=DEV))
    codes = _i32(rng.integers(-2 ** 31, 2 ** 31, size=(n, Hkv, W)))
    norms, V = _randn(7, n, Hkv, 2).half(), _randn(8, n, Hkv, d, dtype=torch.bfloat16)
    src, dst = np.array([[4, 0, 3]]), np.array([[1, 5]])
    jl.jl_store_paged(codes, norms, V, _i32([0, n]), *pools, _i32(src), _i32([0]))
    t = np.arange(n)
    for p, x in zip(pools, (codes, norms, V)):
        assert torch.equal(p[src[0, t // P], :, t % P], x)
        assert torch.all(p[[1, 2, 5]] == 0)
    mass = _randn(9, 1, Hkv, n)
    idx, _, _ = jl.jl_evict_paged(mass, _i32([n]), keep, *pools, _i32(src), _i32(dst), recent=3)
    for h in range(Hkv):
        t = evict64(mass[0, h].cpu().numpy(), n, keep, 3, 0)
        assert np.array_equal(idx[0, h].cpu().numpy(), t)
        j = np.arange(keep)
        for p, x in zip(pools, (codes, norms, V)):
            assert torch.equal(p[dst[0, j // P], h, j % P], x[t, h])


# --------------------------------------------------------------------------
# the operators together

@pytest.mark.parametrize("n", [3, 200])
def test_a_step_captured_and_on_another_stream(n):
    """Rotary, quantizer, store, attention, weights and eviction as one graph,
    replayed on other inputs, and on a stream of their own: bit for bit what the
    calls give one by one."""
    Hq, Hkv, d, m, P, L, keep = 8, 2, 64, 128, 32, 200 + n, 64
    S, freq = jl.jl_sketch_init(m, d, 0), jl.jl_rotary_frequencies(d)
    pages = -(-L // P) + keep // P
    i32 = lambda *a: _i32(np.array(a))
    table = _i32(np.arange(-(-L // P))[None])
    spare = _i32(np.arange(-(-L // P), pages)[None])
    inputs = [(_randn(80 + s, n, Hq + 2 * Hkv, d, dtype=torch.bfloat16), _randn(90 + s, 1, Hq, L))
              for s in range(3)]

    def fresh():
        g = _rng(5)
        return (_i32(g.integers(-2 ** 31, 2 ** 31, size=(pages, Hkv, P, m // 32))),
                _randn(6, pages, Hkv, P).abs().half() * 8,
                _randn(7, pages, Hkv, P, d, dtype=torch.bfloat16))

    def step(qkv, scores, pools, mass, **k):
        q, kk = jl.jl_rotary(qkv[:, :Hq], pos, freq, K=qkv[:, Hq:Hq + Hkv], **k)
        signs, norms = jl.jl_quantize_keys(kk, S, **k)
        jl.jl_store_paged(signs.view(n, Hkv, -1), norms.view(n, Hkv), qkv[:, Hq + Hkv:], cu,
                          *pools, table, before, **k)
        out = jl.jl_chunk_attention_paged(q, S, *pools, table, lens, cu, L, **k)
        jl.jl_accumulate_attention(scores, mass, lens, 0.3, decay=0.9, **k)
        return out, mass, *jl.jl_evict_paged(mass, lens, keep, *pools, table, spare, recent=8,
                                             sink=2, **k)

    pos, cu = _i32(200 + np.arange(n)), i32(0, n)
    before, lens = i32(200), i32(L)
    mass0 = _randn(8, 1, Hkv, L).abs()
    want = []
    for x in inputs:
        pools, mass = fresh(), mass0.clone()
        want.append([t.clone() for t in (*step(*x, pools, mass), *pools)])
    # a graph
    pools, mass = fresh(), mass0.clone()
    x_in = [t.clone() for t in inputs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*x_in, pools, mass)
    for i in (1, 2, 0, 0):
        for a, b in zip((*x_in, *pools, mass), (*inputs[i], *fresh(), mass0)):
            a.copy_(b)
        graph.replay()
        for a, b in zip((*outs, *pools), want[i]):
            assert torch.equal(a, b), i
    # another stream, given to each call, while the current one is at work
    side = torch.cuda.Stream()
    for i in range(3):
        pools, mass = fresh(), mass0.clone()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(2_000_000)                            # (about a millisecond)
        got = step(*inputs[i], pools, mass, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip((*got, *pools), want[i]):
            assert torch.equal(a, b), i
    torch.cuda.synchronize()
    del graph


def test_serving_loop():
    """A prompt in pieces, drafted tokens, decode steps and an eviction over one
    paged cache: every attention output against float64 on the codes that the
    cache then holds, and the cache after the eviction against the kept keys."""
    B, Hq, Hkv, d, m, P, max_len = 2, 8, 2, 128, 256, 64, 512
    G = Hq // Hkv
    S = jl.jl_sketch_init(m, d, 0)
    freq = jl.jl_rotary_frequencies(d)
    pages = 2 * B * (max_len // P)
    pools = (torch.zeros(pages, Hkv, P, m // 32, dtype=torch.int32, device=DEV),
             torch.full((pages, Hkv, P), math.nan, dtype=torch.float16, device=DEV),
             torch.full((pages, Hkv, P, d), math.nan, dtype=torch.bfloat16, device=DEV))
    perm = _rng(0).permutation(pages).astype(np.int32)
    table = _i32(perm[:pages // 2].reshape(B, -1))
    spare = _i32(perm[pages // 2:].reshape(B, -1))
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)

    def view(lens_now, tab):
        c = Cache.__new__(Cache)
        c.lens, c.Hkv, c.d, c.m, c.P, c.S = lens_now.tolist(), Hkv, d, m, P, S
        c.codes, c.norms = H.u32(pools[0]), pools[1].cpu().numpy()
        c.values, c.table = pools[2].cpu(), tab.cpu().numpy()
        return c

    for step, counts in enumerate(([200, 150], [37, 90], [4, 1])):
        N = sum(counts)
        qkv = _randn(30 + step, N, Hq + 2 * Hkv, d, dtype=torch.bfloat16)
        cu = _i32(np.concatenate([[0], np.cumsum(counts)]))
        pos = torch.cat([lens[b] + torch.arange(n, device=DEV, dtype=torch.int32)
                         for b, n in enumerate(counts)])
        q, k = jl.jl_rotary(qkv[:, :Hq], pos, freq, K=qkv[:, Hq:Hq + Hkv])
        signs, norms = jl.jl_quantize_keys(k, S)
        jl.jl_store_paged(signs.view(N, Hkv, -1), norms.view(N, Hkv), qkv[:, Hq + Hkv:], cu,
                          *pools, table, lens)
        lens += cu.diff()
        out = jl.jl_chunk_attention_paged(q, S, *pools, table, lens, cu, max_len)
        c = view(lens, table)
        # the rows' codes are the quantizer's, wherever they lie
        t = c.lens[0] - 1
        assert np.array_equal(c.codes[c.table[0, t // P], :, t % P],
                              H.u32(signs.view(N, Hkv, -1)[counts[0] - 1]))
        check_chunk(c, q, counts, out, d ** -0.5)

    mass = torch.zeros(B, Hkv, max_len, device=DEV)
    for step in range(3):
        q, kn, vn = (_randn(50 + 3 * step + i, B, h, d, dtype=torch.bfloat16)
                     for i, h in enumerate((Hq, Hkv, Hkv)))
        q, kn = jl.jl_rotary(q, lens, freq, K=kn)
        _, sc = jl.jl_decode_attention_paged(q, S, *pools, table, lens, max_len, K_new=kn,
                                             V_new=vn, want_scores=True)
        lens += 1
        jl.jl_accumulate_attention(sc, mass, lens, d ** -0.5)
    for b in range(B):                                           # every head gave weight 1 a step
        assert torch.all((mass[b, :, :lens[b]].sum(-1) - 3 * G).abs() < 1e-3)
    keep = 100
    idx, kept, new = jl.jl_evict_paged(mass, lens, keep, *pools, table, spare, recent=16, sink=4)
    assert new.tolist() == [keep] * B
    before, after = view(lens, table), view(new, spare)
    for b in range(B):
        for h in range(Hkv):
            t = idx[b, h].cpu().numpy()
            assert np.array_equal(t, evict64(mass[b, h].cpu().numpy(), int(lens[b]), keep, 16, 4))
            for x, y in zip(before.keys(b, h), after.keys(b, h)):
                assert np.array_equal(x[t], y)
    # and decoding goes on, over the kept keys
    q = _randn(70, B, Hq, d, dtype=torch.bfloat16)
    out = jl.jl_decode_attention_paged(q, S, *pools, spare, new, max_len)
    ref = chunk64(after, q, [1, 1], d ** -0.5)
    for (r, h), (o, tol) in ref.items():
        # the decode kernel's projections carry 16 bits: inside the same bounds
        assert np.all(np.abs(H.f64(out[r, h]) - o) <= tol + 2 * UB)
    assert jl.jl_device_error() == 0


def test_serving_operators_under_index_checks():
    """These tests once more on the index-checking build: no kernel computes an
    index outside the extents that the call's shapes give its buffers (every
    test ends with the device error word clear)."""
    import os
    import subprocess
    import sys

    if jl.jl_build_flags() & jl.JL_BUILD_INDEX_CHECKS:
        return                                                   # this is that run
    from bit_jl_key_b200 import build
    lib = build.build(debug_index=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p",
                        "no:cacheprovider", os.path.abspath(__file__)],
                       env=dict(os.environ, JLKEY_LIBRARY=lib), capture_output=True, text=True,
                       timeout=900, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
