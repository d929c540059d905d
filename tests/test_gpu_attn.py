"""GPU parity of the attention-side operators against the 64-bit oracle (oracle/attn.py):
norm and rotation, the 4-bit cache, attention over it, and the three between two GEMVs.

Tolerances, from the arithmetic (u = 2^-24, a rounding to bf16 at most 2^-8 relative):

rotation  cos and sin: the fraction of a turn is rounded once (2^-26 turns = 2 pi 2^-26 rad <
          2^-23.3) and sincospi is within 2 ulp (2^-23): below 2^-22 in all.  The two products
          and the sum round three times, (|a| + |b|) 3 u.  Together (|a| + |b|) 2^-21.3; taken
          as 2^-21.  With a norm a term of the sum of squares passes at most 14 roundings (8 in a lane,
          one to join its two sums, 5 shuffles), which the root halves to 7 u; the mean and the sum with
          eps add 1 u, the reciprocal root 4 u (2 ulp), two products 2 u: below 16 u relative, 2^-20, in
          all (|a| + |b|) 2^-19.
cache     codes, steps and low ends are equal bit for bit (one rounding after another, in the
          same order); read back, fl32(m + s c) is exact and bf16 rounds that once more.
attention few rows: x_t = scale * q.k_t is summed in fp32 on codes 0 .. 15: D / 8 sums of 16 products,
          each sum and the operations after it rounded by at most 2^-23 of the largest partial result;
          |dx| <= |scale| * sum|q| * 2^-23 * (143 * max s * (D / 8 + 4) + 3 (max|m| + 136 max s))
          covers it (143 and 136 instead of 15: room of a factor of nine).  p s is rounded to fp16: 2^-11 of
          sum p s c <= 15 max s_v.
          tiles: keys are rounded to fp16, 2^-11 of each: |dx| <= |scale| * sum|q| * max|k| * 2^-11 more;
          values and probabilities likewise, 2^-11 of max|v| each (what of them is below fp16's normal
          range is off by 2^-18 of the page's largest key, 2^-17 of the largest value: below that).
          A probability is off by |dx| and by the exponential's 2^-21, so the output by 2 |dx| + 2^-20
          times max |v|; fp32 sums over L tokens by L 2^-23 of max|v| (L <= 2000: 2^-12).  The bound
          takes 2^-8 * 8 max s_v + 2^-12 max|v| for the roundings of p and v: 2^-5 max s_v is above
          2^-11 * 15 max s_v, and, where a row of values has both signs (max|v| <= 15 max s_v), above the
          tiles' 2^-10 max|v| too.  The last rounding is 2^-8 |o|.

          The bound above takes the largest value of a whole sequence, seen or not.  row_bound counts what a
          row sees, each token with its probability p: with |v| and |k| a token's largest magnitudes,
              |do| <= sum p_t (2 |dx_t| + 2^-20 + L 2^-23) (|v_t| + |o|)   weights, in numerator and total
                      + sum p_t dv_t + L 2^-26 max p_t |v_t| + 2^-8 |o|.
          A weight is off by a factor within e^+-|dx| and the exponential's 2^-21; fp32 sums of L terms by
          L 2^-24, the tensor cores' truncated ones by twice that.
          few rows: |dx_t| as above with the token's own s and m; p s to fp16 is 2^-11 of it, times |c - 8| <= 8,
          and truncated sums of 16-token products with codes up to 15 (and 8 for the centre): dv_t =
          s_t (2^-11 8 + L / 16 2^-23 23).
          tiles: a key's or value's low end and the sum m + s c are each rounded to fp16, half a step of 2^-11
          each, or 2^-25 of units in which the largest of the token is at least 2^-14: 2^-10 of |k| or |v| in
          all; probabilities 2^-11: |dx_t| += |scale| sum|q| |k_t| 2^-10, dv_t = |v_t| (2^-10 + 2^-11).
          Products p s (p v) that are below fp16's normal range are off by 2^-25 where the row's largest is at
          least 2^5: 2^-30 of it for each token, times |c - 8| <= 8.  In the tiles P is off by 2^-25 where the
          largest is at least 2^9, and values are at most 2^-6, the largest's own at least 2^-14: 2^-26 of it.
"""
import ctypes

import numpy as np
import pytest
import torch

from bit_gemv_sherry_b200 import sherry as S
from oracle import attn as A

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def np_of(t):
    return t.float().cpu().numpy()


def bf16_randn(rng, shape, mag=1.0):
    return A.to_bf16((rng.standard_normal(shape) * mag).astype(np.float32))


# ----------------------------------------------------------------------------- rotation
def run_rope(T, hq, hk, D, R, src, dst, norm, inter, seed, far=131071, pad=0):
    rng = np.random.default_rng(seed)
    f = (500000.0 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)
    pos = rng.integers(-far if seed % 2 else 0, far + 1, T).astype(np.int32)
    pos[0] = far
    xs, ws, ins, outs = [], [], [], []
    for h in (hq, hk):
        x = bf16_randn(rng, (T, h, D), 3.0) if src == BF else (rng.standard_normal((T, h, D)) * 3).astype(np.float32)
        w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if norm else None
        big = torch.full((T, h * D + pad), float("nan"), dtype=src, device="cuda")
        big[:, :h * D] = torch.from_numpy(x).reshape(T, h * D).to(src)
        obig = torch.full((T, h * D + pad), 77.0, dtype=dst, device="cuda")
        xs.append(x), ws.append(w)
        ins.append(big[:, :h * D].unflatten(1, (h, D))), outs.append((obig, obig[:, :h * D].unflatten(1, (h, D))))
    dw = [None if w is None else torch.from_numpy(w).cuda() for w in ws]
    q, k = S.qk_norm_rope(ins[0], ins[1], torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), q_weight=dw[0],
                          k_weight=dw[1], eps=1e-5, interleaved=inter, q_out=outs[0][1], k_out=outs[1][1])
    for x, w, o, (obig, _), h in zip(xs, ws, (q, k), outs, (hq, hk)):
        ref = A.rope(x, w, pos, f, 1e-5, inter)
        y = x.astype(np.float64) if w is None else A.rope(x, w, pos, f[:0], 1e-5, inter)
        mag = np.abs(y)
        half = R // 2
        ia = slice(0, R, 2) if inter else slice(0, half)
        ib = slice(1, R, 2) if inter else slice(half, R)
        tol = mag.copy()
        tol[..., ia] = tol[..., ib] = mag[..., ia] + mag[..., ib]
        tol = tol * (2.0 ** -19 if norm else 2.0 ** -21)
        if dst == BF:
            tol = tol + np.abs(ref) * 2.0 ** -8
        err = np.abs(np_of(o).astype(np.float64) - ref)
        assert np.all(err <= tol), (err - tol).max()
        assert pad == 0 or torch.all(obig[:, h * D:] == 77.0)
    assert S.device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("src,dst", [(torch.float32, BF), (BF, BF), (torch.float32, torch.float32), (BF, torch.float32)])
@pytest.mark.parametrize("T,hq,hk,D,R,norm", [
    (1, 32, 8, 64, 64, False), (5, 3, 1, 128, 128, True), (130, 8, 2, 128, 64, True), (7, 5, 5, 64, 32, True),
])
def test_rope_matches_oracle(T, hq, hk, D, R, norm, src, dst, inter):
    run_rope(T, hq, hk, D, R, src, dst, norm, inter, seed=T + R)


@pytest.mark.parametrize("D,R", [(8, 8), (16, 8), (24, 24), (32, 16), (40, 40), (72, 72), (80, 40), (96, 96), (112, 8),
                                 (136, 136), (192, 128), (256, 256), (256, 64), (64, 0), (200, 144)])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_odd_head_sizes_and_strides(D, R, inter):
    run_rope(9, 7, 2, D, R, torch.float32, BF, D % 16 == 0, inter, seed=D, pad=16)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,R,src,dst,norm", [
    (2043, 3, 2, 64, 64, torch.float32, BF, True), (2041, 1, 0, 128, 64, BF, BF, True), (2042, 9, 3, 72, 40, BF, torch.float32, False),
    (1, 80, 9, 128, 128, torch.float32, BF, True), (2040, 17, 1, 16, 8, torch.float32, torch.float32, True),
    (3, 60, 1, 256, 248, BF, BF, True), (2043, 2, 2, 136, 56, BF, BF, False),
])
def test_rope_many_tokens_and_many_heads(T, hq, hk, D, R, src, dst, norm, inter):
    """About 2,000 tokens go four to a CTA, the last one not full; many heads take a warp several steps."""
    if hk:
        run_rope(T, hq, hk, D, R, src, dst, norm, inter, seed=T + D, pad=8)
    else:   # one side alone, against the same rows as the second side of two
        x = torch.randn(T, hq, D, device="cuda").to(src)
        w = torch.rand(D, device="cuda")
        pos = torch.arange(T, dtype=torch.int32, device="cuda")
        f = torch.rand(R // 2, device="cuda")
        q, _ = S.qk_norm_rope(x, None, pos, f, q_weight=w, interleaved=inter, out_dtype=dst)
        _, k = S.qk_norm_rope(torch.zeros_like(x), x, pos, f, k_weight=w, interleaved=inter, out_dtype=dst)
        few, _ = S.qk_norm_rope(x[-5:], None, pos[-5:], f, q_weight=w, interleaved=inter, out_dtype=dst)
        assert torch.equal(q, k) and torch.equal(q[-5:], few)


def test_rope_one_side_and_in_place():
    x = torch.randn(4, 6, 64, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    f = torch.rand(32, device="cuda")
    q, k = S.qk_norm_rope(x, None, pos, f, out_dtype=torch.float32)
    _, k2 = S.qk_norm_rope(None, x, pos, f, out_dtype=torch.float32)
    assert k is None and torch.equal(q, k2)
    y = x.clone()
    S.qk_norm_rope(y, None, pos, f, q_out=y)
    assert torch.equal(y, q)


def test_rope_zero_rows_and_nan_stay_in_their_row():
    x = torch.randn(3, 4, 64, device="cuda")
    x[1, 2] = 0
    x[0, 1, 5] = float("nan")
    w = torch.ones(64, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    q, _ = S.qk_norm_rope(x, None, pos, torch.rand(32, device="cuda"), q_weight=w, eps=1e-5)
    assert not q[1, 2].any()
    bad = torch.isnan(q).any(-1)
    assert bad[0, 1] and bad.sum() == 1


# ----------------------------------------------------------------------------- batches
class Batch:
    """Sequences in shuffled pages; unused slots, pages and table entries hold poison."""

    def __init__(self, ctx, new, H, D, seed, extra_rows=0, spare=2, wide=0):
        rng = self.rng = np.random.default_rng(seed)
        self.ctx, self.new, self.H, self.D = ctx, new, H, D
        need = [(c + 63) // 64 for c in ctx]
        self.width = max(max(need) + 1, 2, wide)
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(ctx), self.width), -7, np.int32)
        self.table[:, 1::2] = 1 << 30
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_rows
        self.one = all(n == 1 for n in new) and extra_rows == 0
        self.cache = np.full((self.pages, H, 2, 64 * (D // 2 + 4)), 0xFF, np.uint8)   # codes 15, NaN pairs

    def fill(self, kmag=1.0, vmag=1.0):
        """Keys and values of every position; returns the values that the cache holds."""
        self.kv = []
        for b, c in enumerate(self.ctx):
            vals = []
            for kv in range(2):
                x = (self.rng.standard_normal((self.H, c, self.D)) * (vmag if kv else kmag)).astype(np.float32)
                if not kv:
                    x += (self.rng.standard_normal((self.H, 1, self.D)) * kmag).astype(np.float32)
                codes, s, m = A.kv4_encode(x)
                for h in range(self.H):
                    for t in range(c):
                        A.kv4_pack(self.cache, self.table[b, t // 64], t % 64, h, kv, codes[h, t], s[h, t], m[h, t])
                vals.append((A.kv4_values(codes, s, m), s, m))
            self.kv.append(vals)
        return self

    def put(self, b, kv, h, t, x):
        """Row x float32 [D] coded as key (kv 0) or value (1) of token t of sequence b, head h."""
        codes, s, m = (a[0] for a in A.kv4_encode(x[None]))
        A.kv4_pack(self.cache, self.table[b, t // 64], t % 64, h, kv, codes, s, m)
        vals, ss, ms = self.kv[b][kv]
        vals[h, t], ss[h, t], ms[h, t] = A.kv4_values(codes, s, m), s, m

    def times(self, b, kv, h, t, f):
        """That row's step and low end times f."""
        codes, s, m = A.kv4_unpack(self.cache, self.table[b, t // 64], t % 64, h, kv)
        s, m = A.to_bf16(np.array([s, m], np.float32) * np.float32(f))
        A.kv4_pack(self.cache, self.table[b, t // 64], t % 64, h, kv, codes, s, m)
        vals, ss, ms = self.kv[b][kv]
        vals[h, t], ss[h, t], ms[h, t] = A.kv4_values(codes, s, m), s, m

    def dev(self):
        self.d_cache = torch.from_numpy(self.cache).cuda()
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_lens = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.d_cu = None if self.one else torch.from_numpy(self.cu).cuda()
        return self


RAGGED = [
    ([1], [1]), ([64], [1]), ([65], [1]), ([130], [130]), ([200, 1, 0, 63, 128], [1] * 5),
    ([70, 5, 0, 64, 300], [9, 5, 2, 1, 17]), ([3, 2], [7, 2]),   # more rows than tokens: no place for the first
]


# ----------------------------------------------------------------------------- cache
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2)])
@pytest.mark.parametrize("ctx,new", RAGGED)
def test_cache_write_and_read(ctx, new, D, H, dtype):
    bt = Batch(ctx, new, H, D, seed=len(ctx) + D, extra_rows=0 if all(n == 1 for n in new) else 3).dev()
    rng = bt.rng
    mags = np.array([1.0, 1e-3, 300.0, 1e-30, 1e30], np.float32)[rng.integers(0, 5, bt.T)][:, None, None]
    x = [A.to_bf16(v) if dtype == BF else v for v in
         [(rng.standard_normal((bt.T, H, D)) * mags).astype(np.float32) for _ in range(2)]]
    x[0][0, 0, 3] = np.nan
    x[1][0, 0, :] = 2.5
    pad = 8
    big = [torch.zeros((bt.T, H * D + pad), dtype=dtype, device="cuda") for _ in range(2)]
    view = [t[:, :H * D].unflatten(1, (H, D)) for t in big]
    for v, a in zip(view, x):
        v.copy_(torch.from_numpy(a))
    S.kv4_write(bt.d_cache, view[0], view[1], bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    expect, back = bt.cache.copy(), [np.full((bt.T, H, D), 77.0, np.float32) for _ in range(2)]
    for kv in range(2):
        codes, s, m = A.kv4_encode(x[kv])
        vals = A.kv4_values(codes, s, m).astype(np.float32)
        for b, (c, n) in enumerate(zip(ctx, new)):
            for i in range(n):
                p, t = c - n + i, bt.cu[b] + i
                if p < 0:
                    continue
                for h in range(H):
                    A.kv4_pack(expect, bt.table[b, p // 64], p % 64, h, kv, codes[t, h], s[t, h], m[t, h])
                back[kv][t] = A.to_bf16(vals[t]) if dtype == BF else vals[t]
    got = bt.d_cache.cpu().numpy()
    nan_pair = np.array([0x7FFF, 0x7FFF], np.uint16).view(np.uint8)
    for kv in range(2):   # a NaN's bits are the library's own
        nan = A.kv4_encode(x[kv])[1]
        for b, (c, n) in enumerate(zip(ctx, new)):
            for i in range(n):
                p = c - n + i
                for h in range(H):
                    if p >= 0 and np.isnan(nan[bt.cu[b] + i, h]):
                        at = 32 * D + 4 * (p % 64)
                        expect[bt.table[b, p // 64], h, kv, at:at + 4] = nan_pair
    assert np.array_equal(got, expect)
    out = [torch.full((bt.T, H * D + pad), 77.0, dtype=dtype, device="cuda") for _ in range(2)]
    k, v = S.kv4_read(bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu,
                      k=out[0][:, :H * D].unflatten(1, (H, D)), v=out[1][:, :H * D].unflatten(1, (H, D)))
    assert np.array_equal(np_of(k), back[0], equal_nan=True)
    assert np.array_equal(np_of(v), back[1], equal_nan=True)
    assert torch.all(out[0][:, H * D:] == 77.0)
    assert S.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("D,H", [(64, 31), (128, 15)])
def test_cache_many_rows_as_few(D, H, dtype):
    """A write and a read of many rows and the same rows sequence by sequence, in parts of a hundred: equal bits."""
    ctx, new = [733, 1, 0, 640], [700, 1, 5, 640]
    bt = Batch(ctx, new, H, D, seed=D, extra_rows=2).dev()
    mag = 10.0 ** torch.randint(-30, 30, (bt.T, H, 1), device="cuda").float()
    x = [(torch.randn(bt.T, H, D, device="cuda") * mag).to(dtype) for _ in range(2)]
    x[0][3, 2, 7], x[1][5, 1, 0], x[0][9, 4] = float("nan"), float("inf"), -2.5
    S.kv4_write(bt.d_cache, x[0], x[1], bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    k, v = S.kv4_read(bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu, rows=bt.T, dtype=dtype)
    parts = torch.from_numpy(bt.cache).cuda()
    for b, (c, n) in enumerate(zip(ctx, new)):
        for i in range(max(n - c, 0), n, 100):
            m = min(100, n - i)
            rows = slice(int(bt.cu[b]) + i, int(bt.cu[b]) + i + m)
            args = (bt.d_table[b:b + 1], torch.tensor([c - n + i + m], dtype=torch.int32, device="cuda"))
            cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            S.kv4_write(parts, x[0][rows].contiguous(), x[1][rows].contiguous(), *args, cu_q=cu)
            pk, pv = S.kv4_read(parts, *args, cu_q=cu, rows=m, dtype=dtype)
            assert torch.equal(pk.nan_to_num(7.0), k[rows].nan_to_num(7.0)) and torch.equal(pv.nan_to_num(7.0), v[rows].nan_to_num(7.0))
    assert torch.equal(parts, bt.d_cache) and S.device_error() == 0
    assert torch.isnan(k[3, 2]).all() and torch.isnan(v[5, 1]).all() and torch.all(k[9, 4] == -2.5)


def test_read_makes_its_own_tensors():
    bt = Batch([5, 64], [1, 1], 2, 64, seed=4).fill().dev()
    k, v = S.kv4_read(bt.d_cache, bt.d_table, bt.d_lens)
    for b, c in enumerate(bt.ctx):
        assert np.array_equal(np_of(k)[b], bt.kv[b][0][0][:, c - 1].astype(np.float32))
        assert np.array_equal(np_of(v)[b], bt.kv[b][1][0][:, c - 1].astype(np.float32))


# ----------------------------------------------------------------------------- attention
def attn_bound(q, kv, ref, scale, tile=False):
    """Per row [n, D]: the bound of the module's head."""
    (k, ks, km), (v, vs, vm) = kv
    D = q.shape[-1]
    sq = np.abs(q).sum(-1, keepdims=True)
    smax, mmax = np.max(ks, initial=0.0), np.max(np.abs(km), initial=0.0)
    dx = abs(scale) * sq * 2.0 ** -23 * (143.0 * smax * (D // 8 + 4) + 3 * (mmax + 136.0 * smax))
    if tile:
        dx = dx + abs(scale) * sq * np.max(np.abs(k), initial=0.0) * 2.0 ** -11
    vmax = np.max(np.abs(v), initial=0.0)
    return (2 * dx + 2.0 ** -12) * vmax + 2.0 ** -8 * 8 * np.max(vs, initial=0.0) + 2.0 ** -8 * np.abs(ref)


def row_bound(q, kv, last, ref, scale, tile=False):
    """Per row [n, D]: the bound by what the row sees."""
    (k, ks, km), (v, vs, vm) = [tuple(np.asarray(x, np.float64) for x in side) for side in kv]
    q = q.astype(np.float64)
    D, tol = q.shape[-1], np.zeros(ref.shape)
    for i in range(len(q)):
        e = min(int(last[i]) + 1, len(k))
        if e <= 0:
            continue
        x = k[:e] @ q[i] * scale
        p = np.exp(x - x.max())
        p /= p.sum()
        va, sq = np.abs(v[:e]).max(-1), np.abs(q[i]).sum()
        dx = abs(scale) * sq * 2.0 ** -23 * (143 * ks[:e] * (D // 8 + 4) + 3 * (np.abs(km[:e]) + 136 * ks[:e]))
        dv = vs[:e] * (2.0 ** -8 + e / 16 * 23 * 2.0 ** -23)
        if tile:
            dx = dx + abs(scale) * sq * np.abs(k[:e]).max(-1) * 2.0 ** -10
            dv = va * (2.0 ** -10 + 2.0 ** -11)
        w = p * (np.exp(2 * np.minimum(dx, 300.0)) - 1 + 2.0 ** -20 + e * 2.0 ** -23)   # e^(2 dx) - 1 >= 2 dx
        a = np.abs(ref[i])
        tol[i] = (w * va).sum() + w.sum() * a + (p * dv).sum() + e * 2.0 ** -26 * (p * va).max() + 2.0 ** -8 * a
    return tol


def check_rows(bt, q, out, hq, scale, tile=False, heads=None, skip=0):
    """Every row but a sequence's last `skip` within row_bound; returns the largest bound over the largest
    magnitude of its row."""
    o, g, worst = np_of(out).astype(np.float64), hq // bt.H, 0.0
    for b, (c, n) in enumerate(zip(bt.ctx, bt.new)):
        r = slice(bt.cu[b], bt.cu[b] + n - skip)
        last = c - n + np.arange(n - skip)
        for j in (heads or range(hq)):
            kv = [tuple(a[j // g] for a in side) for side in bt.kv[b]]
            ref = A.attend(q[r, j].astype(np.float64), kv[0][0], kv[1][0], last, scale)
            tol = row_bound(q[r, j], kv, last, ref, scale, tile)
            err = np.abs(o[r, j] - ref)
            assert np.all(err <= tol), (b, j, np.argwhere(~(err <= tol))[0], err[~(err <= tol)][0], tol[~(err <= tol)][0])
            seen = np.abs(ref).max(-1) > 0
            worst = max(worst, (tol.max(-1)[seen] / np.abs(ref).max(-1)[seen]).max(initial=0.0))
    return worst


def check_attn(bt, q, out, hq, scale, sentinel=None, tile=False):
    g = hq // bt.H
    o = np_of(out).astype(np.float64)
    for b, (c, n) in enumerate(zip(bt.ctx, bt.new)):
        r = slice(bt.cu[b], bt.cu[b] + n)
        last = c - n + np.arange(n)
        for j in range(hq):
            h = j // g
            kv = [(x[h], s[h], m[h]) for x, s, m in bt.kv[b]]
            ref = A.attend(q[r, j].astype(np.float64), kv[0][0], kv[1][0], last, scale)
            tol = attn_bound(q[r, j], kv, ref, scale, tile)
            err = np.abs(o[r, j] - ref)
            assert np.all(err <= tol), (b, j, np.nanmax(err - tol), np.isnan(err).sum())
            assert not o[r, j][last < 0].any()
    if sentinel is not None:
        assert np.all(o[bt.cu[-1]:] == sentinel)


def run_attn(ctx, new, hq, H, D, seed, qmag=1.0, scale=None, extra=0, max_q=0, pad=0, tile=False, wide=0):
    bt = Batch(ctx, new, H, D, seed, extra_rows=extra, wide=wide).fill().dev()
    q = bf16_randn(bt.rng, (bt.T, hq, D), qmag)
    big = torch.full((bt.T, hq * D + pad), float("nan"), dtype=BF, device="cuda")
    big[:, :hq * D] = torch.from_numpy(q).reshape(bt.T, hq * D)
    obig = torch.full((bt.T, hq * D + pad), 77.0, dtype=BF, device="cuda")
    out = S.attn_kv4(big[:, :hq * D].unflatten(1, (hq, D)), bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu,
                     max_q=max_q, scale=scale, out=obig[:, :hq * D].unflatten(1, (hq, D)))
    assert S.device_error() == 0
    check_attn(bt, q, out, hq, D ** -0.5 if scale is None else scale, 77.0 if extra else None, tile)
    assert pad == 0 or torch.all(obig[:, hq * D:] == 77.0)
    return bt, q, out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,H", [(4, 1), (8, 8), (6, 2), (16, 1), (20, 1)])
@pytest.mark.parametrize("ctx,new", RAGGED)
def test_attn_matches_oracle(ctx, new, hq, H, D):
    run_attn(ctx, new, hq, H, D, seed=sum(ctx) + hq, extra=0 if all(n == 1 for n in new) else 3,
             max_q=max(new) if sum(ctx) % 2 else 0, pad=8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,hq,H", [
    ([1500], [1], 4, 1),                       # one long sequence: split over the machine
    ([900, 17, 1300, 0, 64], [1] * 5, 8, 2),
    ([300], [300], 8, 2),                      # a prompt: several tiles of rows
    ([700, 40, 513], [200, 40, 129], 4, 2),    # prompts behind a context, one without
    ([700, 800, 0, 90], [150, 1, 1, 2], 6, 2),  # a prompt and single tokens in one batch
    ([257], [256], 1, 1), ([640], [33], 3, 1),
])
def test_attn_longer(ctx, new, hq, H, D):
    for max_q in (0, max(new)):
        run_attn(ctx, new, hq, H, D, seed=len(ctx) * 7 + hq + D, max_q=max_q,
                 extra=0 if all(n == 1 for n in new) else 2)


# Short tables go to a cluster per row tile where the batch has few; a table of this width (what a sequence
# may grow to) and a batch of many row tiles go to runs over the whole machine and a join.
WIDE = 4096


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,hq,H", [
    ([1], [1], 4, 1), ([1500], [1], 4, 1), ([900, 17, 1300, 0, 64], [1] * 5, 8, 2), ([200, 1, 0, 63, 128], [1] * 5, 8, 8),
    ([70, 5, 0, 64, 300], [9, 5, 2, 1, 17], 20, 1), ([130], [130], 6, 2), ([3, 2], [7, 2], 16, 1),
])
def test_attn_in_runs(ctx, new, hq, H, D):
    one = all(n == 1 for n in new)
    args = dict(hq=hq, H=H, D=D, seed=sum(ctx) + hq, extra=0 if one else 3, max_q=0 if D == 64 else max(new), pad=8)
    _, _, out = run_attn(ctx, new, wide=WIDE, **args)
    _, _, short = run_attn(ctx, new, **args)     # the same numbers, the sums in another order
    rows = sum(new)
    assert torch.allclose(out[:rows].float(), short[:rows].float(), rtol=2.0 ** -7, atol=2.0 ** -10 * short[:rows].abs().max().item())


@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("some", [[1, 1, 2], [5, 1, 3], [40, 2, 1]])
def test_attn_most_sequences_have_no_new_token(some, D, wide):
    new, ctx = [0] * 150, [i % 90 for i in range(150)]
    new[3], new[77], new[149] = some
    bt, q, out = run_attn(ctx, new, 8, 2, D, seed=D, extra=2, wide=wide)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,new,hq,H", [(5, 1, 32, 8), (11, 1, 32, 8), (24, 1, 8, 8), (50, 1, 8, 8), (90, 1, 16, 8), (13, 5, 32, 8), (26, 3, 32, 8),
                                        (45, 3, 32, 8)])
def test_attn_batches_of_every_cluster_size(n, new, hq, H, D):
    ctx = [[70, 1, 129, 0, 64, 200, 3][i % 7] for i in range(n)]
    run_attn(ctx, [new] * n, hq, H, D, seed=n + D, max_q=new)


def test_attn_in_runs_is_deterministic_and_graph_safe():
    bt, q, out = run_attn([800, 650, 150], [1] * 3, 8, 2, 64, seed=11, wide=WIDE)
    dq = torch.from_numpy(q).cuda().bfloat16()
    outs, graphs = [torch.empty_like(out) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)
    bt.d_lens.copy_(torch.tensor([800, 64, 1], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens))
    assert S.device_error() == 0


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_in_runs_nan_and_bad_pages(kv, D):
    bt = Batch([70, 900], [5, 2], 2, D, seed=17, wide=WIDE).fill()
    at = 32 * D + 4 * 3
    bt.cache[bt.table[0, 1], 1, kv, at:at + 4] = 0xFF    # token 67 of sequence 0, head 1: seen by rows 2, 3, 4
    bt.dev()
    q = torch.randn(7, 6, D, device="cuda").bfloat16()
    out = S.attn_kv4(q, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu, max_q=5)
    bad = torch.isnan(out).any(-1)
    assert bad[2:5, 3:].all() and not bad[:2].any() and not bad[5:].any() and not bad[:, :3].any()
    assert S.device_error() == 0
    bt.d_table[0, 1] = bt.pages      # that page away: tokens 0 .. 63 are left
    out = S.attn_kv4(q, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu, max_q=5)
    assert S.device_error() == 8 and not torch.isnan(out).any()
    q = q.float().cpu().numpy().astype(np.float64)
    for j in range(6):
        part = [(x[j // 3][:64], s[j // 3][:64], m[j // 3][:64]) for x, s, m in bt.kv[0]]
        ref = A.attend(q[:5, j], part[0][0], part[1][0], [63] * 5, D ** -0.5)
        assert np.all(np.abs(np_of(out)[:5, j] - ref) <= attn_bound(q[:5, j], part, ref, D ** -0.5))


def is_tiles(bt, hq):
    """The rule by which a batch goes to the tile kernel (sequences of more than 32 rows)."""
    g, sms = hq // bt.H, torch.cuda.get_device_properties(0).multi_processor_count
    rows = bt.T * g
    few, tile = bt.H * (rows // 16 + len(bt.ctx)), bt.H * (rows // 256 + len(bt.ctx))
    return few * 27 >= 100 * sms * -(-tile // sms)


TILES = [
    ([300], [300], 32, 8), ([700], [300], 32, 8), ([129], [129], 128, 8),
    ([700, 800, 0, 90], [330, 1, 1, 2], 32, 8),   # a prompt and single tokens: both kernels
    ([900, 40, 613], [300, 40, 129], 32, 8), ([3, 290], [7, 290], 32, 8),
    ([1150], [1150], 8, 8), ([400], [400], 24, 8), ([576], [576], 16, 8),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,hq,H", TILES)
def test_attn_tiles(ctx, new, hq, H, D):
    bt, _, _ = run_attn(ctx, new, hq, H, D, seed=sum(ctx) + D, max_q=max(new) if D == 64 else 0, extra=3, pad=8, tile=True)
    assert is_tiles(bt, hq)


@pytest.mark.parametrize("kw", [dict(qmag=30.0), dict(qmag=1e-4), dict(scale=0.0), dict(scale=-0.3), dict(qmag=1e20, scale=1e-21)])
def test_attn_tiles_peaked_scores_and_large_values(kw):
    bt, _, _ = run_attn([433], [330], 32, 8, 64, seed=31, tile=True, **kw)
    assert is_tiles(bt, 32)


@pytest.mark.parametrize("growing", [False, True])
def test_attn_tiles_values_of_very_different_size(growing):
    """Values whose size changes a hundredfold from page to page, up or down: O follows their power of two."""
    bt = Batch([640], [330], 8, 64, seed=32)
    scale = np.float32(10.0) ** (np.arange(10) if growing else -np.arange(10))
    bt.fill()
    vals, s, m = bt.kv[0][1]
    for h in range(8):
        for t in range(640):
            f = scale[t // 64]
            c, ss, mm = A.kv4_unpack(bt.cache, bt.table[0, t // 64], t % 64, h, 1)
            s[h, t], m[h, t] = A.to_bf16(np.array([ss, mm]) * f)
            A.kv4_pack(bt.cache, bt.table[0, t // 64], t % 64, h, 1, c, s[h, t], m[h, t])
            vals[h, t] = A.kv4_values(c[None], s[h, t:t + 1], m[h, t:t + 1])[0]
    bt.dev()
    q = bf16_randn(bt.rng, (bt.T, 32, 64))
    out = S.attn_kv4(torch.from_numpy(q).cuda().bfloat16(), bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    assert is_tiles(bt, 32)
    check_attn(bt, q, out, 32, 0.125, tile=True)


def test_attn_tiles_deterministic_and_graph():
    bt, q, out = run_attn([800, 650], [300, 40], 32, 8, 128, seed=33, tile=True)
    assert is_tiles(bt, 32)
    dq = torch.from_numpy(q).cuda().bfloat16()
    o = torch.empty_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu, out=o)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out)


@pytest.mark.parametrize("bad", [-1, 1 << 20, "width"])
def test_attn_tiles_bad_pages(bad):
    new, ctx = 300, [500, 420]
    bt = Batch(ctx, [new] * 2, 8, 64, seed=34).fill()
    there = [np.ones(c, bool) for c in ctx]
    if bad == "width":
        bt.dev()
        bt.d_table = bt.d_table[:, :5].contiguous()
        for t in there:
            t[320:] = False
    else:
        bt.table[0, 1] = bt.table[1, 0] = bad
        there[0][64:128] = there[1][:64] = False
        bt.dev()
    q = bf16_randn(bt.rng, (2 * new, 32, 64))
    out = S.attn_kv4(torch.from_numpy(q).cuda().bfloat16(), bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    assert is_tiles(bt, 32) and S.device_error() == 8 and S.device_error() == 0
    o = np_of(out)
    for b, c in enumerate(ctx):
        for j in range(0, 32, 5):
            kv = [(x[j // 4][there[b]], s[j // 4][there[b]], m[j // 4][there[b]]) for x, s, m in bt.kv[b]]
            last = np.array([there[b][:c - new + i + 1].sum() - 1 for i in range(new)])
            r = slice(b * new, (b + 1) * new)
            ref = A.attend(q[r, j].astype(np.float64), kv[0][0], kv[1][0], last, 0.125)
            assert np.all(np.abs(o[r, j] - ref) <= attn_bound(q[r, j], kv, ref, 0.125, True))


@pytest.mark.parametrize("kv", [0, 1])
def test_attn_tiles_nan_reaches_only_the_rows_that_see_it(kv):
    bt = Batch([500], [300], 8, 64, seed=35).fill()
    at = 64 * 32 + 4 * (400 % 64)
    bt.cache[bt.table[0, 400 // 64], 3, kv, at:at + 4] = 0xFF    # token 400, head 3
    bt.dev()
    q = torch.randn(300, 32, 64, device="cuda").bfloat16()
    out = S.attn_kv4(q, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    assert is_tiles(bt, 32)
    bad = torch.isnan(out).any(-1)      # row i is position 200 + i
    assert bad[200:, 12:16].all() and not bad[:200].any() and not bad[:, :12].any() and not bad[:, 16:].any()


@pytest.mark.parametrize("cu", [[0, -5, 600], [600, 10, 0], [0, 1 << 30, 600], [-9, 300, 1 << 30]])
def test_attn_tiles_malformed_row_offsets_stay_in_bounds(cu):
    bt = Batch([700, 690], [300, 300], 8, 64, seed=36).fill().dev()
    assert is_tiles(bt, 32)
    q = torch.randn(600, 32, 64, device="cuda").bfloat16()
    guard = torch.full((602, 32, 64), 77.0, dtype=BF, device="cuda")
    S.attn_kv4(q, bt.d_cache, bt.d_table, bt.d_lens, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), out=guard[1:601])
    S.device_error()
    assert torch.all(guard[0] == 77.0) and torch.all(guard[601] == 77.0)


@pytest.mark.parametrize("new", [1, 300])
def test_waits_that_run_out_are_reported(new):
    """A limit of a few cycles: the kernels give up, record it and return; the next call is whole again."""
    bt, q, out = run_attn([700, 690], [new, new], 32, 8, 64, seed=37, tile=new > 1)
    dq = torch.from_numpy(q).cuda().bfloat16()
    S.set_wait_limit(16)
    try:
        for _ in range(2):
            S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu)
        # a copy of a page or two may well be there at the first look; the tiles' first product is not
        assert S.device_error() in ((6,) if new > 1 else (0, 6))
    finally:
        S.set_wait_limit(0)
    assert S.device_error() == 0
    assert torch.equal(S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu), out)


def test_waits_that_run_out_in_runs_are_reported():
    bt, q, out = run_attn([700, 690], [1, 1], 32, 8, 64, seed=38, wide=WIDE)
    dq = torch.from_numpy(q).cuda().bfloat16()
    S.set_wait_limit(16)
    try:
        for _ in range(2):
            S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens)
        assert S.device_error() in (0, 6)
    finally:
        S.set_wait_limit(0)
    assert S.device_error() == 0
    assert torch.equal(S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens), out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,wide", [
    ([700, 690], 1, 0), ([700, 690], 1, WIDE),           # a cluster per row tile; runs and a join
    ([700, 690, 64, 0], 3, 0), ([700, 690, 64, 0], 3, WIDE), ([40], 1, 0), ([9000], 1, WIDE),
])
def test_waits_without_a_look_are_reported_and_leave_no_copy_behind(ctx, new, wide, D):
    """With a limit of 1 no wait is given a look while a ring of copies is on its way: the status is the
    timeout's, the next calls' shared memory is their own, and they are exact."""
    bt, q, out = run_attn(ctx, [new] * len(ctx), 32, 8, D, seed=39, wide=wide, max_q=new)
    dq = torch.from_numpy(q).cuda().bfloat16()
    args = (dq, bt.d_cache, bt.d_table, bt.d_lens)
    again = []
    for _ in range(3):
        S.set_wait_limit(1)
        try:
            S.attn_kv4(*args, cu_q=bt.d_cu, max_q=new)
        finally:
            S.set_wait_limit(0)
        # right behind it, with no look at the status between
        again += [S.attn_kv4(*args, cu_q=bt.d_cu, max_q=new) for _ in range(3)]
        assert S.device_error() == 6 and S.device_error() == 0
    assert all(torch.equal(o, out) for o in again)


@pytest.mark.parametrize("new", [[1], [140]])
def test_attn_peaked_scores_and_large_values(new):
    run_attn([333], new, 4, 2, 64, seed=5, qmag=30.0)
    run_attn([333], new, 4, 2, 128, seed=6, qmag=1e-4)
    run_attn([333], new, 4, 2, 64, seed=7, scale=0.0)
    run_attn([333], new, 4, 2, 64, seed=8, scale=-0.3)


@pytest.mark.parametrize("new", [1, 200])
def test_attn_max_q_too_small_changes_nothing_but_rounding(new):
    run_attn([260, 230], [new, new], 4, 2, 64, seed=9, max_q=1)


@pytest.mark.parametrize("new", [1, 150])
def test_attn_is_deterministic_and_graph_safe(new):
    bt, q, out = run_attn([800, 650, 150], [new] * 3, 8, 2, 64, seed=11)
    dq = torch.from_numpy(q).cuda().bfloat16()
    ref = S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    again = S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    assert torch.equal(ref, again) and torch.equal(ref, out)
    # two graphs replayed at the same time share no scratch
    outs, graphs = [], []
    for _ in range(2):
        o = torch.empty_like(ref)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu, out=o)
        outs.append(o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    # lengths that change between replays are read anew
    bt.d_lens.copy_(torch.tensor([800, 64, 1], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu))
    assert S.device_error() == 0


def test_attn_two_streams_at_once():
    bt, q, out = run_attn([800, 650, 150], [1] * 3, 8, 2, 128, seed=12)
    dq = torch.from_numpy(q).cuda().bfloat16()
    torch.cuda.synchronize()
    res = []
    for _ in range(6):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            res.append([S.attn_kv4(dq, bt.d_cache, bt.d_table, bt.d_lens) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(r, out) for rs in res for r in rs)


# ----------------------------------------------------------------------------- bad indexes
@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("bad", [-1, 1 << 20, "width"])
def test_bad_pages_are_recorded_and_passed_over(bad, new):
    ctx = [300, 200]
    bt = Batch(ctx, [new] * 2, 2, 64, seed=13).fill()
    if bad == "width":   # a length beyond the table: the tokens past it are not there
        bt.dev()
        cut = 64 * 3
        bt.d_table = bt.d_table[:, :3].contiguous()
    else:
        cut = None
        hole = 1         # tokens 64 .. 127 of sequence 0
        bt.table[0, hole] = bad
        bt.dev()
    q = bf16_randn(bt.rng, (2 * new, 4, 64))
    out = S.attn_kv4(torch.from_numpy(q).cuda().bfloat16(), bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu)
    assert S.device_error() == 8 and S.device_error() == 0
    o = np_of(out)
    for b, c in enumerate(ctx):
        there = np.ones(c, bool)
        if cut is not None:
            there[cut:] = False
        elif b == 0:
            there[64:128] = False
        for j in range(4):
            kv = [(x[j // 2][there], s[j // 2][there], m[j // 2][there]) for x, s, m in bt.kv[b]]
            last = np.array([there[:c - new + i + 1].sum() - 1 for i in range(new)])
            r = slice(b * new, (b + 1) * new)
            ref = A.attend(q[r, j].astype(np.float64), kv[0][0], kv[1][0], last, 0.125)
            assert np.all(np.abs(o[r, j] - ref) <= attn_bound(q[r, j], kv, ref, 0.125))
    # the write and the read pass such tokens over
    x = torch.randn(2 * new, 2, 64, device="cuda")
    before = bt.d_cache.clone()
    t2 = torch.full_like(bt.d_table, bt.pages if bad == "width" else bad)
    S.kv4_write(bt.d_cache, x, x, t2, bt.d_lens, cu_q=bt.d_cu)
    assert S.device_error() == 8
    assert torch.equal(before, bt.d_cache)
    k, v = S.kv4_read(bt.d_cache, t2, bt.d_lens, cu_q=bt.d_cu, rows=2 * new)
    assert S.device_error() == 8 and not k.any() and not v.any()


@pytest.mark.parametrize("cu", [[0, -5, 40], [40, 10, 0], [0, 1 << 30, 40], [-9, 20, 1 << 30], [7, 7, 7]])
def test_malformed_row_offsets_stay_in_bounds(cu):
    bt = Batch([100, 90], [20, 20], 2, 64, seed=14).fill().dev()
    d_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    q = torch.randn(40, 4, 64, device="cuda").bfloat16()
    guard = torch.full((42, 4, 64), 77.0, dtype=BF, device="cuda")
    for max_q in (0, 1):
        S.attn_kv4(q, bt.d_cache, bt.d_table, bt.d_lens, cu_q=d_cu, max_q=max_q, out=guard[1:41])
    x = torch.randn(40, 2, 64, device="cuda")
    S.kv4_write(bt.d_cache, x, x, bt.d_table, bt.d_lens, cu_q=d_cu)
    S.kv4_read(bt.d_cache, bt.d_table, bt.d_lens, cu_q=d_cu, rows=40)
    S.device_error()
    assert torch.all(guard[0] == 77.0) and torch.all(guard[41] == 77.0)


def test_negative_lengths_are_empty():
    bt = Batch([100, 90], [1, 1], 2, 64, seed=15).fill().dev()
    lens = torch.tensor([-3, 90], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    out = S.attn_kv4(q, bt.d_cache, bt.d_table, lens)
    assert not out[0].any() and out[1].any() and S.device_error() == 0


def test_nan_in_a_visible_token_reaches_only_its_rows():
    bt = Batch([70, 80], [1, 1], 2, 64, seed=16).fill()
    at = 64 * 32 + 4 * 5
    bt.cache[bt.table[0, 0], 1, 0, at:at + 4] = 0xFF    # key 5 of sequence 0, head 1
    bt.dev()
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    out = S.attn_kv4(q, bt.d_cache, bt.d_table, bt.d_lens)
    bad = torch.isnan(out).any(-1)
    assert bad[0, 2:].all() and not bad[0, :2].any() and not bad[1].any()


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_among_drafts_reaches_only_the_rows_that_see_it(kv, D):
    bt = Batch([70, 9], [5, 2], 2, D, seed=17).fill()
    at = 32 * D + 4 * 3
    bt.cache[bt.table[0, 1], 1, kv, at:at + 4] = 0xFF    # token 67 of sequence 0, head 1: seen by rows 2, 3, 4
    bt.dev()
    q = torch.randn(7, 6, D, device="cuda").bfloat16()
    out = S.attn_kv4(q, bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu, max_q=5)
    bad = torch.isnan(out).any(-1)
    assert bad[2:5, 3:].all() and not bad[:2].any() and not bad[5:].any() and not bad[:, :3].any()


@pytest.mark.parametrize("D", [64, 128])
def test_long_context_keeps_bf16_accuracy(D):
    """A bf16 rounding is off by at most 2^-8 / sqrt(12) * 2 of a value (rms of half a step either way, where
    the value's mantissa is smallest); everything before it together by less than 2^-12."""
    bt, q, out = run_attn([20000], [1], 8, 2, D, seed=23)
    for j in range(0, 8, 3):
        kv = [(x[j // 4], s[j // 4], m[j // 4]) for x, s, m in bt.kv[0]]
        ref = A.attend(q[:, j].astype(np.float64), kv[0][0], kv[1][0], [19999], D ** -0.5)
        err = np.linalg.norm(np_of(out)[0, j] - ref[0]) / np.linalg.norm(ref[0])
        assert err <= 2.0 ** -7 / 12 ** 0.5 + 2.0 ** -12


# ----------------------------------------------------------------------------- range
FORMS = [(64, 0), (128, 0), (64, WIDE), (128, WIDE)]     # clusters or a run per row tile; runs and a join


def call(bt, q, **kw):
    return S.attn_kv4(torch.from_numpy(q).cuda().bfloat16(), bt.d_cache, bt.d_table, bt.d_lens, cu_q=bt.d_cu, **kw)


@pytest.mark.parametrize("D,wide", FORMS)
@pytest.mark.parametrize("ctx,new,same", [([1], [1], False), ([1, 70, 900], [1, 1, 1], False), ([9000], [1], True), ([2100, 130], [5, 3], True)])
@pytest.mark.parametrize("value", [1.0, 256.0, 2.0 ** 22, 1e30, -3e38, 1e-30, 0.0])
def test_constant_value_rows(value, ctx, new, same, D, wide):
    """Value rows of one number (step 0): the output is that number, for one token, for thousands of equal
    scores (keys of zero) and of unequal ones."""
    bt = Batch(ctx, new, 2, D, seed=51, wide=wide).fill()
    for b, c in enumerate(ctx):
        for h in range(2):
            for t in range(c):
                bt.put(b, 1, h, t, np.full(D, value, np.float32))
                if same:
                    bt.put(b, 0, h, t, np.zeros(D, np.float32))
    q = bf16_randn(bt.rng, (bt.T, 8, D))
    out = call(bt.dev(), q, max_q=max(new))
    assert S.device_error() == 0
    check_rows(bt, q, out, 8, D ** -0.5, heads=[0, 5])
    # the low end and the result are each rounded to bf16, half a step of 2^-8
    assert torch.all((out.double() / (value or 1.0) - (1.0 if value else 0.0)).abs() <= 2.0 ** -7)


@pytest.mark.parametrize("D,wide", FORMS)
@pytest.mark.parametrize("mag", [1e-33, 1e-20, 1e20, 1e36])
def test_values_of_any_size(mag, D, wide):
    bt = Batch([70, 500, 1000], [1, 5, 2], 2, D, seed=52, wide=wide).fill(vmag=mag)
    q = bf16_randn(bt.rng, (bt.T, 8, D))
    assert check_rows(bt, q, call(bt.dev(), q, max_q=5), 8, D ** -0.5) < 0.25 and S.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("power", [-118, -60, 60, 105])
def test_queries_and_keys_of_any_size(power, tile, D):
    """Queries times a power of two and keys divided by it: the same scores, to the bit where no power of the
    kernels' own stops short of them (keys of 2^118 are taken token by token, each with its own rounding)."""
    bt = Batch([433], [330], 8, D, 68) if tile else Batch([433, 70], [3, 1], 8, D, 68)
    bt.fill()
    assert is_tiles(bt, 32) or not tile
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    q = np.where(np.abs(q) < 2.0 ** -7, np.float32(0), q)      # (no query below the normal numbers)
    ref = call(bt.dev(), q, max_q=max(bt.new))
    check_rows(bt, q, ref, 32, D ** -0.5, tile=tile, heads=[0])
    for b, c in enumerate(bt.ctx):
        for h in range(8):
            for t in range(c):
                bt.times(b, 0, h, t, 2.0 ** -power)
    q *= np.float32(2.0 ** power)
    out = call(bt.dev(), q, max_q=max(bt.new))
    check_rows(bt, q, out, 32, D ** -0.5, tile=tile, heads=[0, 31])
    assert abs(power) > 110 or torch.equal(out, ref)
    assert S.device_error() == 0


@pytest.mark.parametrize("D,wide", FORMS)
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("f", [2.0 ** 12, 2.0 ** 20, 1e30])
def test_drafts_do_not_see_later_tokens(f, side, D, wide):
    """The last draft's key or value made huge: the drafts before it stay within what they see."""
    bt = Batch([300, 90], [5, 3], 2, D, seed=53, wide=wide).fill()
    q = bf16_randn(bt.rng, (bt.T, 8, D))
    for b, c in enumerate(bt.ctx):
        for h in range(2):
            bt.times(b, side, h, c - 1, f)
    out = call(bt.dev(), q, max_q=5)
    assert S.device_error() == 0
    # (scores of 1e30 are beyond what fp32 can subtract: the rows that see such a key are left out)
    check_rows(bt, q, out, 8, D ** -0.5, skip=1 if side == 0 and f > 2.0 ** 20 else 0)


@pytest.mark.parametrize("D,wide", FORMS)
@pytest.mark.parametrize("at", [0, 70, 699])
@pytest.mark.parametrize("f", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40, 1e30])
def test_a_huge_value_without_weight_costs_nothing(f, at, D, wide):
    """One token with huge values and a score far below the others', first, in the middle and last."""
    bt = Batch([700], [3], 2, D, seed=54, wide=wide).fill()
    q = bf16_randn(bt.rng, (3, 8, D))
    q[..., 0] = 8.0
    for h in range(2):
        bt.times(0, 1, h, at, f)
        bt.put(0, 0, h, at, np.concatenate([[-60.0 * D ** 0.5], np.zeros(D - 1)]).astype(np.float32))   # x about -480
    out = call(bt.dev(), q, max_q=3)
    assert check_rows(bt, q, out, 8, D ** -0.5) < 0.25 and S.device_error() == 0


TILE_HEADS = [0, 13, 31]


def tile_batch(D, seed, ctx=(433,), new=(330,), **fill):
    bt = Batch(list(ctx), list(new), 8, D, seed).fill(**fill)
    assert is_tiles(bt, 32)
    return bt


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("at", [300, 383, 412])
@pytest.mark.parametrize("f", [2.0 ** 12, 2.0 ** 20, 1e30])
def test_tiles_rows_do_not_see_later_tokens(f, at, side, D):
    """One token's key or value made huge: the rows before it stay within what they see, and the rows after
    a value of that size too."""
    bt = tile_batch(D, 61)
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    for h in range(8):
        bt.times(0, side, h, at, f)
    out = call(bt.dev(), q)
    assert S.device_error() == 0
    # (scores of 1e30 are beyond what fp32 can subtract: the rows that see such a key are left out)
    check_rows(bt, q, out, 32, D ** -0.5, tile=True, heads=TILE_HEADS, skip=433 - at if side == 0 and f > 2.0 ** 20 else 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [0, 70, 290])
@pytest.mark.parametrize("f", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40, 1e30])
def test_tiles_a_huge_value_without_weight_costs_nothing(f, at, D):
    bt = tile_batch(D, 62)
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    q[..., 0] = 8.0
    for h in range(8):
        bt.times(0, 1, h, at, f)
        bt.put(0, 0, h, at, np.concatenate([[-60.0 * D ** 0.5], np.zeros(D - 1)]).astype(np.float32))   # x about -480
    out = call(bt.dev(), q)
    assert S.device_error() == 0
    check_rows(bt, q, out, 32, D ** -0.5, tile=True, heads=TILE_HEADS)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mag", [1e-34, 1e-20, 1e20, 1e36])
def test_tiles_values_of_any_size(mag, D):
    bt = tile_batch(D, 63, ctx=(433, 3), new=(330, 9), vmag=mag)
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    check_rows(bt, q, call(bt.dev(), q), 32, D ** -0.5, tile=True, heads=TILE_HEADS)
    assert S.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("power", [-90, -13, 60, 110])
def test_a_power_of_two_of_the_values_comes_out_exactly(power, tile, D):
    """Every rounding commutes with powers of two, as long as nothing leaves fp32's normal range."""
    bt = tile_batch(D, 67) if tile else Batch([433, 70], [3, 1], 8, D, 67).fill()
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    ref = call(bt.dev(), q, max_q=max(bt.new))
    for b, c in enumerate(bt.ctx):
        for h in range(8):
            for t in range(c):
                bt.times(b, 1, h, t, 2.0 ** power)
    assert torch.equal(call(bt.dev(), q, max_q=max(bt.new)).double() * 2.0 ** -power, ref.double())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [1.0, 2.0 ** 22, 1e30, -3e38, 1e-30, 0.0])
def test_tiles_constant_value_rows(value, D):
    bt = tile_batch(D, 64)
    for h in range(8):
        for t in range(433):
            bt.put(0, 1, h, t, np.full(D, value, np.float32))
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    out = call(bt.dev(), q)
    assert S.device_error() == 0
    # the low end and the result are each rounded to bf16, half a step of 2^-8
    assert torch.all((out.double() / (value or 1.0) - (1.0 if value else 0.0)).abs() <= 2.0 ** -7)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["pages up", "pages down", "steps up", "steps down", "tokens", "tokens and keys", "one small"])
def test_tiles_tokens_of_very_different_size(kind, D):
    """Values (and keys) whose size changes a hundredfold or more from page to page or token to token."""
    bt = tile_batch(D, 65, ctx=(640, 433), new=(330, 300))
    for b, c in enumerate(bt.ctx):
        for h in range(8):
            for t in range(c):
                if kind.startswith("pages"):
                    bt.times(b, 1, h, t, 10.0 ** (t // 64 if kind == "pages up" else -(t // 64)))
                elif kind.startswith("steps"):   # all alike within a step of 128 tokens, 1e9 from one to the next
                    bt.times(b, 1, h, t, 1e9 ** ((t // 128 if kind == "steps up" else -(t // 128)) + 0.5 * (b - 1)))
                elif kind == "one small":
                    if t % 64 == 5:
                        bt.times(b, 1, h, t, 1e-4), bt.times(b, 0, h, t, 1e-4)
                else:
                    bt.times(b, 1, h, t, 10.0 ** bt.rng.uniform(-9, 9))
                    if kind == "tokens and keys":
                        bt.times(b, 0, h, t, 10.0 ** bt.rng.uniform(-6, 0.5))
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    out = call(bt.dev(), q)
    assert S.device_error() == 0
    check_rows(bt, q, out, 32, D ** -0.5, tile=True, heads=TILE_HEADS)


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_tiles_nan_beside_tokens_of_very_different_size(kv, D):
    bt = tile_batch(D, 66)
    for h in range(8):
        for t in range(433):
            bt.times(0, 1, h, t, 10.0 ** bt.rng.uniform(-9, 9))
    bt.cache[bt.table[0, 300 // 64], 3, kv, 32 * D + 4 * (300 % 64):32 * D + 4 * (300 % 64) + 4] = 0xFF   # token 300, head 3
    q = bf16_randn(bt.rng, (bt.T, 32, D))
    out = call(bt.dev(), q)
    bad = torch.isnan(out).any(-1)      # row i is position 103 + i
    assert bad[197:, 12:16].all() and not bad[:197].any() and not bad[:, :12].any() and not bad[:, 16:].any()
    check_rows(bt, q, out, 32, D ** -0.5, tile=True, heads=[0, 31])
    check_rows(bt, q, out, 32, D ** -0.5, tile=True, heads=[13], skip=330 - 197)


# ----------------------------------------------------------------------------- together
@pytest.mark.parametrize("D,hq,H", [(64, 8, 2), (128, 4, 2)])
def test_attention_block_between_gemvs(D, hq, H):
    """Three decode steps of two sequences: q, k, v GEMVs -> rotation -> cache write -> attention ->
    o GEMV, against the same steps through the oracle from each stage's own device inputs."""
    dim, B = 512, 2
    g = torch.Generator(device="cuda").manual_seed(3)

    def w(n, k):
        return S.pack(torch.randn(n, k, generator=g, device="cuda") * 0.05)

    (wq, sq), (wk, sk), (wv, sv), (wo, so) = w(hq * D, dim), w(H * D, dim), w(H * D, dim), w(dim, hq * D)
    f = (500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    cache = S.kv4_cache(5, H, D, "cuda")
    table = torch.tensor([[3, 1], [0, 4]], dtype=torch.int32, device="cuda")
    held = [[], []]
    for step in range(3):
        lens = torch.tensor([step + 1, step + 1], dtype=torch.int32, device="cuda")
        pos = lens - 1
        x = torch.randn(B, dim, generator=g, device="cuda").bfloat16()
        q = torch.empty(B, hq * D, device="cuda")
        k, v = torch.empty(B, H * D, device="cuda"), torch.empty(B, H * D, device="cuda")
        S.gemv_bf16_grouped([(wq, sq, x, q), (wk, sk, x, k), (wv, sv, x, v)], B=B)
        qr, kr = S.qk_norm_rope(q.view(B, hq, D), k.view(B, H, D), pos, f, out_dtype=BF)
        S.kv4_write(cache, kr, v.view(B, H, D).bfloat16(), table, lens)
        o = S.attn_kv4(qr, cache, table, lens)
        y = S.gemv_bf16(wo, so, o.view(B, hq * D))
        ref = A.rope(np_of(k).reshape(B, H, D), None, pos.cpu().numpy(), f.cpu().numpy(), 0.0, False)
        assert np.all(np.abs(np_of(kr) - ref) <= np.abs(ref) * 2.0 ** -8 + np.abs(np_of(k)).max() * 2.0 ** -20)
        kk, ks, km = A.kv4_encode(np_of(kr))
        vv, vs, vm = A.kv4_encode(np_of(v.bfloat16()).reshape(B, H, D))
        for b in range(B):
            held[b].append((A.kv4_values(kk, ks, km)[b], ks[b], km[b], A.kv4_values(vv, vs, vm)[b], vs[b], vm[b]))
            for j in range(hq):
                h = j // (hq // H)
                kv = [tuple(np.stack([t[3 * i + e][h] for t in held[b]]) for e in range(3)) for i in range(2)]
                qj = np_of(qr)[b, j][None]
                r = A.attend(qj.astype(np.float64), kv[0][0], kv[1][0], [step], D ** -0.5)
                assert np.all(np.abs(np_of(o)[b, j] - r[0]) <= attn_bound(qj, kv, r, D ** -0.5)[0])
        assert torch.equal(y, S.gemv_bf16(wo, so, o.view(B, hq * D).clone())) and torch.isfinite(y).all()
    assert S.device_error() == 0


def test_c_entry_with_a_strided_table_and_workspace_of_the_stated_size():
    bt, q, out = run_attn([90, 300], [1, 1], 4, 2, 64, seed=21)
    wide = torch.full((2, bt.width + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.width] = bt.d_table
    dq = torch.from_numpy(q).cuda().bfloat16()
    o = torch.empty_like(out)
    need = S.attn_kv4_workspace_bytes(2, 4, 64)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    a = S.Kv4Args(bt.d_cache.data_ptr(), bt.pages, 2, 64, wide.data_ptr(), bt.width, wide.stride(0),
                  bt.d_lens.data_ptr(), None, 2, 2)
    st = S.lib().sherry_attn_kv4(ctypes.addressof(a), dq.data_ptr(), 256, o.data_ptr(), 256, 4, 1, 0.125,
                                 ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.all(ws[need:] == 0xA5)
    assert torch.equal(S.attn_kv4(dq, bt.d_cache, wide[:, :bt.width], bt.d_lens), out)


def test_attn_refuses_scratch_of_another_device_or_type():
    bt = Batch([70], [1], 2, 64, seed=22).fill().dev()
    q = torch.zeros(1, 4, 64, dtype=BF, device="cuda")
    need = S.attn_kv4_workspace_bytes(1, 4, 64)
    args = (q, bt.d_cache, bt.d_table, bt.d_lens)
    for ws in (torch.zeros(need, dtype=torch.uint8), torch.zeros(need, dtype=torch.int8, device="cuda"),
               torch.zeros(need, device="cuda")):
        with pytest.raises(TypeError):
            S.attn_kv4(*args, ws=ws)
    with pytest.raises(ValueError):
        S.attn_kv4(*args, ws=torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(RuntimeError):
        S.attn_kv4(*args, ws=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(S.attn_kv4(*args, ws=ws), S.attn_kv4(*args)) and S.device_error() == 0
