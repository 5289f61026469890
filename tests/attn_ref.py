"""Plain 64-bit forms of the attention half of a decode step, on the host (no
code shared with the library), and the error bounds the GPU tests hold it to."""
import math

import torch

U32 = 2.0 ** -24  # half a step of binary32, relative
U16 = 2.0 ** -11


def q4_weights(codes, scales, zeros, group):
    """[rows, cols] float64 weights of the 4-bit form."""
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    q = torch.zeros(rows, cols, dtype=torch.float64)
    q[:, 0::2] = (codes & 15).double()
    q[:, 1::2] = (codes >> 4).double()
    g = torch.arange(cols) // group
    z = torch.full(scales.shape, 8.0, dtype=torch.float64) if zeros is None else \
        (zeros & 15).double()
    return (q - z[:, g]) * scales.double()[:, g]


def q4_matvec(w, x, bias=None, resid=None, rms_eps=None):
    """(y, bound): the product in binary64 and how far fp32 sums may be from it.

    Bound per output: a sum of n fp32 products in any order is within n U32 of
    the sum of magnitudes; the hi + lo split of an activation is within 4 U32 of
    it, the scale product, the RMS factor (a sum of n squares, a square root and
    a division) and the last additions take some more steps each."""
    x = x.double()
    n = x.shape[1]
    r = torch.ones(x.shape[0], 1, dtype=torch.float64)
    if rms_eps is not None:
        r = 1.0 / ((x * x).mean(1, keepdim=True) + rms_eps).sqrt()
    y = (x @ w.t()) * r
    mag = (x.abs() @ w.abs().t()) * r
    for extra in (bias, resid):
        if extra is not None:
            y = y + extra.double()
            mag = mag + extra.double().abs()
    steps = n + 16 + (n if rms_eps is not None else 0)
    return y, steps * U32 * mag


def tables(lens, adds, table, free, page, n_tokens):
    """Python lists in, dict of lists out (table: list of rows, copied)."""
    table = [list(r) for r in table]
    width = len(table[0])
    n_free, asked, used, short = len(free), 0, 0, 0
    starts, slots, positions, new_lens = [0], [], [], []
    for r, (t, a) in enumerate(zip(lens, adds)):
        fits = t >= 0 and a >= 0 and t + a <= width * page
        held = -(-t // page) if fits else 0
        need = -(-(t + a) // page) - held if fits else 0
        first = asked
        asked += need
        ok = fits and (need == 0 or asked <= n_free)
        if ok:
            for j in range(need):
                table[r][held + j] = free[n_free - 1 - (first + j)]
                used += 1
        short += not ok
        for i in range(max(a, 0)):
            e = table[r][(t + i) // page] if ok else -1
            slots.append(e * page + (t + i) % page if e >= 0 else -1)
            positions.append(t + i if t >= 0 else -1)
        starts.append(starts[-1] + max(a, 0))
        new_lens.append(t + a if ok else t)
    pad = max(0, n_tokens - len(slots))
    return dict(table=table, starts=starts, slots=(slots + [-1] * pad)[:n_tokens],
                positions=(positions + [-1] * pad)[:n_tokens], new_lens=new_lens,
                left=[n_free - used, short])


def packet(dtype):
    return 8 if dtype == torch.float16 else 16


def rows_of_k(k):
    """[slots, heads, dim] view-copy of the key pages."""
    P, H, n, p, E = k.shape
    return k.permute(0, 3, 1, 2, 4).reshape(P * p, H, n * E)


def rows_of_v(v):
    P, H, n, D, E = v.shape
    return v.permute(0, 2, 4, 1, 3).reshape(P * n * E, H, D)


def k_of_rows(rows, pages, page):
    E = packet(rows.dtype)
    _, H, D = rows.shape
    return rows.reshape(pages, page, H, D // E, E).permute(0, 2, 3, 1, 4).contiguous()


def v_of_rows(rows, pages, page):
    E = packet(rows.dtype)
    _, H, D = rows.shape
    return rows.reshape(pages, page // E, E, H, D).permute(0, 3, 1, 4, 2).contiguous()


def round_rows(x, dtype, scale=None):
    """fp32/fp16 rows [N, H, D] as cache elements: one rounding (torch's casts on the host)."""
    x = x.float()
    if dtype == torch.float16:
        return x.half()
    return (x / scale.view(1, -1, 1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def attention(q, k_rows, v_rows, k_scale, v_scale, starts, lens, table, page, mask, scale, max_new,
              out0, q16):
    """(out, bound) over host tensors: q [N, heads, D]; k_rows, v_rows [slots, H, D]
    cache elements; rows no request names keep out0.

    Bound per output: a score's fp32 error is within d = (D + 16) U32 of the sum
    of magnitudes scale |q| |k| (products in any order, the split of q, the
    scales, the rounding of the exponent), which moves a weight by at most a
    factor 1 + 2d (d << 1); the n weights, their sum and the sum of products add
    (n + 40) U32 of sum p |v|.  Weights are held in fp16 halves, scaled so that the
    largest is at least 2^6: the smallest step of fp16 adds 2^-25 / 2^6 of the
    largest weight to each.  fp16 queries round each weight (U16) and the output
    (U16 of it, or half the smallest subnormal)."""
    N, heads, D = q.shape
    slots, H, _ = k_rows.shape
    G = heads // H
    pages = slots // page
    out = out0.double().clone()
    bound = torch.zeros_like(out)
    width = table.shape[1]
    for r in range(len(lens)):
        a, b = max(starts[r], 0), min(starts[r + 1], N)
        T = min(max(b - a, 0), max_new)
        L = min(max(lens[r], 0), width * page)
        tot = min(L + T, width * page)
        tok = torch.arange(tot)
        pg = table[r].long()[tok // page]
        there = (pg >= 0) & (pg < pages)
        at = torch.where(there, pg, 0) * page + tok % page
        k, v = k_rows[at].double(), v_rows[at].double()
        if k_scale is not None:
            k, v = k * k_scale.double().view(1, H, 1), v * v_scale.double().view(1, H, 1)
        for i in range(T):
            bits = (int(mask[a + i]) & (2 ** 64 - 1)) if mask is not None else (2 << i) - 1
            see = there.clone()
            for j in range(L, tot):
                see[j] = bool(see[j]) and bool(bits >> (j - L) & 1)
            idx = see.nonzero().view(-1)
            for hq in range(heads):
                if idx.numel() == 0:
                    out[a + i, hq] = 0.0
                    continue
                qq, kk, vv = q[a + i, hq].double(), k[idx, hq // G], v[idx, hq // G]
                s = kk @ qq * scale
                mag = (kk.abs() @ qq.abs() * abs(scale)).nan_to_num(0, 0, 0).max()
                p = torch.softmax(s, 0)
                out[a + i, hq] = (p[:, None] * vv).sum(0)
                d = (D + 16) * U32 * float(mag)
                rel = 2 * d * (1 + d) + (idx.numel() + 40) * U32 + (U16 if q16 else 0.0)
                bound[a + i, hq] = rel * (p[:, None] * vv.abs()).sum(0) + \
                    2.0 ** -31 * p.max() * vv.abs().sum(0)
                if q16:
                    bound[a + i, hq] += U16 * out[a + i, hq].abs() + 2.0 ** -25
    return out, bound


def close(got, ref, bound, any_odd=False):
    """Elementwise |got - ref| <= bound, equal where ref is not finite (any_odd:
    NaN or an infinity there)."""
    got, ref = got.double(), ref.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), "other elements are finite"
    if not any_odd:
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        inf = ~fin & ~torch.isnan(ref)
        assert torch.equal(got[inf], ref[inf])
    off = (got - ref).abs()[fin] - bound.expand_as(ref)[fin]
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 0.0, f"{worst} past the bound; largest error " \
                         f"{float((got - ref).abs()[fin].max())}"


def tree_bits(rnd, n):
    """Ancestor bits, itself included, of a random tree in drafting order."""
    bits = []
    for i in range(n):
        parent = rnd.randint(-1, i - 1)
        bits.append((bits[parent] if parent >= 0 else 0) | 1 << i)
    return bits


def as_int64(bits):
    return torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64)


assert math.isclose(U32, torch.finfo(torch.float32).eps / 2)
