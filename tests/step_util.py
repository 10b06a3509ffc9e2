"""References of a decode step's other parts (numpy): the plan, the normed and
rotated rows in the kernels' own 32-bit steps and in 64 bits, the digests, the
page scores and the selection.

Tolerances, derived from the formats alone:
  - a normed and rotated value against 64 bits: the sum of squares is off by at
    most 7 roundings of 2^-24 (halved by the root), the root, the reciprocal, the
    two products by one each: 9 * 2^-24 relative; the rotation's two products and
    the sum 2^-24 of |a| + |b| each; then the bf16 rounding, 2^-8 relative.  With
    11 instead of 9 for the second order.  With eps the sum's errors only shrink;
  - a page score: 256 exact products summed up in fp32, each addition off by at most
    2^-23 of the sum of magnitudes, and 5 roundings of the scalings (2^-24 each, taken
    as 2^-21).
"""
import numpy as np
import torch

import oracle

PAGE = 16


def bf16_round(x):
    """float32 -> the nearest bf16 values, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def bits(x):
    """bf16 values held as float32 -> their uint16 patterns."""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def same(got, want, what):
    """The two arrays hold the same bits."""
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape and got.dtype == want.dtype, f"{what}: {got.dtype} {got.shape}, {want.dtype} {want.shape}"
    off = int(np.count_nonzero(got != want))
    first = np.argwhere(got != want)[0].tolist() if off else None
    assert off == 0, f"{what}: {off} of {got.size} differ, the first at {first}: {got[tuple(first)]}, not {want[tuple(first)]}"


def plan_ref(table, cached, new, free, count, num_pages, tokens):
    """The plan's outputs, request by request."""
    table = table.copy()
    batch, cols = table.shape
    lens, slots, positions, rows = [], [], [], []
    cu_q, cu_rows = [0], [0]
    flags, open_ = 0, True
    capacity = len(free)
    if not 0 <= count <= capacity:
        flags |= 4
        count = min(max(count, 0), capacity)
    for b in range(batch):
        c, n = int(cached[b]), int(new[b])
        c2 = min(max(c, 0), cols * PAGE)
        n2 = min(max(n, 0), cols * PAGE - c2)
        if (c, n) != (c2, n2):
            flags |= 4
        c, n = c2, n2
        have, all_ = -(-c // PAGE), -(-(c + n) // PAGE)
        if open_ and (all_ - have > count or len(slots) + n > tokens):
            open_ = False
        if not open_:
            flags |= 32 if n > 0 else 0
            n, all_ = 0, have
        for p in range(have, all_):
            count -= 1
            table[b, p] = free[count]
        for pos in range(c, c + n):
            page = int(table[b, pos // PAGE])
            good = 0 <= page < num_pages
            flags |= 0 if good else 2
            slots.append(page * PAGE + pos % PAGE if good else -1)
            positions.append(pos)
            rows.append(cu_rows[-1] + pos)
        lens.append(c + n)
        cu_q.append(len(slots))
        cu_rows.append(cu_rows[-1] + c + n)
    pad = tokens - len(slots)
    return {"table": table, "lens": lens, "slots": slots + [-1] * pad, "positions": positions + [0] * pad,
            "rows": rows + [-1] * pad, "cu_q": cu_q, "cu_rows": cu_rows, "free_left": [count], "flags": flags}


def _pairs(x, rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm_rope_steps(x, weight, eps, cos_sin, positions, interleaved):
    """x float32 [n, heads, 128] -> the rows before their bf16 rounding, every step rounded to 32 bits."""
    f = np.float32
    x = x.astype(f)
    if weight is not None:
        s = x * x
        while s.shape[-1] > 1:
            s = s[..., 0::2] + s[..., 1::2]
        r = f(1) / np.sqrt(s * f(1.0 / 128) + f(eps))
        x = (x * r) * weight.astype(f)
    if cos_sin is not None and cos_sin.shape[1]:
        half = cos_sin.shape[1] // 2
        ok = (positions >= 0) & (positions < len(cos_sin))
        cs = cos_sin[np.where(ok, positions, 0)][:, None]
        a, b = _pairs(x, 2 * half, interleaved)
        ya = x[..., a] * cs[..., :half] - x[..., b] * cs[..., half:]
        yb = x[..., b] * cs[..., :half] + x[..., a] * cs[..., half:]
        y = x.copy()
        y[..., a], y[..., b] = ya, yb
        x = np.where(ok[:, None, None], y, x)
    return x


def norm_rope_exact(x, weight, eps, cos_sin, positions, interleaved):
    """The same in 64 bits, and the tolerance of the bf16 result."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * weight.astype(np.float64)
    off = 11 * 2.0 ** -24 * np.abs(x) if weight is not None else np.zeros_like(x)
    if cos_sin is not None and cos_sin.shape[1]:
        half = cos_sin.shape[1] // 2
        cs = cos_sin.astype(np.float64)[positions][:, None]
        a, b = _pairs(x, 2 * half, interleaved)
        y, o = x.copy(), off.copy()
        y[..., a] = x[..., a] * cs[..., :half] - x[..., b] * cs[..., half:]
        y[..., b] = x[..., b] * cs[..., :half] + x[..., a] * cs[..., half:]
        size = np.abs(x[..., a]) + np.abs(x[..., b])
        o[..., a] = o[..., b] = off[..., a] + off[..., b] + 3 * 2.0 ** -24 * size
        x, off = y, o
    return x, off + 2.0 ** -8 * (np.abs(x) + off) + 2.0 ** -133


E4M3 = np.array(sorted(oracle.e4m3_value(c) for c in range(127)))       # 0 .. 448


def _toward(x, up):
    """x rounded to E4M3, up or down, from the list of its values."""
    mag = np.abs(x)
    above = E4M3[np.searchsorted(E4M3, mag, side="left")]
    below = E4M3[np.searchsorted(E4M3, mag, side="right") - 1]
    return np.where(x >= 0, 1.0, -1.0) * np.where((x >= 0) == up, above, below)


def digest_ref(K):
    """hi, lo (as the E4M3 values of the digest) and scale of a page's keys [tokens, 128] without the global scale."""
    hi, lo = K.max(0), K.min(0)
    most = max(np.abs(hi).max(), np.abs(lo).max())
    scale = 2.0 ** (np.floor(np.log2(most)) - 7) if most > 0 else 1.0
    return _toward(hi / scale, True), _toward(lo / scale, False), scale


def e4m3_values(raw):
    table = np.array([oracle.e4m3_value(c) for c in range(256)])
    return table[raw]


def score_ref(q, hi, lo, scale, factor):
    """The page's score and its tolerance for the group's queries q [G, 128] in 64 bits."""
    u = np.maximum(q * hi, q * lo).sum(-1)
    size = np.maximum(np.abs(q * hi), np.abs(q * lo)).sum(-1) + np.minimum(np.abs(q * hi), np.abs(q * lo)).sum(-1)
    tol = (256 * 2.0 ** -23 * size + 2.0 ** -21 * np.abs(u)).max()
    return u.max() * scale * factor, tol * scale * factor + 2.0 ** -126
