"""The page selection's search for the smallest kept score, step by step as the
kernel makes it (numpy, every float32 operation rounded as there), and scores
that bring it to the ends of its parts."""
import numpy as np

FEW = 256          # so many scores are ranked one by one
LEAST_RANGE = np.float32(1e-30)


def order_keys(x):
    """Unsigned integers that order like the floats: +-0 equal, NaN on top."""
    x = np.ascontiguousarray(x, np.float32)
    u = (x + np.float32(0)).view(np.uint32)
    k = np.where(u & 0x80000000, ~u, u | np.uint32(0x80000000)).astype(np.int64)
    return np.where(np.isnan(x), 0xFFFFFFFF, k)


def key_score(k):
    k = np.uint32(k)
    return np.array([k ^ np.uint32(0x80000000) if k & 0x80000000 else ~k], np.uint32).view(np.float32)[0]


def parts_of(x, bins):
    """Each score's part of the range, or None where the range is not taken in parts."""
    keys = order_keys(x)
    low = key_score(keys.min())
    with np.errstate(over="ignore", invalid="ignore"):
        span = np.float32(key_score(keys.max()) - low)
    if not (span >= LEAST_RANGE and span < np.inf):
        return None
    scale = np.float32(bins - 1) / span
    return np.minimum(((x - low) * scale).astype(np.int64), bins - 1)


class Picked(Exception):
    """More scores picked than were counted."""


def kept(x, want, bins, cut_at_end=True):
    """The kept indices (ascending) of the scores x float32 [n], 0 < want < n, with `bins` parts (1024 or 2048).

    cut_at_end False: a chosen piece of keys is as wide as all others though its part ends inside it.  Raises Picked
    where the kernel would then rank or count keys of the next part as well."""
    x = np.ascontiguousarray(x, np.float32)
    keys, bits = order_keys(x), {1024: 10, 2048: 11}[bins]
    lo, hi, left, width, cut = int(keys.min()), int(keys.max()), want, 0xFFFFFFFF, None

    def find(of):
        """The threshold's part, the scores above it, the scores in it."""
        n = np.bincount(of[of < bins], minlength=bins)
        above = n[::-1].cumsum()[::-1] - n
        at = np.flatnonzero((above < left) & (above + n >= left))
        if len(at) != 1:
            raise Picked(f"{len(at)} parts hold the threshold")
        return int(at[0]), int(above[at[0]]), int(n[at[0]])

    def rank(mask, count):
        k = np.sort(keys[mask])[::-1]
        if len(k) != count:
            raise Picked(f"{len(k)} picked of {count}")
        at = int(k[left - 1])
        return at, left - int((k > at).sum())

    part = parts_of(x, bins)
    if part is not None:
        chosen, above, count = find(part)
        left -= above
        if count <= FEW:
            cut, left = rank(part == chosen, count)
        else:
            lo, hi = int(keys[part == chosen].min()), int(keys[part == chosen].max())
            width = hi - lo + 1
    shift = max(0, (hi - lo).bit_length() - bits)
    while cut is None:
        inside = (keys >= lo) & (keys - lo < width)
        piece, above, count = find(np.where(inside, (keys - lo) >> shift, bins))
        left -= above
        lo += piece << shift
        width = min(1 << shift, hi - lo + 1) if cut_at_end else 1 << shift
        if shift == 0:
            cut = lo
        elif count == left:
            cut, left = lo - 1, 0
        elif count <= FEW:
            cut, left = rank((keys >= lo) & (keys - lo < width), count)
        else:
            shift = max(0, shift - bits)
    equal = np.flatnonzero(keys == cut)[:left]
    return np.sort(np.concatenate([np.flatnonzero(keys > cut), equal]))


def sorted_kept(x, want):
    """The same by a sort: the largest first, equal ones by index."""
    return np.sort(np.lexsort((np.arange(len(x)), -order_keys(x)))[:want])


def border_wants(x, bins):
    """Numbers of kept scores whose threshold lies in the last piece of a part that is searched by keys, where that
    piece as wide as all others would reach scores of the next part."""
    part, keys, bits = parts_of(x, bins), order_keys(x), {1024: 10, 2048: 11}[bins]
    wants = []
    for p, n in enumerate(np.bincount(part, minlength=bins)):
        if n <= FEW:
            continue
        own = keys[part == p]
        lo, hi = int(own.min()), int(own.max())
        shift = max(0, (hi - lo).bit_length() - bits)
        last = lo + ((hi - lo) >> shift << shift)
        if ((keys > hi) & (keys < last + (1 << shift))).any():
            above = int((keys > hi).sum())
            wants += range(above + 1, above + int((own >= last).sum()) + 1)
    return [w for w in wants if 0 < w < len(x)]


def scores_across_an_end(n, bins, close, equal, seed):
    """n scores float32 in mixed order over parts one wide: 601 in the part [1, 2) that do not reach its end, `close`
    within its last steps, `equal` of exactly 2 (the next part's first), the rest in [3, 4), and 0 and bins - 1."""
    rng = np.random.default_rng(seed)
    step = 2.0 ** -23
    inner = np.concatenate([[1 + 3000 * step], rng.uniform(1 + 3000 * step, 1.9, 600)])
    x = np.concatenate([[0, bins - 1], inner, 2 - step * np.arange(1, close + 1), np.full(equal, 2.0)])
    x = np.concatenate([x, rng.uniform(3, 3.999, n - len(x))]).astype(np.float32)
    return rng.permutation(x)


def scores_below_one_far_above(n, seed, far=1000.0):
    """n scores float32, normally distributed but for one far above, so that few parts hold all others."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(n).astype(np.float32)
    x[rng.integers(n)] = far
    return x
