"""Plain 64-bit forms of the token history, the logit rules and the 4-bit
head, row by row from their definitions, with the error that the kernels'
32-bit arithmetic may add to each value."""
import numpy as np

U32 = 2.0 ** -24                                    # half an ulp, relative
HALF_ULP = {"float32": 0.0, "bfloat16": 2.0 ** -8}  # the final rounding (fp32: counted below)


def unpack(words, V):
    """Truth values [.., V] of bit planes [.., ceil(V / 32)]."""
    w = np.ascontiguousarray(words).view(np.uint32)
    bits = (w[..., None] >> np.arange(32, dtype=np.uint32)) & 1
    return bits.reshape(*w.shape[:-1], -1)[..., :V].astype(bool)


def pack(flags):
    """Bit planes (int32 words) of truth values [.., V]."""
    f = np.asarray(flags, dtype=np.uint64)
    f = np.concatenate([f, np.zeros(f.shape[:-1] + (-f.shape[-1] % 32,), np.uint64)], -1)
    f = f.reshape(*f.shape[:-1], -1, 32)
    return (f << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


class History:
    def __init__(self, R, V):
        self.V = V
        self.prompt = np.zeros((R, V), bool)
        self.counts = np.zeros((R, V), np.int64)

    def add(self, slot, tokens, prompt=False):
        for t in tokens:
            if 0 <= t < self.V:
                if prompt:
                    self.prompt[slot, t] = True
                else:
                    self.counts[slot, t] += 1


def process(z, dtype, drafts, pos0, n_pos, prompt, counts, rep, freq, pres, bias, masks):
    """One row.  z [P, V] float64; drafts: block tokens; n_pos: positions to
    process; bias: {token: value}; masks: one truth vector or None per
    position.  Returns (out [P, V], bound [P, V]); positions from n_pos on
    come back unchanged with bound 0."""
    P, V = z.shape
    out, bound = z.copy(), np.zeros_like(z)
    bvec = np.zeros(V)
    for t, v in bias.items():
        bvec[t] = v
    for p in range(n_pos):
        c = counts.astype(np.float64).copy()
        for x in list(drafts)[:pos0 + p]:
            if 0 <= x < V:
                c[x] += 1
        seen = prompt | (c > 0)
        with np.errstate(all="ignore"):
            z1 = np.where(seen, np.where(z[p] > 0, z[p] / rep, z[p] * rep), z[p])
            fc = freq * c
            z2a = z1 - fc
            z2 = z2a - pres * (c > 0)
            z3 = z2 + bvec
            # one rounding each: z1, the product, and the three sums
            err = U32 * 1.01 * (np.abs(z1) * seen + np.abs(fc) + np.abs(z2a) * (fc != 0) +
                                np.abs(z2) * (c > 0) + np.abs(z3) * (bvec != 0))
            err = err + HALF_ULP[dtype] * (np.abs(z3) + err)
        changed = seen | (bvec != 0)
        out[p] = z3
        bound[p] = np.where(changed, err, 0.0)      # an untouched logit keeps its bits
        if masks[p] is not None:
            out[p][~masks[p]] = -np.inf
            bound[p][~masks[p]] = 0.0
    return out, bound


def head(x, codes, scale, zero, group, dtype):
    """x [M, H], codes [V, H] 0..15, scale and zero [V, G] -> (out [M, V], bound)."""
    M, H = x.shape
    V, G = scale.shape
    w = (codes.reshape(V, G, group).astype(np.float64) - zero[:, :, None])
    ws = (w * scale[:, :, None]).reshape(V, H)
    out = x @ ws.T
    mag = np.abs(x) @ np.abs(ws).T
    # The products are exact.  A group's sum has `group` terms, the row's G
    # scaled sums and a few partial sums across warps and CTAs; the matrix
    # unit may drop what lies below the last bit instead of rounding it (a
    # whole ulp, 2^-23).  Scaling rounds once.
    err = 2.0 ** -23 * (group + G + 16) * mag
    return out, err + HALF_ULP[dtype] * (np.abs(out) + err)


def check(got, want, bound, what=""):
    """Infinities and NaN in the same places, finite values within the bound."""
    got = np.asarray(got, np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = ~nan & ~inf
    assert np.all(np.isfinite(got[fine])), f"{what}: infinite where it should not be"
    over = np.abs(got[fine] - want[fine]) - bound[fine]
    assert over.size == 0 or over.max() <= 0, \
        f"{what}: {int((over > 0).sum())} values past the bound, worst by {over.max():.3g}"
