"""Plain 64-bit forms of the paged-cache operators and the bounds the kernels
are held to, for the tests.

Bounds.  A rounding to type t is off by at most half a step, finfo(t).eps / 2
relative.  Attention: the score of a key is a sum of D products in fp32, off by
at most (D + 16) 2^-24 A with A = scale sum_d |q_d k_d| (16 covers the parts q
enters in and the scaling), so a weight p_j is off relatively by twice that of
the largest score (its own and the normaliser's), and by 2^-21 for the two
exponentials; the sums of n weights and products add at most (n / 4 + 64)
2^-24 (sums of 16 positions inside a product, then one after another).  A
softmax weight that enters the product in type t adds eps_t / 2, the output's
rounding eps_t / 2 of it.  All of it times sum_j p_j |v_j|."""
import numpy as np
import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return float(torch.finfo(dtype).eps) / 2


def rope64(max_pos, D, theta=10000.0):
    ang = np.arange(max_pos)[:, None] * theta ** (-2.0 * np.arange(D // 2) / D)
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def rotate(x, c, s):
    """x [..., D] float64, c and s [..., D/2]; also the bound of an fp32 rotation."""
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    y = np.concatenate([a * c - b * s, b * c + a * s], -1)
    m = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)
    return y, 2 * U32 * m


def attend(q, K, V, scale, n_weights_type=None):
    """q [D], K and V [n, D] float64 -> (out [D], the bound without the output's rounding)."""
    s = scale * (K @ q)
    A = scale * (np.abs(K) @ np.abs(q)).max()
    w = np.exp(s - s.max())
    w /= w.sum()
    D, n = K.shape[1], K.shape[0]
    rel = 2 * (D + 16) * U32 * A + 2.0 ** -21 + (n / 4 + 64) * U32
    if n_weights_type is not None:
        rel += half_step(n_weights_type)
    return w @ V, rel * (w @ np.abs(V))


class Pool:
    """Pages of a cache with NaN wherever no test value was written, and the
    table of `lens` positions per sequence in a shuffled order."""

    def __init__(self, rng, lens, Hkv, page, D, dtype, width=None, spare=3):
        need = [-(-n // page) for n in lens]
        self.width = width or max(1, max(need))
        total = sum(need) + spare
        order = rng.permutation(total)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.page, self.Hkv, self.D, self.dtype = page, Hkv, D, dtype
        self.k = torch.full((total, Hkv, page, D), float("nan"), dtype=dtype)
        self.v = torch.full((total, Hkv, page, D), float("nan"), dtype=dtype)

    def where(self, b, positions):
        positions = np.asarray(positions)
        return self.table[b, positions // self.page], positions % self.page

    def put(self, b, positions, k, v):
        pg, sl = self.where(b, positions)
        self.k[pg, :, sl] = torch.from_numpy(np.asarray(k, np.float32)).to(self.dtype)
        self.v[pg, :, sl] = torch.from_numpy(np.asarray(v, np.float32)).to(self.dtype)

    def get(self, pages, b, positions):
        """[len, Hkv, D] float64 of a pool tensor (this one's or the device's, copied back)."""
        pg, sl = self.where(b, positions)
        return pages[pg, :, sl].double().numpy()

    def device(self, q4):
        return q4.KVPages(self.k.cuda(), self.v.cuda(), torch.from_numpy(self.table).cuda())


def check(got, ref, bound, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d out of bounds; first %s: got %r want %r bound %r"
                             % (what, int(bad.sum()), bad.size, i, got[i], ref[i], np.broadcast_to(bound, ref.shape)[i]))
