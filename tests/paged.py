"""Small paged-cache problems for the tests: numpy inputs, the oracle's outputs and their bounds.

Everything a kernel has no business reading is poisoned: rows of the pages that no position reaches
(NaN scales, all-ones codes) and table entries behind a sequence's last page (far out of range).
"""
import numpy as np

from oracle import oracle as O

D = 128


def pack(codes, bits):
    return O.pack_int4(codes) if bits == 4 else codes


def quantize(x, bits):
    codes, scale, zero, v = (O.quant_asym_uint4 if bits == 4 else O.quant_asym_uint8)(x)
    return codes, scale, zero, v


def round_bf16(x):
    return O.round_bf16(np.asarray(x, np.float64))


class Pool:
    """Page arrays (numpy) and block tables of sequences with the given numbers of rows."""

    def __init__(self, rng, lengths, page, hkv, bits, width=None, spare=2, poison=True):
        per = [-(-n // page) for n in lengths]
        total = sum(per) + spare
        self.page, self.hkv, self.bits = page, hkv, bits
        order = rng.permutation(total)
        width = (max(per) if per else 0) + 1 if width is None else width
        self.table = np.full((len(lengths), width), 1 << 29, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.arrays = {}
        for key in ("k", "v"):
            self.arrays[key + "_codes"] = np.full((total, hkv, page, D * bits // 8), 0xFF, np.uint8)
            self.arrays[key + "_scale"] = np.full((total, hkv, page), np.nan if poison else 1.0, np.float32)
            self.arrays[key + "_zero"] = np.full((total, hkv, page), 3, np.uint8)

    def put(self, b, key, x):
        """Quantizes x [n, hkv, D] into the rows of sequence b; returns the values it stands for."""
        codes, scale, zero, _ = quantize(x, self.bits)
        pos = np.arange(x.shape[0])
        pages, rows = self.table[b, pos // self.page], pos % self.page
        self.arrays[key + "_codes"][pages, :, rows] = pack(codes, self.bits)
        self.arrays[key + "_scale"][pages, :, rows] = scale
        self.arrays[key + "_zero"][pages, :, rows] = zero
        return O.dequant_asym(codes, scale, zero)


class Attention:
    """A ragged batch over pages, optionally behind a shared prefix."""

    def __init__(self, seed, new, own, hq=8, hkv=2, page=16, bits=4, prefix=0, pad=0, scale=None,
                 softcap=0.0, window=0, slopes=False, q_size=1.5, k_size=1.0, v_size=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.own, self.hq, self.hkv, self.prefix = list(new), list(own), hq, hkv, prefix
        self.rule = dict(scale=scale, softcap=softcap, window=window)
        self.slopes = (2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)).astype(np.float32) if slopes else None
        self.pool = Pool(rng, list(own) + [prefix], page, hkv, bits)
        self.T = sum(new) + pad
        self.q = round_bf16(q_size * rng.standard_normal((self.T, hq, D)))
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.values = {}
        for key, size in (("k", k_size), ("v", v_size)):
            for b, n in enumerate(list(own) + [prefix]):
                x = size * rng.standard_normal((n, hkv, D)) * np.exp(0.3 * rng.standard_normal((n, hkv, 1)))
                self.values[key, b] = self.pool.put(b, key, x.astype(np.float32)) if n else np.zeros((0, hkv, D))

    def table(self):
        return self.pool.table[:len(self.new)]

    def prefix_table(self):
        return self.pool.table[len(self.new), :-(-self.prefix // self.pool.page)]

    def reference(self):
        """(out, lse, spread, size) of the packed rows; rows behind the last sequence are NaN."""
        out = np.full((self.T, self.hq, D), np.nan)
        lse, spread, size = np.full((self.T, self.hq), np.nan), np.zeros((self.T, self.hq, D)), 0.0
        last = len(self.new)
        for b, (n, own) in enumerate(zip(self.new, self.own)):
            K, V = (np.concatenate([self.values[k, last], self.values[k, b]]) for k in ("k", "v"))
            qpos = self.prefix + own - n + np.arange(n)
            rows = slice(self.cu[b], self.cu[b] + n)
            o, m, s, z = O.causal_attention(self.q[rows], K, V, qpos, np.arange(self.prefix + own),
                                            slopes=self.slopes, **self.rule)
            out[rows], lse[rows], spread[rows] = o, m, s
            size = max(size, z)
        return out, lse, spread, size

    def bounds(self, ref, weight_eps, weight_step=2.0 ** -37):
        """Elementwise bounds of out and lse.

        A score's error: its exact products are summed in float32 in 8 steps of 16, each sum off by at
        most 2^-22 of the summed magnitudes (`size`) even if the adder truncates: 8 * 2^-22 = 2^-19.
        Its scalings (four float32 products) and, with a cap, tanh to 2^-20 of the cap add 2^-21 |s| and
        cap 2^-20; with slopes, slope * distance is rounded at 2^-24 of itself (below 2^-20 (1 + size)
        here).  Together e = 2^-18 (1 + size) + cap 2^-20.
        A weight is then off by e relatively, and by its own rounding and exp's, `weight_eps`; the output
        is a quotient of two such sums, so by 2 (e + weight_eps) spread, and bf16 rounds it by 2^-8.
        Weights (times the value's scale) far below a row's largest are held in fixed steps: half a step
        of fp16's smallest, 2^-25, where the largest weight is 2^14 or more and the scales are measured in
        a power of two at most four times the largest: each key adds 2^-25 2^-14 4 top, with top the
        largest scale times code, at most the range of the codes times the scale.  That is 2^-37, the
        streaming kernel's `weight_step`; where the largest weight is 2^10 or more and the scales are
        measured in a power of two at most eight times the largest (the tile kernel) it is
        2^-25 2^-10 8 = 2^-32."""
        out, lse, spread, size = ref
        e = 2.0 ** -18 * (1 + size) + self.rule["softcap"] * 2.0 ** -20
        top = max(float(np.abs(v).max()) if v.size else 0.0 for (k, _), v in self.values.items() if k == "v")
        top *= 2                                     # an asymmetric grid's other end is no further than its range
        step = (self.prefix + max(self.own, default=0)) * weight_step * top
        return (2.0 ** -8 * np.abs(out) + 2 * (e + weight_eps) * spread + step + 1e-30,
                e + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0))))
