"""A paged cache in plain Python and numpy, one sequence after another, and
attention over it in 64 bits: what the GPU's calls are compared with."""
import numpy as np
import torch

from lossless_kv_cache_scalar_amd import skv


class Refused(Exception):
    pass


class Model:
    """The contract of the page calls, by the letter: lists worked through in order."""

    def __init__(self, sh: skv.SkvPagesShape):
        self.sh = sh
        dt = np.int16 if sh.sym_fmt == skv.SYM_BF16 else np.uint8
        self.pool = np.zeros((sh.layers, sh.n_pages, 2, sh.kv_heads, sh.page_tokens, sh.head_dim), dt)
        self.table = np.full((sh.max_seqs, sh.max_pages), -1, np.int32)
        self.lens = np.zeros(sh.max_seqs, np.int32)
        self.refs = np.zeros(sh.n_pages, np.int32)

    def pages(self, tokens):
        return -(-int(tokens) // self.sh.page_tokens)

    def rows(self, seqs):
        rows = [s for s in seqs if s >= 0]
        if len(set(rows)) < len(rows) or any(s >= self.sh.max_seqs for s in rows):
            raise Refused(skv.ERR_ARG)

    def extend(self, seqs, n_new):
        self.rows(seqs)
        P = self.sh.page_tokens
        if any(s >= 0 and a < 0 for s, a in zip(seqs, n_new)):
            raise Refused(skv.ERR_ARG)
        if any(s >= 0 and self.lens[s] + a > self.sh.max_pages * P for s, a in zip(seqs, n_new)):
            raise Refused(skv.ERR_PAGES)
        free = [p for p in range(self.sh.n_pages) if self.refs[p] == 0]
        refs, table, lens, copies = self.refs.copy(), self.table.copy(), self.lens.copy(), []
        for s, a in zip(seqs, n_new):
            if s < 0 or a == 0:
                continue
            old = int(lens[s])
            want = []
            if old % P and refs[table[s, old // P]] > 1:
                want.append(old // P)
            want += range(self.pages(old), self.pages(old + a))
            for k in want:
                if not free:
                    raise Refused(skv.ERR_PAGES)
                page = free.pop(0)
                if k < self.pages(old):
                    copies.append((table[s, k], page, old % P))
                    refs[table[s, k]] -= 1
                refs[page] = 1
                table[s, k] = page
            lens[s] = old + a
        for src, dst, n in copies:
            self.pool[:, dst, :, :, :n] = self.pool[:, src, :, :, :n]
        self.refs, self.table, self.lens = refs, table, lens

    def fork(self, src, dst, n_tokens=None):
        pairs = [(s, d, None if n_tokens is None else n_tokens[i]) for i, (s, d) in enumerate(zip(src, dst)) if s >= 0 and d >= 0]
        self.rows([d for _, d, _ in pairs])
        if any(s >= self.sh.max_seqs for s, _, _ in pairs) or {s for s, _, _ in pairs} & {d for _, d, _ in pairs}:
            raise Refused(skv.ERR_ARG)
        for s, d, n in pairs:
            if self.lens[d] or (n is not None and not 0 <= n <= self.lens[s]):
                raise Refused(skv.ERR_ARG)
        for s, d, n in pairs:
            n = int(self.lens[s] if n is None else n)
            k = self.pages(n)
            self.table[d, :k] = self.table[s, :k]
            for page in self.table[d, :k]:
                self.refs[page] += 1
            self.lens[d] = n

    def truncate(self, seqs, keep=None):
        self.rows(seqs)
        keep = [0] * len(seqs) if keep is None else keep
        if any(s >= 0 and not 0 <= n <= self.lens[s] for s, n in zip(seqs, keep)):
            raise Refused(skv.ERR_ARG)
        for s, n in zip(seqs, keep):
            if s < 0:
                continue
            for k in range(self.pages(n), self.pages(self.lens[s])):
                self.refs[self.table[s, k]] -= 1
                self.table[s, k] = -1
            self.lens[s] = n

    def compact(self):
        used = [p for p in range(self.sh.n_pages) if self.refs[p] > 0]
        live = len(used)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in used if p >= live]
        for src, dst in zip(movers, holes):
            self.pool[:, dst] = self.pool[:, src]
            self.refs[dst], self.refs[src] = self.refs[src], 0
            self.table[self.table == src] = dst
        return live

    def sequence(self, s):
        """[layers][2][kv_heads][tokens][head_dim] of a sequence."""
        n = int(self.lens[s])
        x = self.pool[:, self.table[s, : self.pages(n)]]
        x = x.transpose(0, 2, 3, 1, 4, 5).reshape(self.sh.layers, 2, self.sh.kv_heads, -1, self.sh.head_dim)
        return x[:, :, :, :n]

    def write(self, s, t, layer, which, rows):
        """One token's symbols [kv_heads][head_dim]."""
        P = self.sh.page_tokens
        self.pool[layer, self.table[s, t // P], which, :, t % P] = rows


def values(x, fmt):
    """float64 values of symbol patterns (a numpy array)."""
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.view(torch.bfloat16) if fmt == skv.SYM_BF16 else t.view(torch.float8_e4m3fn)).double()


def attention(q, x, scale, k_scale, v_scale):
    """out [q_heads][head_dim], lse [q_heads], and for the tolerance sum w |v| and max sum |q k| scale, in
    float64.  q [q_heads][head_dim]; x [2][kv_heads][tokens][head_dim] symbol values."""
    hq, d = q.shape
    h, n = x.shape[1], x.shape[2]
    out, absv = torch.zeros(hq, d, dtype=torch.float64), torch.zeros(hq, d, dtype=torch.float64)
    lse, mass = torch.full((hq,), -float("inf"), dtype=torch.float64), torch.zeros(hq, dtype=torch.float64)
    if n == 0:
        return out, lse, absv, mass
    for j in range(hq):
        k, v = x[0, j // (hq // h)], x[1, j // (hq // h)]
        a = scale * float(k_scale[j // (hq // h)])
        z = k @ q[j] * a
        lse[j] = torch.logsumexp(z, 0)
        w = torch.exp(z - lse[j])
        out[j] = (w @ v) * float(v_scale[j // (hq // h)])
        absv[j] = (w @ v.abs()) * float(v_scale[j // (hq // h)])
        mass[j] = (k.abs() @ q[j].abs()).max() * abs(a)
    return out, lse, absv, mass


def tolerance(out, lse, absv, mass, n, d):
    """How far a fp32 computation with probabilities in bf16 may be from the 64-bit one.

    A score is a sum of d exact products in fp32 and a few roundings of the
    scaled value: off by at most dz = (d + 8) 2^-24 sum |q k| scale.  A weight is
    off by the factor exp(dz) of its score and of the others' (2 dz in all), the
    roundings of the exponential, the rescaling and the sums over n tokens
    (n + 64 half-ulps of fp32), and half a step of bf16 (2^-8).  The result is rounded
    to bf16 (2^-8 of it, or half the smallest step).
    """
    dz = (d + 8) * 2.0 ** -24 * mass
    sums = (n + 64) * 2.0 ** -24
    near = (2.0 ** -8 + 1.01 * (2 * dz + sums))[:, None] * absv
    tol_out = near * (1 + 2.0 ** -8) + 2.0 ** -8 * out.abs() + 2.0 ** -133
    finite = torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))
    return tol_out, dz + sums + 2.0 ** -22 * (finite.abs() + 1)
