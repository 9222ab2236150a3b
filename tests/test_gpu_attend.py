"""Attention over pages against the formula in 64 bits, within bounds that count the roundings."""
import numpy as np
import pytest
import torch

from lossless_kv_cache_scalar_amd import skv
from gpu_util import DEV, ensure_built
from pages_util import attention, tolerance, values

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


class Case:
    """A cache whose sequences have the given lengths, their tokens random, everything else in the pool NaN."""

    def __init__(self, fmt, lens, D, P, kv_heads, q_heads, layers=2, seed=0, spread=1.0):
        self.fmt, self.lens, self.D = fmt, lens, D
        need = sum(-(-n // P) for n in lens)
        sh = skv.pages_shape(layers, kv_heads, D, P, need + 3, len(lens) + 1, max(1, -(-max(lens) // P)) + 1, fmt)
        self.pages = skv.Pages(sh, q_heads=q_heads)
        self.pages.pool.fill_(0x7FC0 if fmt == skv.SYM_BF16 else 0x7F)
        self.g = torch.Generator().manual_seed(1000 * D + 10 * P + seed)
        # pages in scattered order: every page taken, given back one by one, and taken again by the sequences
        perm = torch.randperm(need + 3, generator=self.g)[:need].to(torch.int32)
        table = torch.full((sh.max_seqs, sh.max_pages), 2 ** 31 - 1, dtype=torch.int32)  # nothing behind the last page is looked at
        at = 0
        for s, n in enumerate(lens):
            k = -(-n // P)
            table[s, :k] = perm[at:at + k]
            at += k
        refs = torch.zeros(sh.n_pages, dtype=torch.int32)
        refs[perm.long()] = 1
        self.pages.table.copy_(table)
        self.pages.lens.copy_(torch.tensor(lens + [0], dtype=torch.int32))
        self.pages.refs.copy_(refs)
        self.x = {}
        for s, n in enumerate(lens):
            x = torch.randn(layers, 2, kv_heads, n, D, generator=self.g) * spread * torch.exp(0.5 * torch.randn(layers, 2, kv_heads, 1, D, generator=self.g))
            sym = x.to(torch.bfloat16).view(torch.int16) if fmt == skv.SYM_BF16 else x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.x[s] = sym
            if n:
                self.pages.scatter(s, 0, n, sym.contiguous().to(DEV))
        self.pages.check()
        self.k_scale = self.v_scale = None
        self.kv_heads, self.q_heads, self.layers = kv_heads, q_heads, layers
        if fmt == skv.SYM_E4M3:
            self.k_scale = 0.5 + torch.rand(kv_heads, generator=self.g)
            self.v_scale = 0.5 + torch.rand(kv_heads, generator=self.g)

    def q(self, n):
        return torch.randn(n, self.q_heads, self.D, generator=self.g).to(torch.bfloat16)

    def dev(self, t):
        return None if t is None else t.to(DEV)

    def attend(self, layer, q, seqs, **kw):
        n = len(seqs)
        out = torch.full((n, self.q_heads, self.D), 77.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((n, self.q_heads), 55.0, device=DEV)
        self.pages.attend(layer, q.to(DEV) if q.device.type == "cpu" else q, ints(seqs), k_scale=self.dev(self.k_scale),
                          v_scale=self.dev(self.v_scale), out=out, lse=lse, **kw)
        self.pages.check()
        return out.cpu().double(), lse.cpu().double()

    def compare(self, layer, q, seqs, out, lse, scale=None):
        one = torch.ones(self.kv_heads)
        for i, s in enumerate(seqs):
            if s < 0:
                assert (out[i] == 77).all() and (lse[i] == 55).all()
                continue
            n = self.lens[s]
            x = values(self.x[s][layer].numpy(), self.fmt).view(2, self.kv_heads, n, self.D)
            ref = attention(q[i].double(), x, self.D ** -0.5 if scale is None else scale, self.k_scale if self.k_scale is not None else one,
                            self.v_scale if self.v_scale is not None else one)
            tol_out, tol_lse = tolerance(*ref, n, self.D)
            if n == 0:
                assert (out[i] == 0).all() and (lse[i] == -INF).all()
                continue
            assert torch.isfinite(out[i]).all(), (s, n)
            assert ((out[i] - ref[0]).abs() <= tol_out).all(), (s, n, ((out[i] - ref[0]).abs() / tol_out).max())
            assert ((lse[i] - ref[1]).abs() <= tol_lse).all(), (s, n, ((lse[i] - ref[1]).abs() / tol_lse).max())


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 64, 65, 255, 257, 1000]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D,P,kv_heads,group", [(128, 16, 2, 8), (128, 64, 8, 2), (64, 32, 2, 5), (64, 16, 1, 1), (256, 16, 1, 4), (32, 16, 3, 3),
                                                (16, 16, 2, 4), (8, 16, 2, 2), (512, 16, 1, 2), (128, 256, 1, 16), (128, 16, 1, 17), (64, 128, 2, 40),
                                                (512, 256, 2, 20), (8, 256, 1, 33)])
def test_against_64_bits(fmt, D, P, kv_heads, group):
    c = Case(fmt, LENS, D, P, kv_heads, kv_heads * group)
    seqs = [12, 3, -1, 0, 5, 1, 7, 2, 11, 4, 6, -1, 8, 9, 10, 12, 13]  # 13: a free row; 12 twice
    c.lens = LENS + [0]
    c.x[13] = c.x[0]
    q = c.q(len(seqs))
    for layer in (1, 0):
        out, lse = c.attend(layer, q, seqs)
        c.compare(layer, q, seqs, out, lse)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [1, 2, 100, 4097, 20000])
def test_one_sequence(fmt, n):
    """Few rows over a long axis: the split and the join."""
    c = Case(fmt, [n], 128, 16, 2, 8, layers=1, seed=n)
    q = c.q(1)
    out, lse = c.attend(0, q, [0])
    c.compare(0, q, [0], out, lse)


@pytest.mark.parametrize("fmt", [0, 1])
def test_long_ragged_batch(fmt):
    lens = [9000, 1, 0, 40, 5003, 17, 0, 300]
    c = Case(fmt, lens, 64, 64, 4, 8, layers=1)
    q = c.q(8)
    out, lse = c.attend(0, q, list(range(8)))
    c.compare(0, q, list(range(8)), out, lse)


@pytest.mark.parametrize("rows", [64, 65, 128, 257, 1000, 6000])
def test_many_rows(rows):
    """More rows than a workgroup has threads, padded and empty ones among them."""
    lens = [(7 * i) % 50 for i in range(120)]
    c = Case(0, lens, 64, 16, 1, 2, layers=1)
    seqs = [i % 120 if i % 11 else -1 for i in range(rows)]
    q = c.q(rows)
    out, lse = c.attend(0, q, seqs)
    c.compare(0, q, seqs, out, lse)


def test_rows_beyond_the_first_four_thousand():
    """Long rows at both ends of a list whose places between are padded, empty or short."""
    c = Case(1, [3000, 5, 0, 2500], 64, 64, 2, 4, layers=1)
    seqs = [0] + [(-1, 2, 1)[i % 3] for i in range(4300)] + [3, 0]
    q = c.q(len(seqs))
    out, lse = c.attend(0, q, seqs)
    pick = [0, 1, 2, 3, 64, 66, 4298, 4299, 4300, 4301, 4302]
    c.compare(0, q[pick], [seqs[i] for i in pick], out[pick], lse[pick])


@pytest.mark.parametrize("fmt,D,kv_heads,group", [(0, 128, 8, 2), (1, 64, 4, 20), (0, 512, 2, 33)])
def test_one_long_row_among_many_short_ones(fmt, D, kv_heads, group):
    """Rows too short to be shared by waves, and one that spans many of them."""
    lens = [(11 * i) % 61 for i in range(150)] + [9001]
    c = Case(fmt, lens, D, 16, kv_heads, kv_heads * group, layers=1)
    seqs = list(range(0, 150, 2)) + [150, -1] + list(range(1, 150, 2)) + list(range(40))
    q = c.q(len(seqs))
    out, lse = c.attend(0, q, seqs)
    c.compare(0, q, seqs, out, lse)


def test_all_rows_padded_or_empty():
    c = Case(0, [0, 5], 64, 16, 2, 4)
    for seqs in ([-1], [0], [-1, -1, 0], [2, 0]):
        c.lens = [0, 5, 0]
        c.x[2] = c.x[0]
        q = c.q(len(seqs))
        out, lse = c.attend(0, q, seqs)
        c.compare(0, q, seqs, out, lse)


def test_strided_queries_and_scale():
    """Queries as a part of a wider projection's rows; a scale of one's own, zero and negative ones too; no lse."""
    c = Case(0, [100, 33, 7], 128, 32, 2, 6)
    wide = torch.randn(3, 10, 128, generator=c.g).to(torch.bfloat16)
    q, qd = wide[:, 2:8], wide.to(DEV)[:, 2:8]
    for scale in (None, 0.3, 0.0, -0.05):
        out, lse = c.attend(1, qd, [2, 0, 1], scale=scale)
        c.compare(1, q, [2, 0, 1], out, lse, scale)
        alone = c.pages.attend(1, qd, ints([2, 0, 1]), scale=scale).cpu().double()
        assert torch.equal(alone, out)


@pytest.mark.parametrize("fmt", [0, 1])
def test_large_scores(fmt):
    """Scores in the hundreds: one token has all the weight, and the maximum moves late and early."""
    c = Case(fmt, [700, 129, 64], 128, 16, 1, 4, spread=20.0, layers=1)
    q = c.q(3) * 3
    out, lse = c.attend(0, q, [0, 1, 2])
    c.compare(0, q, [0, 1, 2], out, lse)


def test_special_values():
    """Infinities and NaN among the tokens do what the formula does with them, and nothing outside their rows."""
    c = Case(0, [100, 100, 100, 100], 64, 16, 1, 2, layers=1)
    q = c.q(4).abs() + 0.1
    ninf, inf, nan = -128, 0x7F80, 0x7FC0  # -inf is 0xFF80

    def put(s, which, t, v):
        p = int(c.pages.table[s, t // 16])
        c.pages.pool[0, p, which, 0, t % 16] = v

    for t in range(100):
        put(0, 0, t, ninf)          # every score -inf: no weight at all
        if t % 3 == 0:
            put(1, 0, t, ninf)      # some tokens without weight
            c.x[1][0, 0, 0, t] = ninf
    put(2, 0, 50, nan)              # a score that is not a number
    put(3, 1, 99, inf)              # a value without bound
    out, lse = c.attend(0, q, [0, 1, 2, 3])
    assert (out[0] == 0).all() and (lse[0] == -INF).all()
    assert out[2].isnan().all() and lse[2].isnan().all()
    assert (out[3] == INF).all() and torch.isfinite(lse[3]).all()
    keep = torch.tensor([t % 3 != 0 for t in range(100)])
    x = values(c.x[1][0].numpy(), 0).view(2, 1, 100, 64)[:, :, keep]
    ref = attention(q[1].double(), x, 64 ** -0.5, [1], [1])
    tol_out, tol_lse = tolerance(*ref, 100, 64)
    assert ((out[1] - ref[0]).abs() <= tol_out).all() and ((lse[1] - ref[1]).abs() <= tol_lse).all()


@pytest.mark.parametrize("fmt", [0, 1])
def test_one_token_gives_its_value_back(fmt):
    """With one token the weight is 1: every finite symbol comes out as the value it stands for, subnormal ones too."""
    D = 512 if fmt == 0 else 256
    c = Case(fmt, [1] * (65536 // D if fmt == 0 else 1), D, 16, 1, 1, layers=1)
    n = len(c.lens)
    pat = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16) if fmt == 0 else torch.arange(256, dtype=torch.int32).to(torch.uint8)
    pat = pat.view(n, D)
    for s in range(n):
        x = c.x[s].clone()
        x[0, 1, 0, 0] = pat[s]
        c.pages.scatter(s, 0, 1, x.to(DEV))
    c.v_scale = c.k_scale = None
    out = c.pages.attend(0, c.q(n).to(DEV), ints(range(n)))
    c.pages.check()
    want = values(pat.numpy(), fmt)
    fine = torch.isfinite(want)
    assert torch.equal(out.cpu().double().view(n, D)[fine], want[fine])


def test_scores_of_subnormal_keys():
    """A query picks one channel of keys that are subnormal e4m3 symbols: the scores are those values times the query's."""
    c = Case(1, [256], 64, 16, 1, 1, layers=1)
    x = c.x[0].clone()
    x[0, 0] = 0
    x[0, 0, 0, :, 5] = torch.arange(256, dtype=torch.int32).to(torch.uint8)  # one key for each symbol
    x[0, 0, 0, [127, 255], 5] = 0
    c.pages.scatter(0, 0, 256, x.to(DEV))
    c.x[0] = x
    c.k_scale = torch.ones(1)
    c.v_scale = torch.ones(1)
    for big in (1.0, 1024.0):
        q = torch.zeros(1, 1, 64)
        q[0, 0, 5] = big
        q = q.to(torch.bfloat16)
        out, lse = c.attend(0, q, [0], scale=1.0)
        c.compare(0, q, [0], out, lse, 1.0)


def test_broken_lists_are_reported_and_other_rows_right():
    c = Case(0, [40, 300, 20], 64, 16, 2, 4)
    q = c.q(3)
    for what, wrong in (("table", c.pages.shape.n_pages), ("table", -5), ("table", 2 ** 31 - 1), ("lens", -1),
                        ("lens", c.pages.shape.max_pages * 16 + 1), ("seqs", 4), ("seqs", 2 ** 31 - 1)):
        keep = (c.pages.table.clone(), c.pages.lens.clone())
        seqs = [0, 1, 2]
        if what == "table":
            c.pages.table[1, 3] = wrong
        elif what == "lens":
            c.pages.lens[1] = wrong
        else:
            seqs[1] = wrong
        out = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(3, 4, device=DEV)
        c.pages.attend(0, q.to(DEV), ints(seqs), out=out, lse=lse)
        with pytest.raises(skv.SkvError, match="invalid argument"):
            c.pages.check()
        sel = [0, 2]
        c.compare(0, q[sel], sel, out.cpu().double()[sel], lse.cpu().double()[sel])
        c.pages.table.copy_(keep[0])
        c.pages.lens.copy_(keep[1])
        out, lse = c.attend(0, q, [0, 1, 2])  # nothing of the bad call stays
        c.compare(0, q, [0, 1, 2], out, lse)


def test_same_bits_every_time_and_in_two_graphs():
    """Two captured graphs and eager calls share one workspace, in any order; every run gives the same bits."""
    c = Case(0, [5000, 3, 700], 128, 16, 2, 8, layers=2)
    q = c.q(3).to(DEV)
    seqs = ints([0, 1, 2])
    want = [c.pages.attend(l, q, seqs).clone() for l in (0, 1)]
    outs, graphs = [torch.zeros_like(w) for w in want], []
    torch.cuda.synchronize()
    for l in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[l]):
            c.pages.attend(l, q, seqs, out=outs[l])
    for k in range(5):
        for l in ((0, 1), (1, 0))[k % 2]:
            outs[l].zero_()
            graphs[l].replay()
            assert torch.equal(c.pages.attend(1 - l, q, seqs), want[1 - l])
            torch.cuda.synchronize()
            assert torch.equal(outs[l], want[l])
    c.pages.check()
    c.pages.attend_workspace.fill_(0xFF)  # what the workspace holds before a call does not matter
    assert torch.equal(c.pages.attend(0, q, seqs), want[0])


def test_arguments_are_refused_by_name():
    c = Case(0, [20, 9], 64, 16, 2, 4)
    p, q, seqs = c.pages, c.q(2).to(DEV), ints([0, 1])
    for call, name in ((lambda: p.attend(0, q[:, :2], seqs), "q"), (lambda: p.attend(0, q.float(), seqs), "q"),
                       (lambda: p.attend(0, q.cpu(), seqs), "q"), (lambda: p.attend(0, q, seqs.long()), "seqs"),
                       (lambda: p.attend(0, q, seqs.cpu()), "seqs"), (lambda: p.attend(0, q, seqs, out=q[:1]), "out"),
                       (lambda: p.attend(0, q, seqs, lse=torch.zeros(2, 3, device=DEV)), "lse"),
                       (lambda: p.attend(0, q.transpose(0, 1).contiguous().transpose(0, 1), seqs), "q"),
                       (lambda: p.attend(2, q, seqs), "invalid"), (lambda: p.attend(0, q, seqs, scale=INF), "invalid"),
                       (lambda: p.attend(0, q, seqs, k_scale=torch.ones(2, device=DEV)), "invalid"),
                       (lambda: skv.Pages(p.shape).attend(0, q, seqs), "q_heads"),
                       (lambda: p.store(0, q[:, :2], q[:, 1:3, :32], seqs, seqs), "v"),
                       (lambda: p.extend(seqs, ints([1])), "n_new"), (lambda: p.fork(seqs, ints([2])), "dst"),
                       (lambda: p.gather(0, 0, 20, torch.zeros(4, device=DEV)), "x"), (lambda: p.gather(5, 0, 1), "invalid")):
        with pytest.raises(skv.SkvError, match=name):
            call()
    p.check()
