"""The paged cache on the GPU against a model of its contract in plain Python
(every table entry, length and count, and every symbol of every token), and a
run of the calls as a serving program makes them, with the coder between."""
import random

import numpy as np
import pytest
import torch

from lossless_kv_cache_scalar_amd import skv, synth
from gpu_util import DEV, ensure_built, gpu_calibrate
from pages_util import Model, Refused, attention, tolerance, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def fill(pages, m, seed):
    """The same symbols in both pools."""
    rng = np.random.RandomState(seed)
    m.pool[...] = rng.randint(0, 256, m.pool.shape).astype(m.pool.dtype) if m.pool.dtype == np.uint8 else \
        rng.randint(-32768, 32768, m.pool.shape).astype(np.int16)
    pages.pool.copy_(torch.from_numpy(m.pool))


def same(pages, m):
    assert np.array_equal(pages.table.cpu().numpy(), m.table)
    assert np.array_equal(pages.lens.cpu().numpy(), m.lens)
    assert np.array_equal(pages.refs.cpu().numpy(), m.refs)
    pool = pages.pool.cpu().numpy()
    got = Model(m.sh)
    got.pool, got.table, got.lens = pool, m.table, m.lens
    for s in range(m.sh.max_seqs):
        assert np.array_equal(got.sequence(s), m.sequence(s)), s


def both(pages, m, name, *args):
    """One call on each side; the same verdict."""
    code = skv.OK
    try:
        getattr(m, name)(*args)
    except Refused as e:
        code = e.args[0]
    getattr(pages, name)(*[None if a is None else ints(a) for a in args])
    assert int(pages.status.item()) == code, (name, args)
    pages.status.zero_()
    return code


@pytest.mark.parametrize("fmt,D,P,heads,layers", [(0, 64, 16, 2, 3), (1, 8, 16, 3, 2), (1, 16, 32, 1, 1), (0, 8, 256, 1, 2), (0, 512, 16, 1, 1),
                                                  (1, 128, 64, 5, 2)])
def test_any_order_of_calls(fmt, D, P, heads, layers):
    """Calls in random order, padded places and refused ones among them: the cache equals the model after each."""
    rng = random.Random(100 * D + P)
    sh = skv.pages_shape(layers, heads, D, P, 37, 9, 6, fmt)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, 1)
    same(pages, m)
    codes = set()
    for step in range(60):
        rows = list(range(9))
        rng.shuffle(rows)
        n = rng.randint(1, 7)
        seqs = [s if rng.random() < 0.9 else -1 for s in rows[:n]]
        op = rng.choice(["extend", "extend", "fork", "fork", "truncate", "compact"])
        if op == "extend":
            if rng.random() < 0.05 and n > 1:
                seqs[0] = seqs[-1]
            codes.add(both(pages, m, "extend", seqs, [rng.choice([0, 1, 1, 3, P - 1, P, P + 1, 2 * P]) for _ in seqs]))
        elif op == "fork":
            free = [s for s in rows if m.lens[s] == 0] + [rows[0]] * (rng.random() < 0.1)
            held = [s for s in rows if m.lens[s] > 0] or [rows[1]]
            dst = free[: rng.randint(1, 4)]
            src = [rng.choice(held) for _ in dst]
            part = [rng.randint(0, int(m.lens[s])) for s in src] if rng.random() < 0.5 else None
            codes.add(both(pages, m, "fork", src, dst, part))
        elif op == "truncate":
            keep = None if rng.random() < 0.3 else [rng.randint(0, int(m.lens[s]) + (rng.random() < 0.1)) if s >= 0 else 0 for s in seqs]
            codes.add(both(pages, m, "truncate", seqs[:2], keep and keep[:2]))
        else:
            live = pages.compact()
            assert int(live.item()) == m.compact() and int(pages.status.item()) == skv.OK
        same(pages, m)
    assert skv.OK in codes and len(codes) > 1


def test_forks_growing_together_share_the_last_page_no_longer():
    """Four forks of one sequence of 21 tokens: with the parent alive each copies; with it freed the last keeps the page."""
    sh = skv.pages_shape(2, 2, 64, 16, 40, 8, 4)
    for free_parent in (False, True):
        pages, m = skv.Pages(sh), Model(sh)
        fill(pages, m, 2)
        both(pages, m, "extend", [0], [21])
        both(pages, m, "fork", [0, 0, -1, 0, 0], [1, 2, 6, 3, 4])
        if free_parent:
            both(pages, m, "truncate", [0], None)
        both(pages, m, "extend", [3, 1, 4, 2], [1, 1, 30, 1])
        same(pages, m)
        own = m.table[[3, 1, 4, 2], 1]
        assert len(set(own.tolist())) == 4 and (m.refs[own] == 1).all() and m.refs[m.table[1, 0]] == (4 if free_parent else 5)


def test_larger_lists_than_a_workgroup():
    """3000 listed rows, and a pool of 5000 pages with scattered holes."""
    sh = skv.pages_shape(1, 1, 8, 16, 5003, 3001, 3, skv.SYM_E4M3)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, 3)
    rng = random.Random(5)
    rows = list(range(3001))
    rng.shuffle(rows)
    both(pages, m, "extend", rows[:3000], [rng.choice([0, 1, 16, 17]) for _ in range(3000)])
    same(pages, m)
    both(pages, m, "truncate", rows[:2000], [rng.randint(0, int(m.lens[s])) for s in rows[:2000]])
    free = [s for s in rows if m.lens[s] == 0]
    held = [s for s in rows if m.lens[s] > 0]
    both(pages, m, "fork", [rng.choice(held) for _ in free[:1500]], free[:1500])
    same(pages, m)
    both(pages, m, "extend", rows[:3000], [rng.choice([0, 1]) for _ in range(3000)])
    same(pages, m)
    assert int(pages.compact().item()) == m.compact()
    same(pages, m)
    both(pages, m, "extend", rows[:3000], [17] * 3000)  # too few pages: nothing changes
    same(pages, m)
    both(pages, m, "truncate", rows, None)
    assert (m.refs == 0).all() and int(pages.compact().item()) == 0
    same(pages, m)


def test_the_lowest_values_and_refusals():
    sh = skv.pages_shape(1, 1, 64, 16, 4, 3, 4)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, 4)
    assert both(pages, m, "extend", [-1, -1], [5, 5]) == skv.OK
    assert both(pages, m, "extend", [0, 0], [1, 1]) == skv.ERR_ARG
    assert both(pages, m, "extend", [3], [1]) == skv.ERR_ARG
    assert both(pages, m, "extend", [0, 1], [1, -1]) == skv.ERR_ARG
    assert both(pages, m, "extend", [2], [65]) == skv.ERR_PAGES          # the row overflows
    assert both(pages, m, "extend", [0, 1], [33, 18]) == skv.ERR_PAGES   # five pages of four
    assert both(pages, m, "extend", [0, 2], [64, 0]) == skv.OK           # every page
    assert both(pages, m, "extend", [1], [1]) == skv.ERR_PAGES
    assert both(pages, m, "fork", [0], [0]) == skv.ERR_ARG
    assert both(pages, m, "fork", [0, 0], [1, 1]) == skv.ERR_ARG
    assert both(pages, m, "fork", [0, 1], [1, 2]) == skv.ERR_ARG         # 1 is a target too
    assert both(pages, m, "fork", [0], [3]) == skv.ERR_ARG
    assert both(pages, m, "fork", [0], [1], [65]) == skv.ERR_ARG
    assert both(pages, m, "fork", [0, 2], [1, -1], [0, 9]) == skv.OK     # a prefix of nothing
    assert both(pages, m, "truncate", [0, 0], [1, 1]) == skv.ERR_ARG
    assert both(pages, m, "truncate", [0], [65]) == skv.ERR_ARG
    assert both(pages, m, "truncate", [-1, 0], [7, 64]) == skv.OK
    same(pages, m)
    with pytest.raises(skv.SkvError, match="paged cache"):
        pages.extend(ints([1]), ints([1]))
        pages.check()
    pages.check()  # cleared


def test_broken_tables_are_found():
    """Ids and lengths that do not fit are reported, and nothing outside the arrays is touched."""
    sh = skv.pages_shape(1, 1, 64, 16, 4, 3, 4)
    pages = skv.Pages(sh)
    pages.extend(ints([0, 1]), ints([20, 5]))
    x = torch.zeros(1, 2, 1, 20, 64, dtype=torch.int16, device=DEV)
    one = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV)

    def bad(call):
        call()
        assert int(pages.status.item()) == skv.ERR_ARG
        pages.status.zero_()

    for wrong in (4, -7, 2 ** 31 - 1):
        pages.table[0, 1] = wrong
        bad(lambda: pages.extend(ints([0]), ints([1])))
        bad(lambda: pages.store(0, one, one, ints([0]), ints([17])))
        bad(lambda: pages.gather(0, 0, 20, x))
        bad(lambda: pages.scatter(0, 0, 20, x))
        bad(lambda: pages.compact())
    pages.table[0, 1] = 3
    for wrong in (65, -1, 2 ** 31 - 1):
        pages.lens[0] = wrong
        bad(lambda: pages.extend(ints([0]), ints([0])))
        bad(lambda: pages.truncate(ints([0])))
        bad(lambda: pages.fork(ints([0]), ints([2])))
        bad(lambda: pages.store(0, one, one, ints([0]), ints([64])))
        bad(lambda: pages.compact())


# ---------------------------------------------------------------- store
def e4m3_of(x, scale):
    """e4m3 patterns of bf16 values over a scale per head, by torch's own rounding of the fp32 quotient."""
    y = x.float().cpu() / scale.cpu()[None, :, None]
    y = torch.where(y.isnan(), y, y.clamp(-448, 448))
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("fmt,D,P,heads,n", [(0, 128, 16, 8, 70), (1, 128, 64, 8, 70), (1, 8, 16, 3, 41), (0, 8, 32, 5, 33), (1, 512, 16, 2, 9),
                                             (0, 64, 256, 3, 300), (1, 64, 16, 40, 17), (0, 128, 16, 1, 1)])
def test_store(fmt, D, P, heads, n):
    g = torch.Generator().manual_seed(D + n)
    sh = skv.pages_shape(3, heads, D, P, 64, 5, 4 if P > 64 else 30, fmt)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, 6)
    lens = [n, 0, 7, n // 2 + 1, 1]
    both(pages, m, "extend", range(5), lens)
    places = [(s, t) for s in range(5) for t in range(lens[s])]
    random.Random(n).shuffle(places)
    places = places[:n] + [(-1, 5), (-3, 0)]
    wide = torch.randn(len(places), 3, heads, D, generator=g) * torch.exp(torch.randn(len(places), 3, heads, 1, generator=g))
    wide = wide.to(torch.bfloat16)
    for j, v in enumerate([float("nan"), float("inf"), -float("inf"), -0.0, 448.0, 464.0, 2.0 ** -9, 1.5 * 2.0 ** -9, 2.0 ** -10, 1e-30]):
        wide.view(-1)[j * 7 % wide.numel()] = v
    ks, vs = (0.01 + torch.rand(heads, generator=g), torch.full((heads,), 1.0)) if fmt else (None, None)
    w = wide.to(DEV)
    pages.store(1, w[:, 0], w[:, 2], ints(s for s, _ in places), ints(t for _, t in places), ks.to(DEV) if fmt else None, None)
    pages.check()
    for i, (s, t) in enumerate(places):
        if s >= 0:
            for which, j in ((0, 0), (1, 2)):
                rows = wide[i:i + 1, j].contiguous()
                sym = e4m3_of(rows, vs if which else ks) if fmt else rows.view(torch.int16)
                m.write(s, t, 1, which, sym[0].numpy())
    got, want = pages.pool.cpu().numpy(), m.pool.copy()
    if fmt:  # a NaN may be either of its two patterns
        got, want = np.where((got & 127) == 127, 127, got), np.where((want & 127) == 127, 127, want)
    assert np.array_equal(got, want)  # the whole pool: nothing beside the named places changed


def test_store_every_bf16_value_as_e4m3():
    """All 65536 patterns, with and without a scale."""
    sh = skv.pages_shape(1, 1, 128, 256, 2, 1, 2, skv.SYM_E4M3)
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(512, 1, 128)
    pages = skv.Pages(sh)
    pages.extend(ints([0]), ints([512]))
    for scale in (1.0, 0.3, 7.0, -0.3, 448.0, 1.9999999, 2.0 ** -70, 2.0 ** -60, 2.0 ** 61, 0.0, float("inf"), float("nan")):
        sc = torch.full((1,), scale)
        xd = x.to(DEV)
        pages.store(0, xd, xd, ints([0] * 512), ints(range(512)), sc.to(DEV), None if scale == 1.0 else sc.to(DEV))
        got = pages.gather(0, 0, 512)
        pages.check()
        want = e4m3_of(x, sc)[:, 0]
        for which in (0, 1):
            a, b = got[0, which, 0].cpu(), want
            nan = (b & 127) == 127
            assert torch.equal(a[~nan], b[~nan]) and ((a[nan] & 127) == 127).all()


def test_store_leaves_shared_and_unknown_places_alone():
    sh = skv.pages_shape(1, 2, 64, 16, 8, 4, 4)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, 8)
    both(pages, m, "extend", [0], [20])
    both(pages, m, "fork", [0], [1])
    both(pages, m, "extend", [1], [3])
    one = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    for s, t in ((0, 3), (1, 15), (0, 20), (1, 23), (1, -1), (2, 0), (4, 0), (2 ** 31 - 1, 0)):
        pages.store(0, one, one, ints([s]), ints([t]))
        assert int(pages.status.item()) == skv.ERR_ARG, (s, t)
        pages.status.zero_()
    same(pages, m)
    pages.store(0, one, one, ints([1]), ints([22]))
    pages.check()
    for which in (0, 1):
        m.write(1, 22, 0, which, one[0].cpu().view(torch.int16).numpy())
    same(pages, m)


# ---------------------------------------------------------------- gather, scatter
@pytest.mark.parametrize("fmt,D,P,heads,layers", [(0, 128, 16, 2, 3), (1, 128, 64, 1, 2), (1, 8, 16, 3, 2), (0, 8, 32, 2, 2), (1, 512, 256, 1, 1), (0, 64, 256, 5, 1)])
@pytest.mark.parametrize("first,tokens", [(0, 1), (0, 500), (15, 2), (33, 257), (499, 1), (7, 0), (0, 256)])
def test_gather_scatter(fmt, D, P, heads, layers, first, tokens):
    sh = skv.pages_shape(layers, heads, D, P, 80, 3, -(-500 // P), fmt)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, 9)
    both(pages, m, "extend", [2, 0], [500, 500])
    x = pages.gather(2, first, tokens)
    pages.check()
    want = m.sequence(2)[:, :, :, first:first + tokens]
    assert np.array_equal(x.cpu().numpy(), want)
    pages.scatter(0, first, tokens, x)
    pages.check()
    for t in range(tokens):
        for l in range(layers):
            for which in (0, 1):
                m.write(0, first + t, l, which, want[l, which, :, t])
    assert np.array_equal(pages.pool.cpu().numpy(), m.pool)


def test_gather_scatter_refuse_what_is_not_there():
    sh = skv.pages_shape(1, 1, 64, 16, 8, 3, 4)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, 10)
    both(pages, m, "extend", [0], [20])
    both(pages, m, "fork", [0], [1])
    x = torch.full((1, 2, 1, 21, 64), 77, dtype=torch.int16, device=DEV)
    for call in (lambda: pages.gather(0, 0, 21, x), lambda: pages.gather(0, 20, 1, x), lambda: pages.gather(2, 0, 1, x),
                 lambda: pages.scatter(0, 0, 21, x), lambda: pages.scatter(0, 0, 16, x), lambda: pages.scatter(1, 16, 4, x)):
        call()
        assert int(pages.status.item()) == skv.ERR_ARG
        pages.status.zero_()
    assert (x == 77).all()
    same(pages, m)


def test_beyond_32_bits():
    """A pool of more than 4 GiB a layer: pages at its far end are copied, stored, read and attended like others."""
    n = 70000
    sh = skv.pages_shape(2, 8, 128, 16, n, 3, 4)  # 64 KiB a page and layer, 4.6 GB a layer
    pages = skv.Pages(sh, q_heads=8)
    pages.refs[: n - 6] = 1
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 2, 8, 20, 128, generator=g).to(torch.bfloat16)
    pages.extend(ints([0]), ints([20]))
    pages.scatter(0, 0, 20, x.view(torch.int16).to(DEV))
    pages.fork(ints([0]), ints([2]))
    pages.extend(ints([2]), ints([1]))
    new = torch.randn(1, 8, 128, generator=g).to(torch.bfloat16)
    pages.store(1, new.to(DEV), new.to(DEV), ints([2]), ints([20]))
    pages.check()
    assert pages.table[0, :2].tolist() == [n - 6, n - 5] and pages.table[2, :2].tolist() == [n - 6, n - 4]
    back = pages.gather(2, 0, 20).cpu()
    assert torch.equal(back, x.view(torch.int16))
    q = torch.randn(1, 8, 128, generator=g).to(torch.bfloat16)
    out = pages.attend(1, q.to(DEV), ints([2])).cpu().double()
    whole = torch.cat([x[1].double(), new[0].double().expand(2, 8, 128).unsqueeze(2)], 2)
    ref, lse, absv, mass = attention(q[0].double(), whole, 128 ** -0.5, [1] * 8, [1] * 8)
    tol, _ = tolerance(ref, lse, absv, mass, 21, 128)
    assert ((out[0] - ref).abs() <= tol).all()
    pages.refs[: n - 6] = 0
    assert int(pages.compact().item()) == 3
    pages.check()
    assert torch.equal(pages.gather(2, 0, 20).cpu(), x.view(torch.int16))


# ---------------------------------------------------------------- as a serving program uses them
@pytest.mark.parametrize("fmt", [0, 1])
def test_a_sequence_is_coded_freed_and_restored(fmt):
    """Prompt stored, answers branched and decoded a token at a time, one answer coded, freed, decoded into other
    pages after a compaction: attention over it is the same to the last bit, and right."""
    w = synth.WORKLOADS["qwen3_32b_bf16" if fmt == 0 else "qwen3_32b_e4m3_32k"].with_tokens(300, layers=2)
    heads, D, L = w.kv_heads, w.head_dim, w.layers
    sh = skv.pages_shape(L, heads, D, 16, 120, 6, 24, fmt)
    pages = skv.Pages(sh, q_heads=4 * heads)
    g = torch.Generator().manual_seed(11)
    kv = torch.randn(L, 320, 2, heads, D, generator=g).to(torch.bfloat16).to(DEV)
    sc = torch.full((heads,), 0.05, device=DEV) if fmt else None
    pages.extend(ints([0]), ints([290]))
    for l in range(L):
        pages.store(l, kv[l, :290, 0], kv[l, :290, 1], ints([0] * 290), ints(range(290)), sc, sc)
    pages.fork(ints([0, 0]), ints([1, 2]))
    q = torch.randn(2, 3, 4 * heads, D, generator=g).to(torch.bfloat16).to(DEV)
    for t in range(10):
        pages.extend(ints([1, -1, 2]), ints([1, 1, 1]))
        for l in range(L):
            rows = kv[l, 290 + t: 292 + t]
            pages.store(l, rows[:, 0], rows[:, 1], ints([1, 2]), ints([290 + t] * 2), sc, sc)
    seqs = ints([2, -1, 1])
    before = [pages.attend(l, q[l % 2], seqs, k_scale=sc, v_scale=sc) for l in range(L)]
    x = pages.gather(1, 0, 300)
    pages.check()
    # right: against 64 bits, over what was stored
    scale = [0.05] * heads if fmt else [1.0] * heads
    vals = values(x[0].cpu().numpy(), fmt)
    ref, lse, absv, mass = attention(q[0, 2].cpu().double(), vals, D ** -0.5, scale, scale)
    tol, _ = tolerance(ref, lse, absv, mass, 300, D)
    assert ((before[0][2].cpu().double() - ref).abs() <= tol).all()
    # coded, freed, the pool compacted, and restored
    csh = pages.coder_shape(300)
    mu = values(x.cpu().numpy(), fmt).to(torch.bfloat16).view(torch.int16).to(DEV)
    sigma, hist = skv.calibrate_sequences(csh, [(x, mu)])
    buf = skv.Buffers(csh)
    buf.encode(x, mu, sigma, hist)
    pages.truncate(ints([1, 0]))
    assert int(pages.compact().item()) == -(-300 // 16)  # what row 2 holds
    pages.extend(ints([4]), ints([300]))
    back = torch.empty_like(x)
    buf.decode(mu, sigma, hist, back)
    pages.scatter(4, 0, 300, back)
    pages.check()
    assert int(buf.status.item()) == skv.OK and torch.equal(back, x)
    after = [pages.attend(l, q[l % 2], ints([2, -1, 4]), k_scale=sc, v_scale=sc) for l in range(L)]
    for a, b in zip(before, after):
        assert torch.equal(a, b) and (a[1] == 0).all()


def test_captured_step_replays():
    """A decoding step in a graph: lengths and tables grow from replay to replay, work between them, the same as eager calls."""
    sh = skv.pages_shape(2, 2, 64, 16, 60, 4, 8)

    def fresh():
        p = skv.Pages(sh, q_heads=4)
        p.extend(ints([0, 2]), ints([13, 30]))
        return p

    g = torch.Generator(device=DEV).manual_seed(2)
    steps = [torch.randn(3, 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(6)]
    qs = [torch.randn(3, 4, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(6)]
    x = torch.randn(2, 2, 2, 30, 64, generator=g, device=DEV).to(torch.bfloat16).view(torch.int16)
    one, two = fresh(), fresh()
    for p in (one, two):
        p.scatter(0, 0, 13, x[:, :, :, :13].contiguous())
        p.scatter(2, 0, 30, x)
    seqs, grow = ints([2, -1, 0]), ints([1, 1, 1])
    kv, q, pos = torch.zeros_like(steps[0]), torch.zeros_like(qs[0]), torch.zeros(3, dtype=torch.int32, device=DEV)
    out = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=DEV)

    def step(p):
        p.extend(seqs, grow)
        for l in range(2):
            p.store(l, kv, kv, seqs, pos)
            p.attend(l, q, seqs, out=out[l])

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(one)
    for t in range(6):
        kv.copy_(steps[t])
        q.copy_(qs[t])
        pos.copy_(ints([30 + t, 0, 13 + t]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        step(two)
        torch.cuda.synchronize()
        assert torch.equal(got, out), t
        assert torch.equal(one.table, two.table) and torch.equal(one.lens, two.lens) and torch.equal(one.refs, two.refs)
    one.check()
    two.check()


def test_calls_on_another_stream():
    """Calls given a stream, with the lists made there, while the default stream is busy with other work."""
    sh = skv.pages_shape(1, 2, 64, 16, 20, 4, 8)
    st = torch.cuda.Stream()
    pages = skv.Pages(sh, q_heads=2)
    x = torch.randint(-1000, 1000, (1, 2, 2, 40, 64), dtype=torch.int16, device=DEV)
    torch.cuda.synchronize()
    busy = torch.randn(2048, 2048, device=DEV)
    for _ in range(10):
        busy = busy @ busy * 1e-3
    with torch.cuda.stream(st):
        seqs, grow = ints([1]), ints([40])
        q = torch.randn(1, 2, 64, device=DEV).to(torch.bfloat16)
    for s in (st, st.cuda_stream):
        pages.extend(seqs, grow, stream=s)
        pages.scatter(1, 0, 40, x, stream=s)
        y = pages.gather(1, 0, 40, stream=s)
        out = pages.attend(0, q, seqs, stream=s)
        live = pages.compact(stream=s)
        pages.check(stream=s)
        st.synchronize()
        assert torch.equal(x, y) and int(live.item()) == 3
        # as on the default stream, bit for bit (x holds NaN patterns too)
        assert torch.equal(out.view(torch.int16), pages.attend(0, q, seqs).view(torch.int16))
        pages.truncate(seqs, stream=s)
    st.synchronize()


def test_two_caches_on_two_streams_at_once():
    """Two caches' steps enqueued in turn on two streams, nothing between them waiting: each as alone."""
    g = torch.Generator().manual_seed(9)
    kv = [torch.randn(600, 2, 2, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    q = [torch.randn(3, 8, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    rows, more, forked = ints([0, 1]), ints([590, 5]), ints([2])
    seqs, pos = ints([0] * 590 + [1] * 5), ints(list(range(590)) + list(range(5)))
    one, zero, asked = ints([1]), ints([0]), ints([2, 0, 1])

    def step(pages, i, stream):
        pages.extend(rows, more, stream=stream)
        pages.store(0, kv[i][:595, 0], kv[i][:595, 1], seqs, pos, stream=stream)
        pages.fork(zero, forked, stream=stream)
        pages.extend(forked, one, stream=stream)
        pages.store(0, kv[i][595:596, 0], kv[i][595:596, 1], forked, ints590, stream=stream)
        return pages.attend(0, q[i], asked, stream=stream)

    ints590 = ints([590])
    sh = skv.pages_shape(1, 2, 128, 16, 90, 4, 40)
    alone = [step(skv.Pages(sh, q_heads=8), i, None) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        both_ = [skv.Pages(sh, q_heads=8) for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        outs = [step(both_[i], i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            both_[i].check()
            assert torch.equal(outs[i], alone[i])


def test_captured_page_calls_replay():
    """Fork, growth, compaction and freeing in one graph: each replay as the eager calls on a twin."""
    sh = skv.pages_shape(2, 1, 64, 16, 30, 6, 6)
    one, two = skv.Pages(sh), skv.Pages(sh)
    x = torch.randint(0, 1000, (2, 2, 1, 60, 64), dtype=torch.int16, device=DEV)
    for p in (one, two):
        p.extend(ints([5]), ints([40]))  # pages that the compaction has to pass over later
        p.extend(ints([0, 1]), ints([21, 60]))
        p.scatter(0, 0, 21, x[:, :, :, :21].contiguous())
        p.scatter(1, 0, 60, x)
        p.truncate(ints([5]))
    src, dst, part, grow, keep = ints([0, 1, 0]), ints([2, 3, 4]), ints([21, 50, 5]), ints([1, 1, 20]), ints([0, 1, 0])
    live = [torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2)]

    def step(p, n):
        p.fork(src, dst, part)
        p.extend(dst, grow)
        p.truncate(dst, keep)
        p.compact(n)
        p.truncate(ints3)

    ints3 = ints([3])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(one, live[0])
    for k in range(4):
        graph.replay()
        step(two, live[1])
        torch.cuda.synchronize()
        assert live[0].item() == live[1].item() > 0
        for a, b in ((one.table, two.table), (one.lens, two.lens), (one.refs, two.refs)):
            assert torch.equal(a, b), k
        assert torch.equal(one.gather(1, 0, 60), x) and torch.equal(two.gather(0, 0, 21), x[:, :, :, :21])
    one.check()
    two.check()
