"""The serving ops on the GPU, each against a plain float64 implementation on the CPU, at the
sizes, masks and contents where they can go wrong, and a run of them together.

Tolerances.  u = 2^-24 (half a step of fp32), and for bf16 outputs h = 2^-8 (half a step of bf16).
A sum of n products in fp32, in any order, is off by at most n * u * sum |products| to first
order, twice that where the tensor cores may cut instead of round.

* attention: a score q.k/sqrt(d) is off by E = 2 (d + 3) u |q||k| / sqrt(d); a weight
  p = exp(s - m), and the sum of the weights, by a relative 2 E + (len + 8) u each (the
  exponential's own error is a few u); so an output by (4 E + 3 (len + 8) u) * sum w |v|, to which
  the tensor-core form adds h * sum w |v| (p is rounded to bf16 for the product with v) and a bf16
  output h |out|.
* adapters: the shared product is off by 2 (K + 4) u sum |x||W|, a shrink value by
  2 (K + 4) u sum |x||A| scale, plus h times itself where it is rounded to bf16, and the expand by
  2 (rank + 4) u sum |S||B|; a bf16 output by h |y| more.
"""
import math
import random

import pytest
import torch

from gpu_util import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

U, H = 2.0 ** -24, 2.0 ** -8
BF, FP = torch.bfloat16, torch.float32


def i32(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ---- block tables ---------------------------------------------------------------------------

def tables_ref(old, new, table, ring, head, count, p, max_tokens):
    table, ring = [list(r) for r in table], list(ring)
    n, take, put = len(ring), head, head + count
    free = list(ring)
    cu, slots = [0], []
    for r, (a, b) in enumerate(zip(old, new)):
        for j in range(-(-a // p), -(-b // p)):
            table[r][j] = free[take % n]
            take += 1
        for j in range(-(-b // p), -(-a // p)):
            ring[put % n] = table[r][j]
            put += 1
        slots += [table[r][i // p] * p + i % p for i in range(a, b)]
        cu.append(len(slots))
    return table, ring, [take % n, put - take, 0, 0], cu, slots + [-1] * (max_tokens - len(slots))


def tables_case(seed, R, p, lo, hi, grow, ends, spare=3):
    r = random.Random(seed)
    old = [r.randint(lo, hi) for _ in range(R)]
    new = [0 if r.random() < ends else max(0, a + r.randint(*grow)) for a in old]
    have = [-(-a // p) for a in old]
    blocks = max([1] + have + [-(-b // p) for b in new])
    need = sum(max(0, -(-b // p) - h) for b, h in zip(new, have))
    n = sum(have) + need + spare
    pages = list(range(n))
    r.shuffle(pages)
    table, k = [], 0
    for h in have:
        table.append(pages[k:k + h] + [-7] * (blocks - h))
        k += h
    head = r.randrange(n)
    ring = [-9] * n
    for i, pg in enumerate(pages[k:]):
        ring[(head + i) % n] = pg
    return old, new, table, ring, head, n - k


@pytest.mark.parametrize("R,p,lo,hi,grow,ends", [
    (1, 16, 0, 0, (1, 1), 0.0), (1, 8, 0, 0, (0, 0), 0.0), (3, 16, 15, 17, (1, 1), 0.0),
    (64, 16, 0, 300, (1, 1), 0.1), (257, 32, 0, 500, (-200, 200), 0.2), (40, 256, 0, 2000, (0, 700), 0.0),
    (593, 8, 0, 90, (-20, 40), 0.1), (1500, 16, 0, 40, (0, 3), 0.3), (2, 8, 0, 3, (5000, 5000), 0.0),
    (9, 64, 64, 64, (0, 64), 0.5)])
def test_block_tables_match_the_definition(R, p, lo, hi, grow, ends):
    from zeroth_order_fine_b200 import zo
    old, new, table, ring, head, count = tables_case(R * 7 + p, R, p, lo, hi, grow, ends)
    toks = sum(max(0, b - a) for a, b in zip(old, new))
    want = tables_ref(old, new, table, ring, head, count, p, toks + 3)
    t, g, s, s2 = i32(table), i32(ring), i32([head, count, 5, 6]), i32([0] * 4)
    for _ in range(2):                 # the state is read from one array, written to another:
        cu, slots = zo.zo_op_block_tables(i32(old), i32(new), t, g, s, s2, p, max_tokens=toks + 3)
        got = [x.cpu().tolist() for x in (t, g, s2, cu, slots)]
        assert got == [list(x) for x in want]     # so a second call gives the same


@pytest.mark.parametrize("what", ["pages", "negative", "long", "tokens", "overflow", "head", "count"])
def test_block_tables_refuse_a_step_as_a_whole(what):
    from zeroth_order_fine_b200 import zo
    p, blocks = 16, 4
    old, new = [16, 0, 30], [40, 20, 10]             # takes 2 + 2 pages, gives one back
    table = [[0, -1, -1, -1], [-1] * 4, [1, 2, -1, -1]]
    ring = [3, 4, 5, 6, 7, 0, 0, 0]
    head, count, toks, status = 0, 5, 44, 0
    if what == "pages":
        count, status = 1, 3
    elif what == "negative":
        old, status = [16, -1, 30], -1
    elif what == "long":
        new, status = [65, 20, 10], -1
    elif what == "tokens":
        toks, status = 43, -2
    elif what == "overflow":
        count, status = 8, -3
    elif what == "head":
        head, status = 8, -4
    elif what == "count":
        count, status = -1, -4
    t, g, s, s2 = i32(table), i32(ring), i32([head, count, 0, 0]), i32([9] * 4)
    cu, slots = zo.zo_op_block_tables(i32(old), i32(new), t, g, s, s2, p, max_tokens=toks)
    assert s2.tolist() == [head, count, status, 0]
    assert t.tolist() == table and g.tolist() == ring
    assert cu.tolist() == [0] * 4 and slots.tolist() == [-1] * toks


def test_block_tables_of_no_requests():
    from zeroth_order_fine_b200 import zo
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    ring, s = zo.zo_page_ring(4)
    s2 = i32([0] * 4)
    cu, slots = zo.zo_op_block_tables(e, e, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), ring,
                                      s, s2, 16, max_tokens=2)
    assert cu.tolist() == [0] and slots.tolist() == [-1, -1] and s2.tolist() == [0, 4, 0, 0]


# ---- cache write ------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,Hq,Hkv,hd,wide,off", [(1, 1, 1, 128, 0, 0), (37, 4, 2, 64, 0, 0),
                                                  (300, 8, 8, 128, 24, 0), (5, 3, 1, 33, 1, 1),
                                                  (64, 2, 2, 8, 0, 3)])
def test_kv_write(dt, T, Hq, Hkv, hd, wide, off):
    from zeroth_order_fine_b200 import zo
    g = torch.Generator().manual_seed(T)
    cols = (Hq + 2 * Hkv) * hd
    base = torch.randn(T, cols + wide + off, generator=g).to(dt).cuda()
    qkv = base[:, off:off + cols]                     # a column slice: strided, maybe not 16-byte
    n = 2 * T + 5
    slots = torch.randperm(n, generator=g)[:T].int()
    slots[::5] = -1
    if T > 3:
        slots[1], slots[2], slots[3] = n, -2 ** 31, 2 ** 31 - 1
    cache = torch.full((n, 2 * Hkv * hd), 3.0, dtype=dt, device="cuda")
    zo.zo_op_kv_write(qkv, slots.cuda(), cache, Hq, Hkv, hd)
    want = torch.full((n, 2 * Hkv * hd), 3.0, dtype=dt)
    for t in range(T):
        if 0 <= slots[t] < n:
            want[slots[t]] = qkv[t, Hq * hd:].cpu()
    assert torch.equal(cache.cpu(), want)


# ---- attention over the pages -------------------------------------------------------------------

class Paged:
    """Requests with (cached before, new) tokens in a shuffled paged cache whose every other row,
    and every table entry behind a request's end, is poison."""

    def __init__(self, reqs, Hq, Hkv, hd, p, dt, seed=0, extra=2, tail=2, blocks=0):
        r, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.reqs, self.Hq, self.Hkv, self.hd, self.p, self.dt = reqs, Hq, Hkv, hd, p, dt
        self.lens = [a + b for a, b in reqs]
        used = [-(-n // p) for n in self.lens]
        self.blocks = max(used + [1]) + 1 + blocks
        n_pages = sum(used) + extra
        pages = list(range(n_pages))
        r.shuffle(pages)
        self.cache = torch.full((n_pages * p, 2 * Hkv * hd), float("nan"), dtype=dt)
        self.cache[::3] = float("inf")
        self.table, self.kv, k = [], [], 0
        for n, u in zip(self.lens, used):
            mine = pages[k:k + u]
            k += u
            self.table.append(mine + [r.choice([-1, 2 ** 31 - 1, -2 ** 31, n_pages, 0])
                                      for _ in range(self.blocks - u)])
            rows = torch.randn(n, 2 * Hkv * hd, generator=g).to(dt)
            for i in range(n):
                self.cache[mine[i // p] * p + i % p] = rows[i]
            self.kv.append(rows)
        self.cu = [0]
        for a, b in reqs:
            self.cu.append(self.cu[-1] + b)
        self.T = self.cu[-1] + tail
        self.q = (torch.randn(self.T, (Hq + 2 * Hkv) * hd, generator=g) * 1.5).to(dt)
        self.max_new = max([b for _, b in reqs] + [0])

    def args(self):
        return (self.cache.cuda(), i32(self.table), self.p, i32(self.cu), i32(self.lens))

    def run(self, impl=0, max_new=None, out=None, ws=None):
        from zeroth_order_fine_b200 import zo
        return zo.zo_op_attention_paged(self.q.cuda(), *self.args(),
                                        self.max_new if max_new is None else max_new, self.Hq, self.Hkv,
                                        self.hd, impl=impl, out=out, ws=ws)

    def check(self, out, impl, skip=()):
        """Every row against float64 and its bound; tensor cores round p to bf16."""
        out, g = out.double().cpu(), self.Hq // self.Hkv
        for r, (a, b) in enumerate(self.reqs):
            if r in skip or b == 0:
                continue
            n, hd = a + b, self.hd
            rows = self.kv[r].double().view(n, 2, self.Hkv, hd)
            q = self.q[self.cu[r]:self.cu[r + 1], :self.Hq * hd].double().view(b, self.Hq, hd)
            for h in range(self.Hq):
                k, v = rows[:, 0, h // g], rows[:, 1, h // g]
                s = q[:, h] @ k.T / math.sqrt(hd)
                s = s.masked_fill(torch.ones(b, n, dtype=torch.bool).triu(a + 1), -math.inf)
                w = torch.softmax(s, -1)
                ref, mag = w @ v, w @ v.abs()
                e = 2 * (hd + 3) * U * q[:, h].norm(dim=1) * k.norm(dim=1).max() / math.sqrt(hd)
                rel = 4 * e[:, None] + 3 * (n + 8) * U
                if self.dt == BF:
                    rel = rel + (H if impl != 1 else 0.0)
                tol = rel * mag + (H * ref.abs() if self.dt == BF else 0.0)
                err = (out[self.cu[r]:self.cu[r + 1], h * hd:(h + 1) * hd] - ref).abs()
                assert torch.all(err <= tol), (r, h, (err / tol).max())


LAYOUTS = [(4, 4, 128), (8, 2, 128), (4, 4, 64), (6, 2, 64)]
BATCHES = {
    "single": [(0, 1)], "one-old": [(1, 1)], "edge": [(15, 1), (16, 1), (127, 1), (128, 1), (129, 1)],
    "steps": [(3, 1), (250, 1), (64, 1), (511, 1), (0, 1), (777, 1)],
    "prompts": [(0, 1), (0, 2), (0, 127), (0, 128), (0, 129), (0, 33)],
    "chunks": [(100, 60), (7, 130), (640, 1), (31, 257), (0, 0), (300, 2)],
    "mixed": [(0, 5), (400, 1), (5, 0), (90, 17), (0, 0), (33, 1), (255, 3)],
}


@pytest.mark.parametrize("impl", [0, 1])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("lay", range(len(LAYOUTS)))
def test_attention_paged(name, lay, dt, impl):
    from zeroth_order_fine_b200 import zo
    if dt == FP and impl == 0:
        pytest.skip("the same kernels as impl 1")
    Hq, Hkv, hd = LAYOUTS[lay]
    p = [16, 64, 8, 32][lay]
    c = Paged(BATCHES[name], Hq, Hkv, hd, p, dt, seed=lay)
    out = torch.full((c.T, Hq * hd), 7.0, dtype=dt, device="cuda")
    c.run(impl, out=out)
    assert zo.zo_op_error_word() == 0
    c.check(out, impl)
    assert torch.all(out[c.cu[-1]:] == 7.0)           # rows behind the last request


@pytest.mark.parametrize("Hq,Hkv,hd,p", [(1, 1, 128, 256), (16, 1, 128, 128), (24, 1, 64, 16),
                                         (5, 1, 128, 8), (40, 8, 64, 8), (7, 7, 128, 32),
                                         (128, 1, 64, 64), (2, 1, 32, 16), (3, 1, 256, 16)])
@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_paged_head_groups(Hq, Hkv, hd, p, dt):
    c = Paged([(70, 1), (0, 19), (200, 3), (9, 40)], Hq, Hkv, hd, p, dt, seed=Hq)
    tc = dt == BF and hd in (64, 128)
    c.check(c.run(), 0 if tc else 1)


def test_attention_paged_long_and_few():
    """One request over a long cache (its keys split over the SMs), alone and beside short ones."""
    for reqs in ([(9000, 1)], [(9000, 40)], [(5000, 1), (3, 1), (12000, 2)], [(4000, 300), (17, 1)]):
        c = Paged(reqs, 4, 1, 128, 32, BF, seed=len(reqs))
        c.check(c.run(), 0)


def test_attention_paged_many_requests():
    r = random.Random(5)
    c = Paged([(r.randint(0, 40), r.choice([0, 1, 1, 1, 2])) for _ in range(1300)], 2, 1, 64, 8, BF,
              seed=3)
    c.check(c.run(), 0)
    r = random.Random(6)
    c = Paged([(r.randint(0, 30), r.choice([0, 1, 30])) for _ in range(700)], 2, 2, 128, 16, BF, seed=4)
    c.check(c.run(), 0)


@pytest.mark.parametrize("max_new", [0, 1, 1000])
def test_attention_paged_with_a_wrong_hint(max_new):
    c = Paged([(30, 50), (200, 1), (0, 140), (64, 9)], 8, 2, 128, 16, BF)
    c.check(c.run(max_new=max_new), 0)


@pytest.mark.parametrize("old,new", [(300, 1), (0, 3), (77, 0), (5, 40), (2000, 5), (0, 700)])
@pytest.mark.parametrize("lay", [(8, 2, 128), (6, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("max_new", [1, 1000])
def test_attention_paged_of_a_request_alone(old, new, lay, max_new):
    """One request, whichever kernel the hint picks."""
    c = Paged([(old, new)], *lay, 16, BF)
    c.check(c.run(max_new=max_new), 0)


@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_paged_of_one_long_among_short(dt):
    """An item of many pieces beside whole ones; tiles of every number of rows."""
    reqs = [(4000, 1)] + [(r.randrange(0, 90), r.randrange(1, 6)) for r in [random.Random(4)] for _ in range(40)]
    c = Paged(reqs, 4, 2, 64, 32, dt)
    c.check(c.run(), 0 if dt == BF else 1)
    reqs = [(900, n) for n in (8, 9, 16, 17, 32, 33, 64, 65)]
    c = Paged(reqs, 2, 2, 64, 16, dt)
    c.check(c.run(impl=1), 1)


@pytest.mark.parametrize("dt,impl", [(BF, 0), (BF, 1), (FP, 1)])
@pytest.mark.parametrize("kind", ["page", "page-negative", "short", "long", "rows"])
def test_attention_paged_bad_requests(kind, dt, impl):
    """A bad page or length gives its own request NaN and leaves the others; rows that are not
    inside the batch are left out."""
    reqs = [(40, 1), (100, 1), (60, 30), (300, 200), (5, 1)]
    for bad in (1, 3):
        c = Paged(reqs, 4, 2, 128, 16, dt, seed=bad)
        out = torch.full((c.T, 4 * 128), 7.0, dtype=dt, device="cuda")
        if kind == "page":
            c.table[bad][2] = c.cache.shape[0] // 16
        elif kind == "page-negative":
            c.table[bad][0] = -2 ** 31
        elif kind == "short":
            c.lens[bad] = reqs[bad][1] - 1
        elif kind == "long":
            c.lens[bad] = c.blocks * 16 + 1
        else:
            c.cu[5] = c.T + 1                          # the last request: past the batch
            c.run(impl, out=out)
            c.cu[5] = c.T - 2
            c.check(out, impl, skip=(4,))
            assert torch.all(out[c.cu[4]:] == 7.0)
            continue
        c.run(impl, out=out)
        c.check(out, impl, skip=(bad,))
        assert torch.isnan(out[c.cu[bad]:c.cu[bad + 1]]).all()
        assert torch.all(out[c.cu[-1]:] == 7.0)


def test_attention_paged_strides_and_other_stream():
    from zeroth_order_fine_b200 import zo
    c = Paged([(30, 1), (0, 70), (129, 1)], 4, 2, 128, 16, BF)
    wide = torch.zeros(c.T, c.q.shape[1] + 40, dtype=BF, device="cuda")
    wide[:, 8:8 + c.q.shape[1]] = c.q.cuda()
    store = torch.full((c.T, 4 * 128 + 24), 7.0, dtype=BF, device="cuda")
    args = c.args()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        zo.zo_op_attention_paged(wide[:, 8:8 + c.q.shape[1]], *args, c.max_new, 4, 2, 128,
                                 out=store[:, 8:8 + 512])
    st.synchronize()
    c.check(store[:, 8:520], 0)
    assert torch.all(store[:, :8] == 7.0) and torch.all(store[:, 520:] == 7.0)
    # an offset that is no multiple of 16 bytes: the CUDA cores take it
    odd = torch.full((c.T, 4 * 128 + 3), 7.0, dtype=BF, device="cuda")
    zo.zo_op_attention_paged(c.q.cuda(), *args, c.max_new, 4, 2, 128, out=odd[:, 1:513])
    c.check(odd[:, 1:513], 0)


def test_attention_paged_extreme_scores():
    """Scores of 10^4 and more, all keys alike, and one key far above the rest."""
    c = Paged([(200, 1), (100, 150)], 4, 2, 128, 16, BF)
    for r in range(2):
        c.kv[r][:, :256] *= 0
        c.kv[r][5, :256] = 40.0
    for r, n in enumerate(c.lens):
        for i in range(n):
            c.cache[c.table[r][i // 16] * 16 + i % 16] = c.kv[r][i]
    c.q[:] = c.q.abs() * 4
    out = c.run().double().cpu()
    for r, (a, b) in enumerate(c.reqs):
        q0 = c.cu[r]
        for i in range(b):
            v = c.kv[r][:, 256:].double().view(-1, 2, 128)
            want = v[5] if a + i >= 5 else v[:a + i + 1].mean(0)
            got = out[q0 + i].view(2, 2, 128)
            assert torch.allclose(got, want[:, None].expand(2, 2, 128), rtol=2 * H, atol=1e-3)


def test_attention_paged_in_a_graph_follows_the_arrays():
    """A captured call reads lengths, tables and offsets anew at each replay."""
    from zeroth_order_fine_b200 import zo
    a = Paged([(20, 1), (300, 1), (64, 60)], 8, 2, 128, 16, BF, seed=1, extra=40, blocks=10)
    b = Paged([(119, 40), (7, 1), (260, 21)], 8, 2, 128, 16, BF, seed=2, extra=39, blocks=5)
    rows, blocks = max(a.cache.shape[0], b.cache.shape[0]), max(a.blocks, b.blocks)
    q = torch.zeros(a.T, a.q.shape[1], dtype=BF, device="cuda")
    cache = torch.zeros(rows, a.cache.shape[1], dtype=BF, device="cuda")
    table = torch.zeros(3, blocks, dtype=torch.int32, device="cuda")
    cu, lens = i32([0] * 4), i32([0] * 3)
    out = torch.zeros(a.T, 8 * 128, dtype=BF, device="cuda")
    ws = torch.empty(zo.zo_op_attention_paged_workspace(a.T, 3, 8, 2, 128), dtype=torch.uint8,
                     device="cuda")

    def load(c):
        q.copy_(c.q[:a.T])
        cache[:c.cache.shape[0]] = c.cache.cuda()
        table[:, :c.blocks] = i32(c.table)
        cu.copy_(i32(c.cu))
        lens.copy_(i32(c.lens))

    assert a.T == b.T
    load(a)
    call = lambda: zo.zo_op_attention_paged(q, cache, table, 16, cu, lens, 60, 8, 2, 128, out=out, ws=ws)
    call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for c in (b, a, b):
        load(c)
        out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        c.check(out, 0)
    assert zo.zo_op_error_word() == 0


def test_attention_paged_is_deterministic():
    c = Paged([(700, 1), (33, 1), (2000, 1)], 8, 2, 128, 16, BF)
    x = c.run()[:c.cu[-1]]             # the rows behind the last request are not written
    for _ in range(3):
        assert torch.equal(c.run()[:c.cu[-1]], x)


# ---- adapters ---------------------------------------------------------------------------------

def adapt_case(M, N, K, n, r, ids, dt, seed=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(dt)
    W = (torch.randn(N, K, generator=g) * K ** -0.5).to(dt)
    A = (torch.randn(n * r, K, generator=g) * K ** -0.5).to(dt)
    B = (torch.randn(N, n * r, generator=g) * r ** -0.5).to(dt)
    sc = torch.rand(n, generator=g) * 2 - 0.5
    b = torch.randn(N, generator=g) if bias else None
    return x, W, A, B, i32(ids, "cpu"), sc, b


def adapt_ref(x, W, A, B, ids, sc, b, n, r, bf16, tc):
    x, W, A, B, sc = (t.double() for t in (x, W, A, B, sc))
    M, K = x.shape
    y = x @ W.T
    tol = 2 * (K + 4) * U * (x.abs() @ W.abs().T)
    for a in range(n):
        at = (ids == a).nonzero().flatten()
        if not len(at):
            continue
        Aa, Ba = A[a * r:(a + 1) * r], B[:, a * r:(a + 1) * r]
        S = sc[a] * (x[at] @ Aa.T)
        eS = 2 * (K + 4) * U * abs(sc[a]) * (x[at].abs() @ Aa.abs().T) + (H if tc else 0.0) * S.abs()
        y[at] += S @ Ba.T
        tol[at] += eS @ Ba.abs().T + 2 * (r + 4) * U * (S.abs() @ Ba.abs().T)
    if b is not None:
        y += b.double()
        tol += 2 * U * (y.abs() + b.double().abs())
    tol += 4 * U * y.abs()
    return y, tol + (H * y.abs() if bf16 else 0.0)


def spans(M, n, seed, lo=1, hi=40):
    r, ids = random.Random(seed), []
    while len(ids) < M:
        ids += [r.randrange(-1, n)] * r.randint(lo, hi)
    return ids[:M]


ADAPT = [(1, 256, 64, 1, 8, 1, 1), (1, 512, 1024, 3, 16, 1, 1), (7, 264, 200, 4, 8, 1, 1),
         (48, 1024, 512, 32, 16, 1, 1), (100, 640, 328, 9, 64, 1, 3), (128, 384, 256, 5, 24, 1, 1),
         (129, 512, 256, 6, 16, 1, 1), (300, 1000, 512, 7, 16, 10, 90), (257, 256, 128, 40, 8, 1, 4),
         (513, 768, 640, 3, 128, 1, 300), (1000, 520, 264, 20, 40, 5, 30), (600, 136, 72, 2, 256, 50, 300),
         (260, 64, 64, 4, 16, 3, 60)]


@pytest.mark.parametrize("impl", [0, 1])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("case", range(len(ADAPT)))
def test_linear_adapters(case, act, dt, impl):
    from zeroth_order_fine_b200 import zo
    if dt == FP and impl == 0:
        pytest.skip("the same kernels as impl 1")
    M, N, K, n, r, lo, hi = ADAPT[case]
    ids = spans(M, n, case, lo, hi)
    c = adapt_case(M, N, K, n, r, ids, dt, seed=case, bias=case % 3 != 0)
    y = zo.zo_op_linear_adapters(*(t.cuda() for t in c[:6]), bias=None if c[6] is None else c[6].cuda(),
                                 act=act, impl=impl)
    assert zo.zo_op_error_word() == 0
    ref, tol = adapt_ref(*c, n, r, dt == BF, dt == BF and impl != 1)
    ref = torch.relu(ref) if act else ref
    err = (y.double().cpu() - ref).abs()
    assert torch.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("dt,impl", [(BF, 0), (BF, 1), (FP, 1)])
@pytest.mark.parametrize("M", [3, 120, 400])
def test_linear_adapters_accumulate(M, dt, impl):
    from zeroth_order_fine_b200 import zo
    N, K, n, r = 320, 192, 5, 16
    c = adapt_case(M, N, K, n, r, spans(M, n, M), dt, seed=M)
    y0 = torch.randn(M, N, generator=torch.Generator().manual_seed(9))
    y = y0.cuda().clone()
    zo.zo_op_linear_adapters(*(t.cuda() for t in c[:6]), bias=c[6].cuda(), accumulate=True, out=y,
                             impl=impl)
    ref, tol = adapt_ref(*c, n, r, False, dt == BF and impl != 1)
    err = (y.double().cpu() - ref - y0.double()).abs()
    assert torch.all(err <= tol + 2 * U * (ref.abs() + y0.double().abs()))


@pytest.mark.parametrize("dt,impl", [(BF, 0), (BF, 1), (FP, 1)])
@pytest.mark.parametrize("M", [5, 90, 500])
@pytest.mark.parametrize("act", [0, 1])
def test_linear_adapters_rows_without_and_with_bad_ids(M, act, dt, impl):
    """-1: the plain linear layer; any other id outside the adapters: a NaN row, ReLU or not."""
    from zeroth_order_fine_b200 import zo
    N, K, n, r = 264, 128, 3, 16
    ids = spans(M, n, M, 1, 9)
    ids[0], ids[M // 2], ids[M - 1] = n, -2, 2 ** 31 - 1
    c = adapt_case(M, N, K, n, r, ids, dt, seed=M)
    y = zo.zo_op_linear_adapters(*(t.cuda() for t in c[:6]), bias=c[6].cuda(), act=act, impl=impl)
    bad = torch.tensor([i < -1 or i >= n for i in ids])
    assert torch.isnan(y[bad.cuda()]).all()
    ref, tol = adapt_ref(*c, n, r, dt == BF, dt == BF and impl != 1)
    ref = torch.relu(ref) if act else ref
    err = (y.double().cpu() - ref).abs()[~bad]
    assert torch.all(err <= tol[~bad])


@pytest.mark.parametrize("M", [40, 300])
def test_linear_adapters_foreign_adapters_cannot_reach_a_row(M):
    """NaN and infinity in adapters that no row names, and in those of other rows' tiles."""
    from zeroth_order_fine_b200 import zo
    N, K, n, r = 264, 128, 6, 16
    ids = [i if i != 4 else -1 for i in spans(M, n, 5, 1, 70)]
    c = adapt_case(M, N, K, n, r, ids, BF, seed=1)
    ref, tol = adapt_ref(*c, n, r, True, True)
    c[2][4 * r:5 * r] = float("nan")                  # adapter 4: named by no row
    c[3][:, 4 * r:5 * r] = float("inf")
    for impl in (0, 1):
        y = zo.zo_op_linear_adapters(*(t.cuda() for t in c[:6]), bias=c[6].cuda(), impl=impl)
        err = (y.double().cpu() - ref).abs()
        assert torch.all(err <= tol)


@pytest.mark.parametrize("M", [6, 200])
def test_linear_adapters_in_a_graph_follow_the_ids(M):
    from zeroth_order_fine_b200 import zo
    N, K, n, r = 512, 256, 8, 16
    c = adapt_case(M, N, K, n, r, spans(M, n, 1), BF, seed=3)
    d = [t.cuda() for t in c[:6]]
    out = torch.empty(M, N, dtype=BF, device="cuda")
    ws = torch.empty(zo.zo_op_linear_adapters_workspace(M, N, K, n, r), dtype=torch.uint8, device="cuda")
    call = lambda: zo.zo_op_linear_adapters(*d, out=out, ws=ws)
    call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for seed in (11, 12):
        ids = i32(spans(M, n, seed, 1, 5), "cpu")
        d[4].copy_(ids)
        gr.replay()
        torch.cuda.synchronize()
        ref, tol = adapt_ref(*c[:4], ids, c[5], None, n, r, True, True)
        assert torch.all((out.double().cpu() - ref).abs() <= tol)
    assert zo.zo_op_error_word() == 0


def test_attention_paged_length_at_the_end_of_int():
    """A length whose last unit of keys would not fit an int: NaN rows, the other request as ever."""
    from zeroth_order_fine_b200 import zo
    for dt, impl in ((BF, 0), (BF, 1), (FP, 1)):
        for new in (1, 40):
            c = Paged([(0, new), (300, new)], 4, 2, 128, 256, dt)
            table = torch.zeros(2, 2 ** 31 // 256, dtype=torch.int32, device="cuda")
            table[:, :c.blocks] = i32(c.table)
            out = zo.zo_op_attention_paged(c.q.cuda(), c.cache.cuda(), table, 256, i32(c.cu),
                                           i32([2 ** 31 - 1, 300 + new]), new, 4, 2, 128, impl=impl)
            assert torch.isnan(out[:new]).all()
            c.check(out, impl, skip=(0,))
    assert zo.zo_op_error_word() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_attention_paged_and_write_far_into_a_cache(new):
    """Pages past 2^32 bytes and 2^32 elements of the cache: the same rows as from a small one."""
    from zeroth_order_fine_b200 import zo
    Hq, Hkv, hd, p = 8, 8, 128, 16
    rows = 2 ** 21 + 64 * p                           # 4 KB each in bf16, 2^32 elements at 2^21 rows
    big = torch.empty(rows, 2 * Hkv * hd, dtype=BF, device="cuda")
    pages = torch.arange(rows // p - 8, rows // p).flip(0)
    g = torch.Generator().manual_seed(new)
    lens, T = [50, 61], 2 * new
    qkv = torch.randn(sum(lens), (Hq + 2 * Hkv) * hd, generator=g).to(BF).cuda()
    q = qkv[:T]
    for impl in (0, 1):
        outs = []
        for cache, first in ((big, pages[:8].tolist()), (torch.empty(8 * p, 2 * Hkv * hd, dtype=BF,
                                                                     device="cuda"), list(range(8)))):
            table = [first[:4], first[4:]]
            slots = sum([[table[r][i // p] * p + i % p for i in range(n)] for r, n in enumerate(lens)], [])
            zo.zo_op_kv_write(qkv, i32(slots), cache, Hq, Hkv, hd)
            outs.append(zo.zo_op_attention_paged(q, cache, i32(table), p, i32([0, new, T]), i32(lens), new,
                                                 Hq, Hkv, hd, impl=impl))
        assert torch.equal(*outs) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("ids", [[0], [-1], [6], [2, 5], [3, 3], [-1, 4], [-2, 1]])
@pytest.mark.parametrize("N,K,r", [(8, 8, 4), (296, 1024, 16), (1000, 264, 8), (304, 5120, 12), (20008, 40, 1),
                                   (512, 8200, 256), (152, 20480, 64)])
def test_linear_adapters_one_and_two_rows(ids, N, K, r):
    """Ranges of W's rows that do not divide, K's tails, ranks, ids that name no adapter; bias, ReLU and
    accumulate; an infinite factor of another adapter."""
    from zeroth_order_fine_b200 import zo
    M, n = len(ids), 6 if r != 1 else 8
    x, W, A, B, idt, sc, b = adapt_case(M, N, K, n, r, ids, BF, seed=K)
    ref, tol = adapt_ref(x, W, A, B, idt, sc, b, n, r, True, True)
    own = [a for a in range(n) if a not in ids]
    A[own[0] * r:(own[0] + 1) * r] = math.inf
    B[:, own[-1] * r:(own[-1] + 1) * r] = math.inf
    x, W, A, B, idt, sc, b = (t.cuda() for t in (x, W, A, B, idt, sc, b))
    ok = [m for m in range(M) if -1 <= ids[m] < n]
    for act in (0, 1):
        y = zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b, act=act).double().cpu()
        want = ref.clamp(min=0) if act else ref
        assert torch.all((y - want).abs()[ok] <= tol[ok])
        assert all(torch.isnan(y[m]).all() for m in range(M) if m not in ok)
    base = torch.randn(M, N, generator=torch.Generator().manual_seed(1))
    out = base.cuda()
    zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b, accumulate=True, out=out)
    got = out.double().cpu() - base.double()
    slack = tol + 2 * U * (base.double().abs() + ref.abs())      # the fp32 sum's rounding
    assert torch.all((got - ref).abs()[ok] <= slack[ok])
    assert torch.equal(zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b)[ok], zo.zo_op_linear_adapters(
        x, W, A, B, idt, sc, b)[ok])
    assert zo.zo_op_error_word() == 0


@pytest.mark.parametrize("M", [1, 2])
def test_linear_adapters_one_and_two_rows_on_the_tensor_cores(M):
    from zeroth_order_fine_b200 import zo
    x, W, A, B, idt, sc, b = adapt_case(M, 520, 1032, 5, 16, [3, -1][:M], BF, seed=M)
    y = zo.zo_op_linear_adapters(x.cuda(), W.cuda(), A.cuda(), B.cuda(), idt.cuda(), sc.cuda(), b.cuda(), impl=2)
    ref, tol = adapt_ref(x, W, A, B, idt, sc, b, 5, 16, True, True)
    assert torch.all((y.double().cpu() - ref).abs() <= tol)
    assert zo.zo_op_error_word() == 0


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 16, 23, 24, 25])
@pytest.mark.parametrize("N,K,r", [(1, 4, 1), (149, 516, 7), (1000, 2048, 16), (296, 8196, 256)])
def test_linear_adapters_few_rows_in_fp32(M, N, K, r):
    """Groups of rows that do not fill, ids that name no adapter, ReLU and accumulate."""
    from zeroth_order_fine_b200 import zo
    n = 5
    ids = spans(M, n - 1, M + K, 1, 3)
    x, W, A, B, idt, sc, b = adapt_case(M, N, K, n, r, ids, FP, seed=K)
    ref, tol = adapt_ref(x, W, A, B, idt, sc, b, n, r, False, False)
    B[:, (n - 1) * r:] = math.inf
    bad = torch.zeros(M, dtype=torch.bool)
    if M > 1:
        idt[M - 1] = n
        bad[M - 1] = True
    x, W, A, B, idt, sc, b = (t.cuda() for t in (x, W, A, B, idt, sc, b))
    for act in (0, 1):
        y = zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b, act=act)
        assert torch.equal(y[~bad], zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b, act=act)[~bad])
        want = ref.clamp(min=0) if act else ref
        assert torch.all((y.double().cpu() - want).abs()[~bad] <= tol[~bad])
        assert torch.isnan(y[bad]).all()
    base = torch.randn(M, N, generator=torch.Generator().manual_seed(1))
    out = base.cuda()
    zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b, accumulate=True, out=out)
    got = out.double().cpu() - base.double()
    slack = tol + 2 * U * (base.double().abs() + ref.abs())      # the fp32 sum's rounding
    assert torch.all((got - ref).abs()[~bad] <= slack[~bad])


@pytest.mark.parametrize("M,N,K,n,r", [(300, 8200, 264, 7, 16), (1500, 1544, 200, 9, 24), (1030, 512, 640, 5, 64),
                                       (260, 1024, 64, 40, 8)])
def test_linear_adapters_of_many_tiles(M, N, K, n, r):
    """Batches above the decode form's: ids that name no adapter, an infinite factor of another adapter,
    ReLU and accumulate."""
    from zeroth_order_fine_b200 import zo
    ids = spans(M, n - 1, M, 1, 90)
    x, W, A, B, idt, sc, b = adapt_case(M, N, K, n, r, ids, BF, seed=M)
    ref, tol = adapt_ref(x, W, A, B, idt, sc, b, n, r, True, True)
    B[:, (n - 1) * r:] = math.inf
    idt[7], idt[M - 1] = n, -5
    bad = torch.zeros(M, dtype=torch.bool)
    bad[7] = bad[M - 1] = True
    x, W, A, B, idt, sc, b = (t.cuda() for t in (x, W, A, B, idt, sc, b))
    for act in (0, 1):
        y = zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b, act=act).double().cpu()
        want = ref.clamp(min=0) if act else ref
        assert torch.all((y - want).abs()[~bad] <= tol[~bad])
        assert torch.isnan(y[bad]).all()
    base = torch.randn(M, N, generator=torch.Generator().manual_seed(1))
    out = base.cuda()
    zo.zo_op_linear_adapters(x, W, A, B, idt, sc, b, accumulate=True, out=out)
    got = out.double().cpu() - base.double()
    slack = tol + 2 * U * (base.double().abs() + ref.abs())      # the fp32 sum's rounding
    assert torch.all((got - ref).abs()[~bad] <= slack[~bad])
    assert zo.zo_op_error_word() == 0


@pytest.mark.parametrize("M", [5, 40, 300, 2500])
def test_linear_adapters_of_65536_factor_columns(M):
    """The most adapters there can be; 2500 rows: two passes of the tiles form."""
    from zeroth_order_fine_b200 import zo
    n, r, N, K = 4096, 16, 64, 64
    ids = [0, n - 1] + spans(M - 2, n, M, 1, 60)
    x, W, A, B, idt, sc, b = adapt_case(M, N, K, n, r, ids, BF, seed=M)
    y = zo.zo_op_linear_adapters(x.cuda(), W.cuda(), A.cuda(), B.cuda(), idt.cuda(), sc.cuda(), b.cuda())
    ref, tol = adapt_ref(x, W, A, B, idt, sc, b, n, r, True, True)
    assert torch.all((y.double().cpu() - ref).abs() <= tol)
    assert zo.zo_op_error_word() == 0


def test_linear_adapters_output_past_32_bits():
    from zeroth_order_fine_b200 import zo
    M, N, K, n, r = 270000, 8192, 64, 8, 16           # 2^31 elements at row 262144
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, K, generator=g).to(BF)
    _, W, A, B, _, sc, b = adapt_case(1, N, K, n, r, [0], BF)
    xs = x.repeat(-(-M // 64), 1)[:M].cuda()
    ids = [(i * 7) % 9 - 1 for i in range(64)]
    idt = i32(ids).repeat(-(-M // 64))[:M]
    y = zo.zo_op_linear_adapters(xs, W.cuda(), A.cuda(), B.cuda(), idt, sc.cuda(), b.cuda())
    ref, tol = adapt_ref(x, W, A, B, i32(ids, "cpu"), sc, b, n, r, True, True)
    for m in (0, 262080, 262144, 262208, 269952 - 64):  # blocks of 64 rows, on both sides of the pass
        assert torch.all((y[m:m + 64].double().cpu() - ref).abs() <= tol), m
    assert zo.zo_op_error_word() == 0


# ---- two at once --------------------------------------------------------------------------------

def shared_calls():
    """Calls of every kernel, each with its own output and workspace; the result of each alone."""
    from zeroth_order_fine_b200 import zo
    calls = []
    for dt, reqs in ((BF, [(700, 1), (33, 1), (2000, 1)]), (BF, [(500, 200), (40, 1), (0, 130)]),
                     (FP, [(300, 1), (20, 70), (900, 3)])):
        c = Paged(reqs, 8, 2, 128, 16, dt, seed=len(calls), tail=0)
        q, args = c.q.cuda(), c.args()
        out = torch.zeros(c.T, 8 * 128, dtype=dt, device="cuda")
        ws = torch.empty(zo.zo_op_attention_paged_workspace(c.T, len(reqs), 8, 2, 128, dt),
                         dtype=torch.uint8, device="cuda")
        calls.append((out, lambda q=q, a=args, m=c.max_new, o=out, w=ws: zo.zo_op_attention_paged(
            q, *a, m, 8, 2, 128, out=o, ws=w)))
    for M, N, K, dt in ((1, 1024, 512, BF), (70, 1024, 512, BF), (700, 1024, 512, BF), (90, 512, 256, FP)):
        x, W, A, B, ids, sc, b = (t.cuda() for t in adapt_case(M, N, K, 6, 16, spans(M, 6, M), dt))
        out = torch.zeros(M, N, dtype=dt, device="cuda")
        ws = torch.empty(zo.zo_op_linear_adapters_workspace(M, N, K, 6, 16, dt), dtype=torch.uint8,
                         device="cuda")
        calls.append((out, lambda x=x, W=W, A=A, B=B, i=ids, s=sc, b=b, o=out, w=ws:
                      zo.zo_op_linear_adapters(x, W, A, B, i, s, b, out=o, ws=w)))
    want = []
    for out, call in calls:
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
    return calls, want


def test_serving_calls_on_two_streams_at_once():
    from zeroth_order_fine_b200 import zo
    (one, want), (two, _) = shared_calls(), shared_calls()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for shift in range(len(one)):
        for out, _ in one + two:
            out.zero_()
        torch.cuda.synchronize()
        for i in range(len(one)):                     # every call beside every other
            with torch.cuda.stream(s[0]):
                one[i][1]()
            with torch.cuda.stream(s[1]):
                two[(i + shift) % len(two)][1]()
        torch.cuda.synchronize()
        for set_ in (one, two):
            for i, (out, _) in enumerate(set_):
                assert torch.equal(out, want[i]), (shift, i)
    assert zo.zo_op_error_word() == 0


def test_serving_calls_in_two_graphs_at_once():
    from zeroth_order_fine_b200 import zo
    sets = [shared_calls(), shared_calls()]
    graphs, s = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for k, (calls, _) in enumerate(sets):
        order = calls if k == 0 else calls[::-1]
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _, call in order:
                call()
        graphs.append(gr)
    for _ in range(5):
        for calls, _ in sets:
            for out, _ in calls:
                out.zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, s):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for calls, want in sets:
            for i, (out, _) in enumerate(calls):
                assert torch.equal(out, want[i]), i
    assert zo.zo_op_error_word() == 0


# ---- together ---------------------------------------------------------------------------------

def test_serving_run_over_pages_equals_the_packed_attention():
    """Requests admitted in chunks, then single tokens, some ending and their pages taken over by
    later ones: tables, projection under adapters, write and attention of every step, against the
    packed attention of each request's whole sequence."""
    from zeroth_order_fine_b200 import zo
    g = torch.Generator().manual_seed(0)
    Hq, Hkv, hd, p, d, n, r = 8, 2, 128, 16, 256, 4, 16
    cols = (Hq + 2 * Hkv) * hd
    W = (torch.randn(cols, d, generator=g) * d ** -0.5).to(BF).cuda()
    A = (torch.randn(n * r, d, generator=g) * d ** -0.5).to(BF).cuda()
    B = (torch.randn(cols, n * r, generator=g) * r ** -0.5).to(BF).cuda()
    sc = torch.rand(n, generator=g).cuda()
    R, blocks, pages, cap = 4, 24, 40, 256
    table = torch.full((R, blocks), -1, dtype=torch.int32, device="cuda")
    ring, state = zo.zo_page_ring(pages)
    state2 = torch.zeros_like(state)
    cache = torch.full((pages * p, 2 * Hkv * hd), float("nan"), dtype=BF, device="cuda")
    # per step: the requests' lengths after it (0 ends the request; a later step starts another)
    plan = [[60, 17, 0, 100], [61, 80, 33, 101], [62, 81, 34, 0], [63, 0, 35, 150], [0, 200, 36, 151],
            [9, 201, 37, 152]]
    xs = [torch.zeros(0, d, dtype=BF) for _ in range(R)]
    outs = [[] for _ in range(R)]
    adapter = [0, 3, -1, 2]

    def finish(q):
        if outs[q]:
            x = xs[q].cuda()
            ids = i32([adapter[q]] * len(x))
            qkv = zo.zo_op_linear_adapters(x, W, A, B, ids, sc)
            whole = zo.zo_op_attention(qkv, [len(x)], Hq, Hkv, hd)
            got = torch.cat(outs[q])
            # a row's projection may differ by one bf16 rounding between batch sizes, which moves a
            # score by 2 * 2^-8 |q||k| / sqrt(d) at most and the weights and values with it
            assert (got.float() - whole.float()).abs().max() <= 0.1, q
            assert ((got.float() - whole.float()).norm() / whole.float().norm()) <= 4 * H
        outs[q] = []
        xs[q] = torch.zeros(0, d, dtype=BF)

    old = [0] * R
    for new in plan:
        new_t = list(new)
        T = sum(max(0, b - a) for a, b in zip(old, new_t))
        cu, slots = zo.zo_op_block_tables(i32(old), i32(new_t), table, ring, state, state2, p,
                                          max_tokens=T + 3)
        state, state2 = state2, state
        assert state[2].item() == 0
        fresh = [torch.randn(max(0, b - a), d, generator=g).to(BF) for a, b in zip(old, new_t)]
        x = torch.cat(fresh + [torch.zeros(3, d, dtype=BF)]).cuda()
        ids = sum([[adapter[q]] * len(f) for q, f in enumerate(fresh)], []) + [-1] * 3
        qkv = zo.zo_op_linear_adapters(x, W, A, B, i32(ids), sc)
        zo.zo_op_kv_write(qkv, slots, cache, Hq, Hkv, hd)
        most = max(len(f) for f in fresh)
        out = zo.zo_op_attention_paged(qkv, cache, table, p, cu, i32(new_t), most, Hq, Hkv, hd)
        at = cu.tolist()
        for q in range(R):
            if new_t[q] < old[q]:
                finish(q)
            elif len(fresh[q]):
                xs[q] = torch.cat([xs[q], fresh[q]])
                outs[q].append(out[at[q]:at[q + 1]])
        old = new_t
    for q in range(R):
        finish(q)
    assert zo.zo_op_error_word() == 0
