"""The serving ops at contents and settings that a server meets rarely: keys and values that are not
finite where a request sees them, and the other ends of what the calls promise.

Bounds as in test_gpu_serving.py (u = 2^-24, h = 2^-8), with one term more: a weight of the chunk
kernel may come from its own polynomial for 2^x, whose relative error is at most 2.7e-6, and a score
of that kernel is scaled and shifted in one rounding.  A weight and the sum of the weights are off by
that much each, an output by 2 * 2.7e-6 * sum w |v|.
"""
import math

import pytest
import torch

from gpu_util import needs_gpu
from test_gpu_serving import BF, FP, H, U, Paged, adapt_case, adapt_ref, i32, spans

pytestmark = [pytest.mark.gpu, needs_gpu]

POLY = 2.7e-6
NAN, INF = float("nan"), float("inf")


def set_key(c, r, i, col, x):
    """Element col of token i's cache row (k, then v) of request r, in the cache and in the model."""
    c.cache[c.table[r][i // c.p] * c.p + i % c.p, col] = x
    c.kv[r][i, col] = x


def compare(c, out, impl, may_be_nan=None):
    """Every row against the definition in float64 (of finite values): NaN where that is NaN, else within
    the bound.  may_be_nan[r]: rows of request r (by their new token) that may be NaN although they need not be."""
    out, g, n_nan = out.double().cpu(), c.Hq // c.Hkv, 0
    for r, (a, b) in enumerate(c.reqs):
        if b == 0:
            continue
        n, hd = a + b, c.hd
        rows = c.kv[r].double().view(n, 2, c.Hkv, hd)
        q = c.q[c.cu[r]:c.cu[r + 1], :c.Hq * hd].double().view(b, c.Hq, hd)
        unseen = torch.ones(b, n, dtype=torch.bool).triu(a + 1)
        for h in range(c.Hq):
            k, v = rows[:, 0, h // g], rows[:, 1, h // g]
            s = (q[:, h] @ k.T / math.sqrt(hd)).masked_fill(unseen, -INF)
            w = torch.softmax(s, -1)
            ref, mag = w @ v, w @ v.abs()
            kf = torch.where(k.isfinite(), k, torch.zeros((), dtype=torch.float64))
            e = 2 * (hd + 3) * U * q[:, h].norm(dim=1) * kf.norm(dim=1).max() / math.sqrt(hd)
            rel = 4 * e[:, None] + 3 * (n + 8) * U + 2 * POLY
            if c.dt == BF:
                rel = rel + (H if impl != 1 else 0.0)
            tol = rel * mag + (H * ref.abs() if c.dt == BF else 0.0)
            got = out[c.cu[r]:c.cu[r + 1], h * hd:(h + 1) * hd]
            nan = ref.isnan()
            n_nan += int(nan.sum())
            assert got[nan].isnan().all(), (r, h, "finite where the definition has NaN")
            fine = ~nan & ((got - ref).abs() <= tol)
            if may_be_nan is not None:
                fine |= got.isnan() & may_be_nan[r][:, None]
            assert (fine | nan).all(), (r, h, (got - ref).abs()[~nan].max())
    return n_nan


# (new tokens of each request, types, impl): the step kernel, the chunk kernel, CUDA cores
KERNELS = [(1, BF, 0), (200, BF, 0), (200, BF, 1), (9, FP, 1)]


@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("lay", [(8, 4, 128), (8, 4, 64)])
@pytest.mark.parametrize("new,dt,impl", KERNELS)
@pytest.mark.parametrize("at", ["early", "new"])
def test_a_key_that_is_not_finite(new, dt, impl, lay, what, at):
    """One such key at each of 16 places in a row: rows that see a NaN score or one of +infinity are
    NaN, a score of -infinity has no weight, and rows that do not see the key are as without it."""
    if at == "new" and new < 100:
        pytest.skip("few new tokens")
    c = Paged([(300, new)] * 16, *lay, 16, dt)
    hd = lay[2]
    c.q[:, ::hd] = c.q[:, ::hd].abs() + 0.5           # what x 0 would be NaN
    for r in range(16):
        set_key(c, r, (32 if at == "early" else 364) + r, hd * (r % 4), what)
    n_nan = compare(c, c.run(impl), impl)
    assert (n_nan > 0) == (what != -INF)


@pytest.mark.parametrize("lay", [(8, 4, 128), (8, 4, 64)])
@pytest.mark.parametrize("new,dt,impl", KERNELS)
@pytest.mark.parametrize("reqs", [1, 16])
def test_all_keys_at_minus_infinity(new, dt, impl, lay, reqs):
    """No score is above -infinity: 0 / 0 in the rows of that kv head, whole items and cut ones."""
    c = Paged([(300, new)] * reqs, *lay, 16, dt)
    hd = lay[2]
    c.q[:, ::hd] = c.q[:, ::hd].abs() + 0.5
    for i in range(300 + new):
        set_key(c, 0, i, hd, -INF)
    assert compare(c, c.run(impl), impl) == new * 2 * hd


@pytest.mark.parametrize("lay", [(8, 4, 128), (8, 4, 64)])
@pytest.mark.parametrize("new,dt,impl", KERNELS)
def test_a_value_that_is_not_finite(new, dt, impl, lay):
    """Rows that see it take it over; rows before it may be NaN (0 times it)."""
    c = Paged([(300, new)] * 4, *lay, 16, dt)
    hd = lay[2]
    for r, x in enumerate((NAN, INF, -INF, NAN)):
        set_key(c, r, 300 + new // 2 if r < 3 else 40, (4 + r) * hd + 3, x)
    seen = torch.arange(new) >= new // 2
    out = c.run(impl).double().cpu()
    for r in range(4):
        col = 2 * r * hd + 3
        got = out[c.cu[r]:c.cu[r + 1], [col, col + hd]]
        rows = seen if r < 3 else torch.ones(new, dtype=torch.bool)
        assert not got[rows].isfinite().any(), r
        # the other columns and heads are not touched
        clean = [x for x in range(c.Hq * hd) if x not in (col, col + hd)]
        assert out[c.cu[r]:c.cu[r + 1], clean].isfinite().all()


@pytest.mark.parametrize("e", [8, 22, 31, 37, 60])
@pytest.mark.parametrize("lay", [(8, 4, 128), (8, 4, 64)])
@pytest.mark.parametrize("new,dt,impl", KERNELS)
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(new, dt, impl, lay, e, sign):
    """Scores around 2^e of either sign, every factor with all its bits: the softmax goes to the largest,
    which is far above the others, and its value row comes out.  One term of q.k is not zero, so a
    product's error is its own rounding's."""
    c = Paged([(300, new)] * 5, *lay, 16, dt)
    Hq, Hkv, hd = lay
    kmax = torch.tensor(2.0 ** (e - e // 2)).to(dt).item()
    c.q[:, :Hq * hd] = 0
    c.q[:, 0:Hq * hd:hd] = sign * 1.2890625 * 2.0 ** (e // 2)
    g = torch.Generator().manual_seed(e)
    for r in range(5):
        k = torch.zeros(300 + new, Hkv, hd)
        k[:, :, 0] = (1 + torch.rand(300 + new, Hkv, generator=g)) * kmax
        k[70 + r, :, 0] = kmax * (2.609375 if sign > 0 else 0.3359375)
        c.kv[r][:, :Hkv * hd] = k.view(300 + new, Hkv * hd).to(dt)
        for i in range(300 + new):
            c.cache[c.table[r][i // 16] * 16 + i % 16] = c.kv[r][i]
    out = c.run(impl).double().cpu()
    for r in range(5):
        v = c.kv[r][70 + r, Hkv * hd:].double().view(Hkv, 1, hd).expand(Hkv, Hq // Hkv, hd).reshape(Hq * hd)
        # 0.609 * 1.289 2^e / sqrt(hd) and more between the largest score and the others (|v| < 6)
        others = (300 + new) * 12 * math.exp(-0.75 * 2.0 ** e / math.sqrt(hd))
        tol = v.abs() * (2 * H if dt == BF else 2.0 ** -20) + others
        assert ((out[c.cu[r]:c.cu[r + 1]] - v).abs() <= tol).all()


@pytest.mark.parametrize("reqs,lay", [([(2500, 1)] * 64, (32, 8, 128)), ([(3000, 512)] * 8, (16, 8, 128)),
                                      ([(3000, 512)] * 8, (16, 8, 64)), ([(2500, 1)] * 40 + [(3000, 512)] * 6, (16, 8, 128))])
def test_expired_wait_is_reported_and_the_next_launch_is_clean(reqs, lay):
    """With the bound of the waits at one cycle an ordinary launch gives up at a wait for its first copies,
    says so in the error word and returns; with the default bound the same call is clean and has the
    same bits as before.  (Single tokens at head_dim 128 only: at 64 the decode-step kernel, the same
    code, is slower than its copies and may never have to wait.)"""
    from zeroth_order_fine_b200 import zo
    Hq, Hkv, hd = lay
    g = torch.Generator(device="cuda").manual_seed(7)
    page, R = 16, len(reqs)
    blocks = max(-(-(a + b) // page) for a, b in reqs)
    cache = torch.randn(R * blocks * page, 2 * Hkv * hd, generator=g, device="cuda").to(BF)
    table = torch.randperm(R * blocks, generator=g, device="cuda").to(torch.int32).view(R, blocks)
    cu = [0]
    for _, b in reqs:
        cu.append(cu[-1] + b)
    q = torch.randn(cu[-1], Hq * hd, generator=g, device="cuda").to(BF)
    args = (q, cache, table, page, i32(cu), i32([a + b for a, b in reqs]), max(b for _, b in reqs), Hq, Hkv, hd)
    want = zo.zo_op_attention_paged(*args)
    assert zo.zo_op_error_word() == 0
    old = zo.zo_op_set_wait_limit(1)
    try:
        zo.zo_op_attention_paged(*args)               # queued: returns
        assert zo.zo_op_error_word() & 1
    finally:
        assert zo.zo_op_set_wait_limit(0) == 1
    assert old > 10 ** 9
    assert zo.zo_op_error_word() == 0
    for _ in range(2):
        assert torch.equal(zo.zo_op_attention_paged(*args), want)
        assert zo.zo_op_error_word() == 0


# ---- adapters -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dt,impl", [(BF, 0), (BF, 1), (FP, 1)])
@pytest.mark.parametrize("M,N,K", [(2, 264, 128), (48, 1000, 328), (300, 264, 200), (700, 1032, 264), (1100, 520, 64)])
@pytest.mark.parametrize("form", ["store", "relu", "accumulate"])
def test_a_row_that_is_not_finite_leaves_the_others_their_bits(M, N, K, form, dt, impl):
    """NaN and infinity in two rows of x, an id that names no adapter, an infinite factor: these rows are as
    the definition has them, every other element has the bits of the call without them."""
    from zeroth_order_fine_b200 import zo
    n, r = 6, 16
    ids = spans(M, n, M, 1, 9)
    x, W, A, B, idt, sc, b = adapt_case(M, N, K, n, r, ids, dt, seed=M)
    y0 = torch.randn(M, N, generator=torch.Generator().manual_seed(1))

    def call(x, B, idt):
        y = y0.cuda().clone() if form == "accumulate" else None
        return zo.zo_op_linear_adapters(x.cuda(), W.cuda(), A.cuda(), B.cuda(), idt.cuda(), sc.cuda(), bias=b.cuda(),
                                        act=int(form == "relu"), accumulate=form == "accumulate", out=y, impl=impl)

    clean = call(x, B, idt)
    _, tol = adapt_ref(x, W, A, B, idt, sc, b, n, r, dt == BF and form != "accumulate", dt == BF and impl != 1)
    tol += 2 * U * (tol + y0.abs().double() + 40) if form == "accumulate" else 0.0    # |y| < 40
    for kind in ("rows", "id", "factor"):
        x2, B2, id2 = x.clone(), B.clone(), idt.clone()
        touched = torch.zeros(M, N, dtype=torch.bool)
        if kind == "rows":
            x2[M // 2, 3], x2[0, 5] = NAN, INF
            touched[[0, M // 2]] = True
        elif kind == "id":
            id2[M // 3] = n
            touched[M // 3] = True
        else:
            B2[N // 2, 2 * r + 3] = -INF
            touched[:, N // 2] = True                 # (another form of the same element's sum)
        y = call(x2, B2, id2).cpu()
        assert torch.equal(y[~touched], clean.cpu()[~touched]), kind
        ref = x2.double() @ W.double().T + b.double()
        for m in range(M):
            a = int(id2[m])
            if 0 <= a < n:
                ref[m] += B2[:, a * r:(a + 1) * r].double() @ (sc[a].double() * (A[a * r:(a + 1) * r].double() @ x2[m].double()))
            elif a != -1:
                ref[m] = NAN
        if form == "relu":
            ref = torch.where(ref < 0, torch.zeros((), dtype=torch.float64), ref)
        elif form == "accumulate":
            ref += y0.double()
        odd = ~ref.isfinite()
        assert torch.equal(y.isnan(), ref.isnan()), kind
        assert torch.equal(y[odd & ~ref.isnan()].double(), ref[odd & ~ref.isnan()]), kind
        assert ((y.double() - ref).abs() <= tol)[~odd].all(), kind
    assert zo.zo_op_error_word() == 0


@pytest.mark.parametrize("M,N,K,r", [(5000, 16384, 8, 4), (4161, 16448, 12, 40)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_fp32_adapters_in_several_passes(M, N, K, r, accumulate):
    """Outputs past 256 MB: rows in passes, each with its own slices; every row against float64."""
    from zeroth_order_fine_b200 import zo
    n = 3
    c = adapt_case(M, N, K, n, r, spans(M, n, 3, 1, 700), FP, seed=K)
    d = [t.cuda() for t in c]
    y0 = torch.randn(M, N, device="cuda") if accumulate else None
    y = zo.zo_op_linear_adapters(*d[:6], bias=d[6], accumulate=accumulate, out=y0.clone() if accumulate else None)
    for m0 in range(0, M, 1000):
        rows = slice(m0, m0 + 1000)
        ref, tol = adapt_ref(d[0][rows], *d[1:4], d[4][rows], d[5], d[6], n, r, False, False)
        if accumulate:
            ref += y0[rows]
            tol += 2 * U * (ref.abs() + y0[rows].double().abs())
        assert ((y[rows].double() - ref).abs() <= tol).all(), m0


@pytest.mark.parametrize("dt,impl,hint", [(BF, 0, 1000), (BF, 0, 1), (BF, 1, 1000), (FP, 1, 1000)])
@pytest.mark.parametrize("lay", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("page", [2 ** 31 - 1, -1])
def test_a_bad_page_behind_the_first_tiles(dt, impl, hint, lay, page):
    """Rows that see a page outside the pool are NaN; rows of the same request before it are right or NaN,
    other requests' rows right."""
    c = Paged([(3, 1), (0, 700), (20, 30)], *lay, 16, dt)
    c.table[1][40] = page
    out = c.run(impl, max_new=hint)
    kv2 = lay[1] * lay[2]
    c.kv[1][640:656, :kv2] = NAN                      # (the oracle's rows that see it: NaN)
    no = torch.zeros(700, dtype=torch.bool)
    n_nan = compare(c, out, impl, may_be_nan=[no[:1], ~no, no[:30]])
    assert n_nan == 60 * lay[0] * lay[2]
    assert out[1:1 + 128].isfinite().all()            # a tile that is done by then is not held back


COLD = """
import sys, torch
sys.path.insert(0, {root!r})
from zeroth_order_fine_b200 import zo
BF, FP, dev = torch.bfloat16, torch.float32, "cuda"
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
g = torch.Generator(device=dev).manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
calls, outs = [], []
for hd, dt, new in ((128, BF, 1), (128, BF, 100), (64, BF, 1), (64, BF, 100), (64, FP, 3)):
    q, cache, table = rnd(2 * new, 4 * hd).to(dt), rnd(64 * 16, 4 * hd).to(dt), i32([list(range(32)), list(range(32, 64))])
    out, ws = torch.zeros(2 * new, 4 * hd, dtype=dt, device=dev), torch.empty(
        zo.zo_op_attention_paged_workspace(2 * new, 2, 4, 2, hd, dt), dtype=torch.uint8, device=dev)
    a = (q, cache, table, 16, i32([0, new, 2 * new]), i32([300, 400]), new, 4, 2, hd)
    calls.append(lambda a=a, out=out, ws=ws: zo.zo_op_attention_paged(*a, out=out, ws=ws)); outs.append(out)
for M, dt in ((1, BF), (2, BF), (40, BF), (400, BF), (3, FP), (300, FP)):
    N, K, n, r = 1024, 512, 4, 16
    a = (rnd(M, K).to(dt), rnd(N, K).to(dt), rnd(n * r, K).to(dt), rnd(N, n * r).to(dt), i32([m % 5 - 1 for m in range(M)]),
         rnd(n))
    out, ws = torch.zeros(M, N, dtype=dt, device=dev), torch.empty(
        zo.zo_op_linear_adapters_workspace(M, N, K, n, r, dt), dtype=torch.uint8, device=dev)
    calls.append(lambda a=a, out=out, ws=ws: zo.zo_op_linear_adapters(*a, out=out, ws=ws)); outs.append(out)
ring, s = zo.zo_page_ring(64)
t, s2, cu, sl = i32([[0] * 8] * 2), i32([0] * 4), i32([0] * 3), i32([0] * 50)
o, nw, qkv, pool = i32([0, 0]), i32([17, 30]), rnd(50, 4 * 64), rnd(64 * 16, 2 * 64)
calls.append(lambda: zo.zo_op_block_tables(o, nw, t, ring, s, s2, 16, cu_new=cu, slot_map=sl))
calls.append(lambda: zo.zo_op_kv_write(qkv, sl, pool, 2, 1, 64))
outs += [t, s2, cu, sl, pool]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for f in calls:
        f()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in outs]
for f in calls:
    f()
assert zo.zo_op_error_word() == 0
assert all(torch.equal(a, b) for a, b in zip(got, outs)) and all(x.float().isfinite().all() and x.any() for x in outs)
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """Every op captured before it ever ran: the replay gives the bits of the calls."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", COLD.format(root=root)], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "same" in p.stdout, p.stderr[-3000:]


@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("delta", [1e-5, 1e-4])
def test_the_exponentials_of_a_row_agree_however_they_are_computed(new, hd, delta):
    """The rounding of p to bf16 hides an exponential's error, unless p lies next to a rounding border.  Here
    it does: 16 keys in a row share a score whose weight is delta (relative) beside the middle of two
    bf16 numbers, now on one side, now on the other, and their values are 3 at four of the 16 places
    and -1 at twelve, four places taken in turn.  The sum is 0 exactly if all 16 weights round alike, so every
    exponential is right to delta: 2.7e-6 of the chunk kernel's polynomial, 2^-22 of the other, 3 2^-24 * 3 of
    the scores are below it.  (Weights are 2^-3 to 1, multiples of 2^-11, and sums stay below 2^10: no sum
    is rounded.)"""
    heads, ctx = 8, 512
    c2 = float(torch.tensor(1 / math.sqrt(hd), dtype=FP) * torch.tensor(1.4426950408889634, dtype=FP))
    c = Paged([(ctx, new)], heads, heads, hd, 16, BF)
    g = torch.Generator().manual_seed(hd)
    kv = c.kv[0].view(ctx + new, 2, heads, hd)
    kv.zero_()
    kv[ctx:, 0, :, 0] = -400.0                        # the new tokens: next to no weight, value 0
    for h in range(heads):
        for group in range(ctx // 16):
            s = 0.0                                   # in every 128 keys one group at the maximum
            if group % 8 != h % 8:
                mid = (1 + (2 * int(torch.randint(128, (), generator=g)) + 1) / 256) * 2.0 ** -int(
                    torch.randint(1, 4, (), generator=g))
                s = math.log2(mid * (1 + delta * (1 if group % 2 else -1))) / c2
            for d in range(3):                        # the score as a sum of three bf16 numbers
                part = torch.tensor(s).to(BF)
                kv[group * 16:group * 16 + 16, 0, h, d] = part
                s -= part.item()
        at = torch.arange(ctx)
        for d in range(4):
            kv[:ctx, 1, h, d] = torch.where(at % 16 // 4 == d, 3.0, -1.0).to(BF)
    for i in range(ctx + new):
        c.cache[c.table[0][i // 16] * 16 + i % 16] = c.kv[0][i]
    c.q.zero_()
    c.q.view(c.T, 3 * heads, hd)[:, :heads, :3] = 1.0
    out = c.run()[:new].view(new, heads, hd).float()
    assert (out[:, :, :4] == 0).all(), out[:, :, :4].abs().max()
