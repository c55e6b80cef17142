"""GPU tests of the attention over a paged cache against the softmax over
each row's permitted set in fp64.

Tolerances, from the arithmetic (h = half a step of the 16-bit type,
finfo.eps / 2; u = 2^-24; A = sum_j p_j |v_j| / l, the magnitude behind o):
  s     products of 16-bit values are exact in fp32, their sum over d is off
        by at most d u sum |q k| (<= 2^-17 sum |q k| for d = 128), times scale
  p     2^x of x = s log2(e) - m: the argument's rounding, 2 u |x| with
        |x| < 64 below which p no longer counts: 8e-6; exp2 2^-22
  P     rounded to 16 bits for the product with V: h of itself; fp16 below
        2^-14 in steps of 2^-24: 2^-25 each (the largest p is at least 1)
  o     rounded once: h |o|; sums in fp32, joined across splits: 1e-5 A
so |o - ref| <= h |o| + (h + 2e-5 + e_s) A + 2^-25 (n max|v| + 1) for fp16,
with e_s = 2^-17 scale max_j sum |q k_j|, and |lse - ref| <= e_s + 2e-5.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def spa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from head_partitioned_distance_b200 import spa as mod
    return mod


def bands_of(kind, Hq, N):
    if kind == "balanced":
        return [h * N // Hq for h in range(Hq)], [(h + 1) * N // Hq for h in range(Hq)]
    if kind == "full":
        return [0] * Hq, [N] * Hq
    if kind.startswith("window"):
        return [0] * Hq, [min(N, int(kind[6:]))] * Hq
    if kind.startswith("far"):  # nothing nearer than this
        return [int(kind[3:])] * Hq, [N] * Hq
    return [h % 3 for h in range(Hq)], [h % 3 + 1 for h in range(Hq)]  # one key each


class Case:
    """Sequences (new tokens, length) in random pages; every place that no row
    attends to holds NaN, every unused page table entry a wrong number."""

    def __init__(self, seqs, page, Hq, Hk, d, dtype, kind, seed=0, pad=2, N=None, k_gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.page, self.dtype, self.Hq, self.Hk, self.d = seqs, page, dtype, Hq, Hk, d
        used = [-(-max(c, 0) // page) for _, c in seqs]
        self.N = N or max(max(used) * page, Hq)
        self.lo, self.hi = bands_of(kind, Hq, self.N)
        pages, width = sum(used) + 2, max(max(used), 1) + 1
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        table, at = torch.full((len(seqs), width), -9, dtype=torch.int32), 0
        self.T = sum(n for n, _ in seqs) + pad
        self.q = torch.randn(self.T, Hq, d, generator=g).to(dtype)
        self.k = [torch.randn(Hk, max(c, 0), d, generator=g).mul_(k_gain).to(dtype) for _, c in seqs]
        self.v = [torch.randn(Hk, max(c, 0), d, generator=g).to(dtype) for _, c in seqs]
        kp = torch.full((pages, Hk, page, d), float("nan"), dtype=dtype)
        vp = kp.clone()
        G = Hq // Hk
        for s, (n, c) in enumerate(seqs):
            j = torch.arange(max(c, 0))
            pos = torch.arange(c - n, c)
            seen_any = torch.zeros(Hk, max(c, 0), dtype=torch.bool)
            for h in range(Hq):
                gap = pos[:, None] - j
                seen_any[h // G] |= ((gap >= self.lo[h]) & (gap < self.hi[h])).any(0)
            for i in range(used[s]):
                span = slice(i * page, min((i + 1) * page, c))
                m = span.stop - span.start
                if not seen_any[:, span].any():
                    continue  # the page is not needed: its number stays wrong
                table[s, i] = perm[at + i]
                keep = seen_any[:, span, None]
                kp[perm[at + i], :, :m] = torch.where(keep, self.k[s][:, span], float("nan"))
                vp[perm[at + i], :, :m] = torch.where(keep, self.v[s][:, span], float("nan"))
            at += used[s]
        self.kp, self.vp, self.table = kp.to(DEV), vp.to(DEV), table.to(DEV)
        self.cu = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32).to(DEV)
        self.kv = torch.tensor([c for _, c in seqs], dtype=torch.int32, device=DEV)
        self.max_q = max(max(n for n, _ in seqs), 1)
        self.qd = self.q.to(DEV)

    def run(self, spa, **kw):
        out = torch.full((self.T, self.Hq, self.d), 3.0, dtype=self.dtype, device=DEV)
        lse = torch.full((self.T, self.Hq), 5.0, device=DEV)
        args = dict(lo=self.lo, hi=self.hi, N=self.N, out=out, lse=lse)
        args.update(kw)
        return spa.paged_attention(self.qd, self.kp, self.vp, self.table, self.cu, self.kv,
                                   args.pop("max_q", self.max_q), **args)

    def check(self, o, lse, rows=None):
        """Every row (or the given token rows) of o and lse."""
        scale, G, h16 = self.d ** -0.5, self.Hq // self.Hk, HALF[self.dtype]
        o, lse = o.double().cpu(), lse.double().cpu()
        t0 = 0
        for s, (n, c) in enumerate(self.seqs):
            pick = [t for t in range(n) if rows is None or t0 + t in rows]
            if pick:
                pos = torch.tensor([c - n + t for t in pick])
                q = self.q[[t0 + t for t in pick]].double()
                j = torch.arange(max(c, 0))
                for h in range(self.Hq):
                    k, v = self.k[s][h // G].double(), self.v[s][h // G].double()
                    gap = pos[:, None] - j
                    ok = (gap >= self.lo[h]) & (gap < self.hi[h])
                    x = torch.where(ok, q[:, h] @ k.T * scale, -math.inf)
                    e_s = torch.where(ok, q[:, h].abs() @ k.abs().T, 0.0).amax(-1) * scale * 2.0 ** -17 \
                        if c > 0 else torch.zeros(len(pick))
                    z = torch.logsumexp(x, -1) if c > 0 else torch.full((len(pick),), -math.inf)
                    p = torch.exp(x - torch.where(z.isinf(), 0.0, z)[:, None])
                    want, mag = p @ v, p @ v.abs()
                    tol = h16 * want.abs() + (h16 + 2e-5 + e_s[:, None]) * mag
                    if self.dtype == FP and c > 0:
                        tol = tol + 2.0 ** -25 * (ok.sum(-1)[:, None] * v.abs().max() + 1)
                    at = [t0 + t for t in pick]
                    err = (o[at, h] - want).abs()
                    assert (err <= tol + 1e-30).all(), (s, h, float((err / (tol + 1e-30)).max()))
                    got = lse[at, h]
                    assert torch.equal(got.isneginf(), z.isneginf()), (s, h)
                    fin = ~z.isinf()
                    assert ((got - z).abs()[fin] <= (e_s + 2e-5)[fin]).all(), (s, h)
            t0 += n
        if rows is None:
            assert (o[t0:] == 3.0).all() and (lse[t0:] == 5.0).all()  # rows behind the last sequence


SMALL = [
    # seqs (new, length), page, Hq, Hk, d, dtype, bands
    ([(1, 1)], 16, 1, 1, 64, BF, "full"),
    ([(1, 1001)], 16, 8, 8, 64, BF, "balanced"),
    ([(1, 130), (1, 64), (1, 65), (1, 7)], 16, 4, 4, 128, BF, "balanced"),
    ([(1, 400), (1, 33), (0, 90), (1, 1)], 32, 8, 2, 128, FP, "full"),
    ([(1, 777), (1, 300)], 64, 6, 2, 64, BF, "window100"),
    ([(1, 777), (1, 20)], 128, 12, 2, 128, BF, "far30"),
    ([(1, 500)], 256, 32, 1, 128, FP, "full"),
    ([(1, 300), (1, 299)], 16, 6, 6, 64, FP, "one"),
    ([(2, 200), (5, 5), (3, 90)], 16, 4, 2, 64, BF, "full"),
    ([(7, 300), (1, 12), (16, 16)], 32, 4, 4, 128, BF, "balanced"),
    ([(4, 260), (2, 100)], 64, 8, 2, 128, FP, "window33"),
    ([(5, 2), (3, 0), (2, 40)], 16, 2, 1, 64, BF, "full"),  # more new tokens than the sequence has
    ([(1, 100 + 7 * i) for i in range(40)], 16, 4, 1, 64, BF, "full"),
]


@pytest.mark.parametrize("seqs,page,Hq,Hk,d,dtype,kind", SMALL)
def test_few_rows(spa, seqs, page, Hq, Hk, d, dtype, kind):
    c = Case(seqs, page, Hq, Hk, d, dtype, kind, seed=len(seqs) + page)
    c.check(*c.run(spa))
    assert spa.spa_device_status() == spa.SPA_OK


MANY = [
    ([(17, 17)], 16, 1, 1, 64, BF, "full"),
    ([(128, 128)], 128, 2, 2, 128, BF, "full"),
    ([(129, 400)], 64, 4, 1, 128, BF, "full"),
    ([(300, 300), (1, 77), (0, 5), (40, 513)], 16, 4, 2, 64, FP, "window100"),
    ([(257, 600), (255, 255)], 32, 8, 8, 64, BF, "balanced"),
    ([(100, 90), (30, 0), (64, 64)], 16, 3, 1, 128, BF, "full"),
    ([(200, 500), (31, 700)], 256, 6, 2, 128, FP, "balanced"),
    ([(90, 700)], 128, 5, 5, 64, BF, "far200"),
    ([(70, 300), (50, 333)], 16, 6, 1, 64, BF, "one"),
    ([(33, 1000), (20, 20), (1, 999)], 64, 16, 2, 128, BF, "window257"),
    ([(513, 513)], 32, 2, 1, 64, BF, "full"),
]


@pytest.mark.parametrize("seqs,page,Hq,Hk,d,dtype,kind", MANY)
def test_many_rows(spa, seqs, page, Hq, Hk, d, dtype, kind):
    c = Case(seqs, page, Hq, Hk, d, dtype, kind, seed=len(seqs) + page)
    c.check(*c.run(spa))
    assert spa.spa_device_status() == spa.SPA_OK


# more items than CTAs: the plan cuts the line of all items (with and without
# dividing one), over empty sequences, sequences without keys and single rows
def _crowd(n, most, seed, rows):
    g = torch.Generator().manual_seed(seed)
    seqs = []
    for i in range(n):
        new = 0 if i % 11 == 5 else int(torch.randint(1, rows + 1, (1,), generator=g))
        seqs.append((new, new + int(torch.randint(0, most, (1,), generator=g)) if i % 7 else new // 2))
    return seqs


@pytest.mark.parametrize("seqs,page,Hq,Hk,d,dtype,kind", [
    (_crowd(170, 200, 1, 1), 16, 4, 4, 64, BF, "balanced"),
    (_crowd(90, 900, 2, 4), 32, 8, 2, 128, FP, "full"),
    ([(1, 4000)] + _crowd(80, 60, 3, 1), 64, 4, 4, 64, BF, "full"),
    (_crowd(60, 150, 4, 150), 16, 4, 2, 64, FP, "window70"),
    (_crowd(40, 500, 5, 60), 64, 4, 4, 128, BF, "balanced"),
    ([(300, 3000)] + _crowd(50, 40, 6, 30), 32, 4, 1, 128, BF, "full"),
])
def test_more_items_than_ctas(spa, seqs, page, Hq, Hk, d, dtype, kind):
    c = Case(seqs, page, Hq, Hk, d, dtype, kind, seed=len(seqs))
    o, lse = c.run(spa)
    c.check(o, lse)
    again = c.run(spa)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert spa.spa_device_status() == spa.SPA_OK


# long sequences: items cut over many CTAs, their pieces joined by the last to arrive
@pytest.mark.parametrize("seqs,Hq,Hk,d,dtype,kind", [
    ([(1, 30001)], 4, 1, 128, BF, "full"), ([(1, 9000), (1, 50), (1, 4000)], 8, 8, 64, BF, "full"),
    ([(3, 20000)], 2, 1, 64, FP, "far100"), ([(20, 12000), (1, 100)], 4, 1, 128, BF, "full"),
    ([(200, 9000)], 2, 2, 64, FP, "window5000"), ([(1, 150001)], 1, 1, 64, BF, "full"),
    ([(2, 40000), (1, 39000)], 3, 3, 64, FP, "balanced"), ([(300, 20000), (130, 17000)], 2, 1, 128, BF, "far15000"),
])
def test_split_rows(spa, seqs, Hq, Hk, d, dtype, kind):
    c = Case(seqs, 64, Hq, Hk, d, dtype, kind, seed=3)
    o, lse = c.run(spa)
    c.check(o, lse)
    again = c.run(spa)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # the same from call to call
    assert spa.spa_device_status() == spa.SPA_OK


@pytest.mark.parametrize("max_q,new", [(1, 1), (40, 40)])
def test_large_scores_and_no_numbers(spa, max_q, new):
    # scores of a few hundred (one key takes the whole softmax, the running
    # maximum moves often), then a query that is no number: its own rows only
    c = Case([(new, 900), (new, 300)], 16, 4, 2, 64, BF, "full", seed=8, k_gain=30.0)
    c.check(*c.run(spa))
    c.qd[0, 1] = float("nan")
    o, lse = c.run(spa)
    assert o[0, 1].isnan().all() and lse[0, 1].isnan()
    mask = torch.ones(c.T, 4, dtype=torch.bool, device=DEV)
    mask[0, 1] = False
    assert not o[mask].isnan().any() and not lse[mask].isnan().any()


@pytest.mark.parametrize("new", [1, 50])
def test_wrong_pages_and_lengths(spa, new):
    c = Case([(new, 200), (new, 100), (new, 70)], 16, 2, 1, 64, BF, "full", seed=4)
    good, good_lse = (t.clone() for t in c.run(spa))
    c.table[0, 3] = c.kp.shape[0]
    c.table[1, 0] = -1
    o, lse = c.run(spa)
    assert spa.spa_device_status() == spa.SPA_ERR_INVAL
    assert spa.spa_device_status() == spa.SPA_OK
    # the third sequence is untouched by the others' errors; theirs are finite
    assert torch.equal(o[2 * new:], good[2 * new:]) and torch.equal(lse[2 * new:], good_lse[2 * new:])
    assert not o.isnan().any()
    c.kv[1] = 16 * c.table.shape[1] + 5  # longer than its row of the page table
    c.run(spa)
    assert spa.spa_device_status() == spa.SPA_ERR_INVAL
    # more new tokens than max_q: the rows past it stay
    c = Case([(new + 3, 200), (1, 60)], 16, 2, 1, 64, BF, "full", seed=5)
    o, lse = c.run(spa, max_q=new)
    c.check(o, lse, rows=set(range(new)) | {new + 3})
    assert (o[new:new + 3] == 3.0).all() and (lse[new:new + 3] == 5.0).all()
    assert spa.spa_device_status() == spa.SPA_OK


def test_equals_the_training_forward(spa):
    # prompts in chunks, then single tokens, through norm, rotation and cache:
    # the rows of spattention on the whole sequence
    H, N, d, page = 4, 333, 64, 16
    g = torch.Generator().manual_seed(21)
    qkv = torch.randn(N, 3 * H, d, generator=g).to(BF).to(DEV)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2))
    rope = spa.rope_table(N, d)
    view = [t.transpose(0, 1)[None] for t in qkv.split(H, 1)]
    qn, kn = spa.qk_norm_rope(view[0], view[1], wq, wk, rope)
    want, want_lse = spa.attention_forward(qn, kn, view[2].contiguous())
    pages = -(-N // page)
    kp = torch.full((pages, H, page, d), float("nan"), dtype=BF, device=DEV)
    vp = kp.clone()
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].to(DEV)
    at, outs, lses = 0, [], []
    for n in (100, 1, 60, 17, 16, 5) + (1,) * 4 + (N - 203,):
        q, k, v = qkv[at:at + n].split(H, 1)
        at += n
        cu, kv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, n], [at]))
        qr = spa.paged_append(q, k, v, kp, vp, table, cu, kv, wq, wk, rope)
        o, lse = spa.paged_attention(qr, kp, vp, table, cu, kv, n, N=N)
        outs.append(o)
        lses.append(lse)
    assert at == N and spa.spa_device_status() == spa.SPA_OK
    got, got_lse = torch.cat(outs).transpose(0, 1)[None], torch.cat(lses).T[None]
    assert torch.equal(got_lse.isneginf(), want_lse.isneginf())
    fin = ~want_lse.isinf()
    # the same inputs bit for bit; both are off by the tolerance above from the
    # exact rows: |o| <= A <= max|v|
    vmax = float(view[2].abs().max())
    assert float((got.float() - want.float()).abs().max()) <= 2 * (2 * HALF[BF] + 3e-5) * vmax
    assert float((got_lse - want_lse).abs()[fin].max()) <= 1e-4


@pytest.mark.parametrize("new", [1, 64])
def test_graph_follows_the_lengths(spa, new):
    # one captured call per step: lengths, pages and queries change on the device
    c = Case([(new, 900), (new, 700)], 16, 4, 2, 64, BF, "full", seed=9)
    out = torch.full((c.T, 4, 64), 3.0, dtype=BF, device=DEV)
    lse = torch.full((c.T, 4), 5.0, device=DEV)
    kw = dict(lo=c.lo, hi=c.hi, N=c.N, out=out, lse=lse)
    call = lambda: spa.paged_attention(c.qd, c.kp, c.vp, c.table, c.cu, c.kv, new, **kw)  # noqa: E731
    call()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    with torch.cuda.graph(other):
        call()
    c.seqs = [(new, 320), (new, 699)]
    c.kv.copy_(torch.tensor([320, 699], dtype=torch.int32))
    c.k, c.v = ([t[:, :n] for t, (_, n) in zip(x, c.seqs)] for x in (c.k, c.v))
    out.fill_(3.0)
    lse.fill_(5.0)
    other.replay()
    graph.replay()
    c.check(out, lse)


def test_two_streams_at_once(spa):
    cases = [Case([(1, 3000), (1, 2000)], 16, 8, 2, 64, BF, "full", seed=i) for i in range(2)]
    want = [tuple(t.clone() for t in c.run(spa)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append([c.run(spa) for _ in range(5)])
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o, lse in outs:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("new", [1, 30])
def test_offsets_past_32_bits(spa, new):
    # the last pages of a cache of 2^31 + elements, written and read
    pages, page, Hk, d, n = 33000, 128, 4, 128, 200
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    kp = torch.empty(pages, Hk, page, d, dtype=BF, device=DEV)
    vp = torch.empty(pages, Hk, page, d, dtype=BF, device=DEV)
    assert kp.numel() > 2 ** 31
    small = [torch.empty(2, Hk, page, d, dtype=BF, device=DEV) for _ in range(2)]
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(n, 3 * Hk, d, generator=g).to(BF).to(DEV)
    w, rope = torch.ones(d, device=DEV), spa.rope_table(n, d)
    outs = []
    for k_pages, v_pages, table in ((kp, vp, [pages - 1, pages - 2]), (*small, [0, 1])):
        table, kv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([table], [n]))
        cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        q = spa.paged_append(*qkv.split(Hk, 1), k_pages, v_pages, table, cu, kv, w, w, rope)
        cu = torch.tensor([0, new], dtype=torch.int32, device=DEV)
        outs.append(spa.paged_attention(q[-new:].contiguous(), k_pages, v_pages, table, cu, kv, new, lo=[0] * Hk,
                                        hi=[n] * Hk, N=n))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert spa.spa_device_status() == spa.SPA_OK and not outs[0][0].isnan().any()


def test_sequences_may_share_pages(spa):
    # a common prefix, read by two sequences through the same pages
    c = Case([(1, 64), (1, 64)], 16, 4, 2, 64, BF, "full", seed=2)
    c.table[1, :4] = c.table[0, :4]
    c.k[1], c.v[1] = c.k[0], c.v[0]
    c.check(*c.run(spa))


def test_no_rows(spa):
    c = Case([(0, 50), (0, 0)], 16, 2, 1, 64, BF, "full", pad=3)
    o, lse = c.run(spa)
    assert (o == 3.0).all() and (lse == 5.0).all()
    c.qd = c.qd[:0]
    c.T = 0
    o, lse = c.run(spa)
    assert o.shape == (0, 2, 64)


@pytest.mark.parametrize("new", [1, 40])
def test_a_pending_timeout_stays_reported(spa, new):
    # a later call with a wrong page must not hide that an earlier kernel gave
    # up on a wait: the status word keeps the gravest report
    c = Case([(new, 200)], 16, 2, 1, 64, BF, "full", seed=4)
    c.table[0, 3] = -1
    assert spa.spa_device_status() == spa.SPA_OK
    spa.spa_debug_wait_timeout(1_000_000)  # 1 ms
    c.run(spa)
    assert spa.spa_device_status() == spa.SPA_ERR_TIMEOUT
    assert spa.spa_device_status() == spa.SPA_OK
    c.kv[0] = 16 * c.table.shape[1] + 5
    spa.spa_debug_wait_timeout(1_000_000)
    c.run(spa)
    assert spa.spa_device_status() == spa.SPA_ERR_TIMEOUT
    rope, w = spa.rope_table(8, 64), torch.ones(64, device=DEV)  # too short for the positions
    k = torch.zeros(c.T, 1, 64, dtype=BF, device=DEV)
    spa.spa_debug_wait_timeout(1_000_000)
    spa.paged_append(c.qd, k, k, c.kp, c.vp, c.table, c.cu, c.kv, w, w, rope)
    assert spa.spa_device_status() == spa.SPA_ERR_TIMEOUT
    assert spa.spa_device_status() == spa.SPA_OK


@pytest.mark.parametrize("new,T", [(1, 1), (9, 15), (9, 9), (40, 61), (40, 40)])
def test_sequences_past_the_last_row_are_reported(spa, new, T):
    # cu_q on the device names more token rows than the call has: the rows that
    # exist are right, and the status says that some are missing
    c = Case([(new, 200), (new, 100)], 16, 2, 1, 64, BF, "full", seed=6, pad=0)
    c.qd, c.T = c.qd[:T].contiguous(), T
    assert spa.spa_device_status() == spa.SPA_OK
    o, lse = c.run(spa)
    assert spa.spa_device_status() == spa.SPA_ERR_INVAL
    c.check(o, lse, rows=set(range(T)))
    w, rope = torch.ones(64, device=DEV), spa.rope_table(200, 64)
    k = torch.randn(T, 1, 64, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    table = torch.arange(26, dtype=torch.int32, device=DEV).view(2, 13)
    kp, vp = torch.full((26, 1, 16, 64), 7.0, dtype=BF, device=DEV), torch.full((26, 1, 16, 64), 7.0, dtype=BF, device=DEV)
    q = spa.paged_append(c.qd, k, k, kp, vp, table, c.cu, c.kv, w, w, rope)
    assert spa.spa_device_status() == spa.SPA_ERR_INVAL
    assert (q != 0).flatten(1).any(1).all()
    flat = vp.view(2, -1, 64)  # [sequence][position]
    first = min(new, T)
    assert torch.equal(flat[0, 200 - new:200 - new + first], k[:first, 0])
    assert torch.equal(flat[1, 100 - new:100 - new + T - first], k[first:, 0])
    assert int((flat != 7.0).any(-1).sum()) == T
    # rows of no sequence in front: left as they are, and no error
    c = Case([(new, 200), (new, 100)], 16, 2, 1, 64, BF, "full", seed=7, pad=0)
    c.cu, c.T = c.cu + 2, c.T + 2
    c.qd = torch.cat((torch.full_like(c.qd[:2], float("nan")), c.qd))
    o, lse = c.run(spa)
    assert spa.spa_device_status() == spa.SPA_OK
    assert (o[:2] == 3.0).all() and (lse[:2] == 5.0).all()
    c.check(o[2:], lse[2:], rows=set(range(2 * new)))


@pytest.mark.parametrize("seqs,page,Hq,Hk,d,dtype,kind", [
    ([(1, 9), (1, 33), (1, 80)], 16, 8, 2, 64, BF, "full"),
    ([(1, 700), (1, 40)], 32, 8, 8, 128, BF, "window24"),
    ([(4, 30), (3, 300)], 64, 8, 2, 128, BF, "window50"),
    ([(1, 9), (1, 33), (1, 80)], 16, 8, 2, 128, FP, "full"),
    ([(1, 9000), (1, 20)], 64, 4, 1, 64, BF, "full"),
])
def test_few_rows_keep_p_in_two_terms(spa, seqs, page, Hq, Hk, d, dtype, kind):
    """The kernel for few rows multiplies V by P in two 16-bit terms.  The
    second is the first's error, at most h p, and is off by h of itself, so P
    is off by h^2 p (fp16: or half the smallest subnormal, 2^-25), not by h p:
      |o - ref| <= h |o| + (h^2 + 2e-5 + e_s) A + 2^-25 (n max|v| + 1) for fp16.
    Every second value is close to the opposite of the one before, so that |o|
    is far below A; P rounded once, formed here in fp64, has to miss the bound."""
    c = Case(seqs, page, Hq, Hk, d, dtype, kind, seed=41)
    h16, scale, G = HALF[dtype], d ** -0.5, Hq // Hk
    for s, (n, length) in enumerate(seqs):
        even = length // 2 * 2
        c.v[s][:, 1:even:2] = -c.v[s][:, 0:even:2] * (1 + 2.0 ** -5)
        for i in range(-(-length // page)):  # what is attended to; NaN stays where it is
            if c.table[s, i] < 0:
                continue
            m = min(page, length - i * page)
            place = c.vp[int(c.table[s, i]), :, :m]
            place.copy_(torch.where(place.isnan(), place, c.v[s][:, i * page:i * page + m].to(DEV)))
    o, lse = (t.double().cpu() for t in c.run(spa))
    t0, missed = 0, False
    for s, (n, length) in enumerate(seqs):
        gap = torch.arange(length - n, length)[:, None] - torch.arange(length)
        for h in range(Hq):
            k, v = c.k[s][h // G].double(), c.v[s][h // G].double()
            q = c.q[t0:t0 + n, h].double()
            ok = (gap >= c.lo[h]) & (gap < c.hi[h])
            x = torch.where(ok, q @ k.T * scale, -math.inf)
            e_s = torch.where(ok, q.abs() @ k.abs().T, 0.0).amax(-1) * scale * 2.0 ** -17
            p = torch.exp(x - x.amax(-1, keepdim=True))
            total = p.sum(-1, keepdim=True)
            want, mag = p @ v / total, p @ v.abs() / total
            tol = h16 * want.abs() + (h16 * h16 + 2e-5 + e_s[:, None]) * mag
            if dtype == FP:
                tol = tol + 2.0 ** -25 * (ok.sum(-1)[:, None] * v.abs().max() + 1)
            err = (o[t0:t0 + n, h] - want).abs()
            assert (err <= tol).all(), (s, h, float((err / tol).max()))
            assert ((lse[t0:t0 + n, h] - torch.logsumexp(x, -1)).abs() <= e_s + 2e-5).all()
            missed |= bool(((p.to(dtype).double() @ v / total - want).abs() > tol).any())
        t0 += n
    assert missed


def test_two_streams_at_once_many_rows(spa):
    # both kernels and both element types in flight together
    cases = [Case([(300, 3000), (40, 900)], 16, 8, 2, 64, BF, "full", seed=1),
             Case([(513, 2000)], 64, 4, 4, 128, FP, "balanced", seed=2),
             Case([(1, 3000), (1, 2000)], 16, 8, 2, 64, BF, "full", seed=3)]
    want = [tuple(t.clone() for t in c.run(spa)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for c, s, g in zip(cases, streams, got):
            with torch.cuda.stream(s):
                g.append(c.run(spa))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o, lse in outs:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    assert spa.spa_device_status() == spa.SPA_OK


def test_random_bands_on_heads_that_share_keys(spa):
    # every query head its own band, four heads to a key/value head
    for seed, new in ((1, 1), (2, 9), (3, 70)):
        c = Case([(new, 500), (new, 333), (0, 40), (new, new)], 32, 8, 2, 64, BF, "full", seed=seed, N=512)
        g = torch.Generator().manual_seed(seed)
        c.lo = torch.randint(0, 300, (8,), generator=g).tolist()
        c.hi = [a + int(torch.randint(1, 212, (1,), generator=g)) for a in c.lo]
        c.check(*c.run(spa))
    assert spa.spa_device_status() == spa.SPA_OK


def median_ms(spa, case):
    """Device time of one call, from a graph of eight (no host time in it)."""
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(8):
            case.run(spa)
    times = []
    for _ in range(9):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) / 8)
    return sorted(times)[4]


def test_long_prompt_among_single_tokens(spa):
    # max_q gives every sequence the prompt's row blocks, almost all of them
    # empty: 16 sequences x 8 head groups x 128 blocks, 8 x 15 of which exist
    # behind the prompt's
    seqs = [(1, 200)] * 5 + [(8192, 8192)] + [(0, 70), (1, 256)] + [(1, 100)] * 8
    c = Case(seqs, 64, 32, 8, 64, BF, "window100", seed=12)
    o, lse = c.run(spa)
    t0 = 5 + 8192
    c.check(o, lse, rows=set(range(8)) | {4096, t0 - 1} | set(range(t0, c.T - 2)))
    assert (o[-2:] == 3.0).all() and (lse[-2:] == 5.0).all()
    assert spa.spa_device_status() == spa.SPA_OK
    # 14 single tokens next to 8192 are a fifth of its items and far less of
    # its work; steps over the empty blocks, one by one, took it several times
    alone = Case([(8192, 8192)], 64, 32, 8, 64, BF, "window100", seed=12)
    alone.run(spa)
    assert median_ms(spa, c) < 3 * median_ms(spa, alone)


@pytest.mark.parametrize("order", ["behind", "before", "between"])
def test_batch_padded_with_idle_sequences(spa, order):
    # a captured batch of 512 places, 16 of them taken
    live, idle = [(1, 900 + i) for i in range(16)], [(0, 0)] * 496
    seqs = {"behind": live + idle, "before": idle + live, "between": live[:15] + idle + live[15:]}[order]
    c = Case(seqs, 64, 32, 32, 64, BF, "full", seed=13, pad=496)
    c.check(*c.run(spa))
    assert spa.spa_device_status() == spa.SPA_OK
    # the idle places are 15872 items: stepping over each, at 0.17 us, took 2.7 ms
    # in the CTA they fell to.  As 496 sequences they cost the plan 16 us (1.5
    # times the attention alone), and 0.3 us each (5.6 times) where one CTA's run
    # goes across them
    alone = Case(live, 64, 32, 32, 64, BF, "full", seed=13)
    alone.run(spa)
    assert median_ms(spa, c) < (15 if order == "between" else 4) * median_ms(spa, alone)


def test_generation_captured_in_one_graph(spa):
    # append and attention of one token per sequence, captured once and replayed
    # while the lengths grow; then the same tokens as one prompt (the kernel for
    # many rows).  Both are off by the tolerance above: |o| <= A <= max|v|
    S, H, Hk, d, page, steps = 3, 8, 2, 64, 16, 50
    kp = torch.full((60, Hk, page, d), float("nan"), dtype=BF, device=DEV)
    vp = kp.clone()
    table = torch.randperm(60, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(S, 20).to(DEV)
    w, rope = torch.ones(d, device=DEV), spa.rope_table(320, d)
    kv, x = torch.ones(S, dtype=torch.int32, device=DEV), torch.zeros(S, H + 2 * Hk, d, dtype=BF, device=DEV)
    bands = dict(lo=[0] * H, hi=[320] * H, N=320)

    def tokens(x, cu, n):
        q, k, v = x.split([H, Hk, Hk], 1)
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV) if isinstance(cu, list) else cu
        return spa.paged_attention(spa.paged_append(q, k, v, kp, vp, table, cu, kv, w, w, rope), kp, vp, table, cu, kv,
                                   n, **bands)

    cu = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    tokens(x, cu, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = tokens(x, cu, 1)
    kp.fill_(float("nan"))
    vp.fill_(float("nan"))
    seen = torch.randn(steps, S, H + 2 * Hk, d, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    got = []
    for t in range(steps):
        kv.fill_(t + 1)
        x.copy_(seen[t])
        graph.replay()
        got.append((o.clone(), lse.clone()))
    keys, values = kp.clone(), vp.clone()
    kp.fill_(float("nan"))
    vp.fill_(float("nan"))
    o, lse = tokens(seen.transpose(0, 1).reshape(S * steps, -1, d), [0, steps, 2 * steps, 3 * steps], steps)
    assert spa.spa_device_status() == spa.SPA_OK
    for a, b in ((kp, keys), (vp, values)):  # one by one or together, the cache is the same
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
    far = 2 * (2 * HALF[BF] + 3e-5) * float(seen[:, :, H + Hk:].abs().max())
    for t, (ot, lt) in enumerate(got):
        assert float((o.view(S, steps, H, d)[:, t].float() - ot.float()).abs().max()) <= far
        assert float((lse.view(S, steps, H)[:, t] - lt).abs().max()) <= 1e-4
