"""GPU tests of the query/key norm and rotation (forward, backward, table)
and of the append to a paged cache, against the formulas in fp64.

Tolerances, from the arithmetic.  A result is rounded once to its type: half a
step, finfo(type).eps / 2 of its value (and half the smallest subnormal of
fp16, 2^-25).  Before that it is formed in fp32 with unit roundoff u = 2^-24:
  r      sum of squares over at most 8 fused steps and 4 shuffles, halved by
         the root (6 u), rsqrtf 2 ulp (4 u)                    -> 10 u
  y      two products on top of r, two products and a sum of the rotation
                                      -> 16 u < 1e-6 of |a c| + |b s|
  dx     g: 3 u; the row's dot product: 16 u of sum |g w x|; its factors: 24 u
         -> less than 60 u < 4e-6 of r (|g w| + |x| r^2 mean|g w x|)
  dw     every term 20 u; summed along at most 64 rows of a lane, 16 lane
         groups, 28 partials and 5 shuffles: 113 u -> 140 u < 1e-5 of sum |g n|
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from head_partitioned_distance_b200 import spa as mod
    return mod


DEV = "cuda:0"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def ref_table(length, rot, base=10000.0):
    ang = torch.arange(length, dtype=torch.float64)[:, None] * base ** (
        -2 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    return torch.stack((ang.cos(), ang.sin()), -1)


def pairs_of(x, rot, interleaved):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def turn(x, cs, interleaved, back=False, absolute=False):
    """x (fp64) rotated by the rows cs [.., rot / 2, 2]; absolute: the sum of
    the magnitudes instead (for error bounds)."""
    rot = 2 * cs.shape[-2]
    a, b = pairs_of(x, rot, interleaved)
    c, s = cs[..., 0], -cs[..., 1] if back else cs[..., 1]
    y = x.clone()
    ya, yb = pairs_of(y, rot, interleaved)
    if absolute:
        ya.copy_((a * c).abs() + (b * s).abs())
        yb.copy_((b * c).abs() + (a * s).abs())
        y[..., rot:] = x[..., rot:].abs()
    else:
        ya.copy_(a * c - b * s)
        yb.copy_(b * c + a * s)
    return y


def ref_fwd(x, w, cs, eps, interleaved):
    """y and the magnitude its fp32 error is relative to."""
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return turn(n, cs, interleaved), turn(n, cs, interleaved, absolute=True)


def check_fwd(got, x, w, cs, eps, interleaved):
    want, mag = ref_fwd(x, w, cs, eps, interleaved)
    err = (got.double().cpu() - want).abs()
    tol = HALF[got.dtype] * want.abs() + 1e-6 * mag + 2.0 ** -25
    assert (err <= tol).all(), float((err / tol).max())


def make(B, Hq, Hk, N, d, dtype, seed, layout="token"):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, N, Hq + 2 * Hk, d, generator=g).to(dtype).to(DEV)
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    if layout == "head":
        q, k = q.contiguous(), k.contiguous()
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    return q, k, wq.to(DEV), wk.to(DEV)


def rows_of(table, positions, N):
    """Table rows [1 or B, 1, N, rot / 2, 2] and validity [.., 1, N, 1]."""
    pos = torch.arange(N)[None] if positions is None else positions.cpu().long().reshape(-1, N)
    ok = (pos >= 0) & (pos < table.shape[0])
    return table[pos.clamp(0, table.shape[0] - 1)][:, None], ok[:, None, :, None]


SHAPES = [
    # B, Hq, Hk, N, d, rot, interleaved, dtype, layout
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, "token"),
    (1, 4, 4, 256, 64, 64, False, torch.bfloat16, "token"),
    (2, 8, 2, 101, 64, 32, True, torch.float16, "token"),
    (1, 3, 1, 33, 128, 48, False, torch.float16, "head"),
    (3, 5, 5, 77, 128, 128, False, torch.bfloat16, "head"),
    (2, 7, 1, 130, 128, 96, True, torch.bfloat16, "token"),
    (1, 32, 8, 600, 128, 128, False, torch.bfloat16, "token"),
    (1, 2, 6, 19, 64, 16, False, torch.bfloat16, "token"),
]


@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,il,dtype,layout", SHAPES)
def test_forward(spa, B, Hq, Hk, N, d, rot, il, dtype, layout):
    q, k, wq, wk = make(B, Hq, Hk, N, d, dtype, N + d, layout)
    table = spa.rope_table(N, rot)
    qo, ko = spa.qk_norm_rope_forward(q, k, wq, wk, table, eps=1e-5, interleaved=il)
    assert qo.is_contiguous() and ko.is_contiguous()
    cs = table.double().cpu()
    check_fwd(qo, q.double().cpu(), wq.double().cpu(), cs, 1e-5, il)
    check_fwd(ko, k.double().cpu(), wk.double().cpu(), cs, 1e-5, il)


def ref_bwd(dy, x, w, cs, eps, il, ok):
    g = turn(dy, cs, il, back=True) * ok
    mag_g = turn(dy, cs, il, absolute=True) * ok
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    mag = r * ((mag_g * w).abs() + x.abs() * r * r * (mag_g * w * x).abs().mean(-1, keepdim=True))
    return dx, mag, (g * n).sum((0, 1, 2)), (mag_g * n).abs().sum((0, 1, 2))


@pytest.mark.parametrize("with_positions", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,il,dtype,layout", SHAPES)
def test_backward(spa, B, Hq, Hk, N, d, rot, il, dtype, layout, with_positions):
    q, k, wq, wk = make(B, Hq, Hk, N, d, dtype, 3 * N + d, layout)
    g = torch.Generator().manual_seed(5)
    dqo = torch.randn(B, Hq, N, d, generator=g).to(dtype).to(DEV)
    dko = torch.randn(B, Hk, N, d, generator=g).to(dtype).to(DEV)
    table = spa.rope_table(N + 3, rot)
    positions = None
    if with_positions:  # two documents and, past them, padding
        positions = torch.arange(N).repeat(B, 1)
        positions[:, N // 2:] -= N // 2
        positions[-1, N - N // 4:] = -1
        positions = positions.to(torch.int32).to(DEV)
    got = spa.qk_norm_rope_backward(dqo, dko, q, k, wq, wk, table, positions, 1e-5, il)
    cs, ok = rows_of(table.double().cpu(), positions, N)
    for dx, dw, dy, x, w in ((got[0], got[2], dqo, q, wq), (got[1], got[3], dko, k, wk)):
        want, mag, dw_want, dw_mag = ref_bwd(dy.double().cpu(), x.double().cpu(), w.double().cpu(), cs, 1e-5, il, ok)
        err = (dx.double().cpu() - want).abs()
        tol = HALF[dtype] * want.abs() + 4e-6 * mag + 2.0 ** -25
        assert (err <= tol).all(), float((err / tol).max())
        err = (dw.double().cpu() - dw_want).abs()
        assert (err <= 1e-5 * dw_mag + 1e-30).all(), float((err / dw_mag).max())


def test_gradient_against_differences(spa):
    # the formula itself, by central differences in fp64 along random
    # directions of x and w (step h: error O(h^2) ~ 1e-8 of values of order 1
    # to 100, against a slope of that order)
    g = torch.Generator().manual_seed(1)
    x, dy = torch.randn(1, 2, 9, 64, generator=g).double(), torch.randn(1, 2, 9, 64, generator=g).double()
    w = 1 + 0.3 * torch.randn(64, generator=g).double()
    cs = ref_table(9, 64)
    f = lambda x_, w_: (ref_fwd(x_, w_, cs, 1e-5, False)[0] * dy).sum()  # noqa: E731
    dx, _, dw, _ = ref_bwd(dy, x, w, cs, 1e-5, False, torch.ones(1, 1, 9, 1))
    h = 1e-5
    for _ in range(3):
        u, v = torch.randn(x.shape, generator=g).double(), torch.randn(64, generator=g).double()
        diff = (f(x + h * u, w + h * v) - f(x - h * u, w - h * v)) / (2 * h)
        slope = (dx * u).sum() + (dw * v).sum()
        assert abs(diff - slope) <= 1e-6 * (1 + abs(slope))


def test_positions_and_padding(spa):
    B, H, N, d = 2, 3, 40, 64
    q, k, wq, wk = make(B, H, H, N, d, torch.bfloat16, 9)
    q[1, :, 30:] = float("nan")  # padded rows may hold anything
    k[1, :, 30:] = float("inf")
    table = spa.rope_table(25, 64)
    pos = torch.arange(N, dtype=torch.int32).repeat(B, 1) % 25
    pos[1, 30:] = torch.tensor([-1, 25, 1 << 30, -5, 26, -1, -1, 1000, -1, 25], dtype=torch.int32)
    pos = pos.to(DEV)
    qo, ko = spa.qk_norm_rope_forward(q, k, wq, wk, table, pos)
    assert (qo[1, :, 30:] == 0).all() and (ko[1, :, 30:] == 0).all()
    cs, _ = rows_of(table.double().cpu(), pos, N)
    check_fwd(qo[:, :, :30], q[:, :, :30].double().cpu(), wq.double().cpu(), cs[:, :, :30], 1e-6, False)
    # the padded rows leave the weights' gradients alone
    dqo, dko = torch.ones_like(qo), torch.ones_like(ko)
    got = spa.qk_norm_rope_backward(dqo, dko, q, k, wq, wk, table, pos)
    q2, k2 = q.clone(), k.clone()
    q2[1, :, 30:] = 0
    k2[1, :, 30:] = 0
    again = spa.qk_norm_rope_backward(dqo, dko, q2, k2, wq, wk, table, pos)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    assert (got[0][1, :, 30:] == 0).all()
    # one row of positions for the whole batch
    one = torch.arange(N, dtype=torch.int32, device=DEV) % 25
    a = spa.qk_norm_rope_forward(q2, k2, wq, wk, table, one)
    b = spa.qk_norm_rope_forward(q2, k2, wq, wk, table, one.repeat(B, 1))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_table_far_positions(spa):
    # pos * freq in fp32 would be off by pos * 2^-24 rad; the table is formed in fp64
    length, rot = 1 << 20, 32
    table = spa.rope_table(length, rot, 500000.0)
    want = ref_table(length, rot, 500000.0)
    err = (table.double().cpu() - want).abs()
    # one rounding to fp32 (2^-25 of at most 1); the fp64 angles differ by a few 2^-53 of 2^20
    assert float(err.max()) <= 2.0 ** -25 + 1e-9


def test_repeated_calls_are_equal(spa):
    q, k, wq, wk = make(2, 8, 8, 3001, 128, torch.bfloat16, 4)
    table = spa.rope_table(3001, 128)
    a = spa.qk_norm_rope_backward(q.contiguous(), k.contiguous(), q, k, wq, wk, table)
    b = spa.qk_norm_rope_backward(q.contiguous(), k.contiguous(), q, k, wq, wk, table)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_autograd_from_fused_projection_to_attention(spa):
    # a layer's path: fused projection -> norm and rotation -> spattention,
    # gradients back to the projection and the weights
    B, H, N, d = 2, 4, 300, 64
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, N, 3 * H, d, generator=g).to(torch.bfloat16).to(DEV).requires_grad_()
    wq = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV).requires_grad_()
    wk = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).to(DEV).requires_grad_()
    table = spa.rope_table(N, d)
    q, k, v = (t.transpose(1, 2) for t in qkv.split(H, 2))
    qn, kn = spa.qk_norm_rope(q, k, wq, wk, table)
    o = spa.spattention(qn, kn, v)
    do = torch.randn(o.shape, generator=g).to(torch.bfloat16).to(DEV)
    o.backward(do)
    assert spa.spa_device_status() == spa.SPA_OK
    # the same chain call by call
    qs, ks, vs = (t.detach() for t in (q, k, v))
    q2, k2 = spa.qk_norm_rope_forward(qs, ks, wq.detach(), wk.detach().float(), table)
    vc = vs.contiguous()
    o2, lse = spa.attention_forward(q2, k2, vc)
    dq2, dk2, dv2 = spa.attention_backward(q2, k2, vc, o2, do, lse)
    dq, dk, dwq, dwk = spa.qk_norm_rope_backward(dq2, dk2, qs, ks, wq.detach(), wk.detach().float(), table)
    assert torch.equal(o, o2)
    assert torch.equal(qkv.grad, torch.cat([t.transpose(1, 2) for t in (dq, dk, dv2)], 2))
    assert torch.equal(wq.grad, dwq) and torch.equal(wk.grad, dwk.to(torch.bfloat16))


def test_broadcast_key_and_odd_layout(spa):
    # one key head expanded to four (stride 0): its gradient is the sum; a
    # layout that is not of whole vectors is copied by the autograd function
    B, H, N, d = 1, 4, 50, 64
    q, k, wq, wk = make(B, H, 1, N, d, torch.bfloat16, 6)
    table = spa.rope_table(N, 64)
    leaf = k.detach().clone().requires_grad_()
    qo, ko = spa.qk_norm_rope(q, leaf.expand(B, H, N, d), wq, wk, table)
    dko = torch.randn(ko.shape, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    (ko * dko).sum().backward()
    full = spa.qk_norm_rope_backward(torch.zeros_like(qo), dko, q, k.expand(B, H, N, d), wq, wk, table)
    assert torch.equal(leaf.grad, full[1].sum(1, keepdim=True))
    odd = torch.randn(B, H, N, d + 1, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)[..., :d]
    with pytest.raises(ValueError, match="16-byte"):
        spa.qk_norm_rope_forward(odd, odd, wq, wk, table)
    a = spa.qk_norm_rope(odd, odd, wq, wk, table)
    b = spa.qk_norm_rope_forward(odd.contiguous(), odd.contiguous(), wq, wk, table)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_other_stream_and_graph(spa):
    q, k, wq, wk = make(1, 8, 8, 200, 64, torch.bfloat16, 8)
    table = spa.rope_table(200, 64)
    dq, dk = torch.randn_like(q).contiguous(), torch.randn_like(k).contiguous()
    want = spa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = spa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, table)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd = spa.qk_norm_rope_forward(q, k, wq, wk, table)
        bwd = spa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, table)
    q.copy_(torch.randn_like(q))
    graph.replay()
    for a, b in zip(fwd + bwd, spa.qk_norm_rope_forward(q, k, wq, wk, table)
                    + spa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, table)):
        assert torch.equal(a, b)


def test_forward_and_backward_in_one_graph(spa):
    # a training step's part, captured: autograd inside the capture
    q, k, wq, wk = make(1, 4, 2, 100, 64, torch.bfloat16, 3)
    table = spa.rope_table(100, 64)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, wq, wk)]
    dq, dk = torch.randn(1, 4, 100, 64, device=DEV).bfloat16(), torch.randn(1, 2, 100, 64, device=DEV).bfloat16()
    step = lambda: torch.autograd.grad(spa.qk_norm_rope(*leaves, table), leaves, (dq, dk))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        leaves[0].copy_(torch.randn_like(q))
    graph.replay()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ append
def paged(seqs, page, Hk, d, dtype, seed, spare=2, fill=0.0):
    """seqs: list of (new tokens, length with them).  Pages in random order."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-c // page) for _, c in seqs]
    pages, width = sum(used) + spare, max(max(used), 1) + 1
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table, at = torch.full((len(seqs), width), -7, dtype=torch.int32), 0
    for s, n in enumerate(used):
        table[s, :n] = perm[at:at + n]
        at += n
    cu = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32)
    kv = torch.tensor([c for _, c in seqs], dtype=torch.int32)
    cache = lambda: torch.full((pages, Hk, page, d), fill, dtype=dtype, device=DEV)  # noqa: E731
    return table.to(DEV), cu.to(DEV), kv.to(DEV), cache(), cache()


APPENDS = [
    # seqs, page, Hq, Hk, d, rot, interleaved, dtype, padded rows
    ([(1, 1)], 16, 1, 1, 64, 64, False, torch.bfloat16, 0),
    ([(1, 40), (1, 17), (1, 1), (1, 64)], 16, 8, 2, 64, 32, True, torch.float16, 3),
    ([(70, 70), (0, 33), (1, 200), (31, 95), (0, 0)], 32, 6, 3, 128, 96, False, torch.bfloat16, 5),
    ([(300, 513)], 128, 4, 4, 128, 128, False, torch.bfloat16, 0),
    ([(1, 300 + i) for i in range(70)], 64, 5, 1, 128, 128, False, torch.bfloat16, 2),
    ([(257, 600), (5, 256)], 256, 2, 1, 64, 48, False, torch.float16, 1),
]


@pytest.mark.parametrize("seqs,page,Hq,Hk,d,rot,il,dtype,pad", APPENDS)
def test_append(spa, seqs, page, Hq, Hk, d, rot, il, dtype, pad):
    table, cu, kv, kp, vp = paged(seqs, page, Hk, d, dtype, 11, fill=7.0)
    n = int(cu[-1])
    T = n + pad
    g = torch.Generator().manual_seed(12)
    qkv = torch.randn(T, Hq + 2 * Hk, d, generator=g).to(dtype).to(DEV)
    q, k, v = qkv.split([Hq, Hk, Hk], 1)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(DEV) for _ in range(2))
    rope = spa.rope_table(max(c for _, c in seqs), rot)
    out = torch.full((T, Hq, d), 3.0, dtype=dtype, device=DEV)
    got = spa.paged_append(q, k, v, kp, vp, table, cu, kv, wq, wk, rope, 1e-5, il, out)
    assert got is out and spa.spa_device_status() == spa.SPA_OK
    pos, kw, vw = [], torch.full_like(kp, 7.0), torch.full_like(vp, 7.0)
    for (m, c) in seqs:
        pos += list(range(c - m, c))
    cs = rope.double().cpu()[pos][:, None]
    if n:
        check_fwd(out[:n], q[:n].double().cpu(), wq.double().cpu(), cs, 1e-5, il)
    assert (out[n:] == 3.0).all()
    # every key and value in its place, everything else untouched
    t = 0
    places = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    knew = torch.empty(n, Hk, d, dtype=dtype, device=DEV)
    for s, (m, c) in enumerate(seqs):
        for p in range(c - m, c):
            pg = int(table[s, p // page])
            knew[t] = kp[pg, :, p % page]
            vw[pg, :, p % page] = v[t]
            places[pg, p % page] = True
            t += 1
    if n:
        check_fwd(knew, k[:n].double().cpu(), wk.double().cpu(), cs, 1e-5, il)
    assert torch.equal(vp, vw)
    assert (kp.transpose(1, 2)[~places.to(DEV)] == 7.0).all()


def test_append_refuses_places_on_the_device(spa):
    # a page number outside the pages, a position past the page table or the
    # rope table: nothing cached, a zero query row, an error from the status
    table, cu, kv, kp, vp = paged([(1, 20), (1, 5), (1, 30), (1, 3)], 16, 1, 64, torch.bfloat16, 1, fill=7.0)
    table[0, 1] = kp.shape[0]
    table[1, 0] = -1
    kv[2] = 16 * table.shape[1] + 1
    q = torch.randn(4, 2, 64, device=DEV, dtype=torch.bfloat16)
    k, v = q[:, :1], q[:, 1:]
    w = torch.ones(64, device=DEV)
    out = torch.full_like(q, 3.0)
    spa.paged_append(q, k, v, kp, vp, table, cu, kv, w, w, spa.rope_table(1000, 64), out=out)
    assert spa.spa_device_status() == spa.SPA_ERR_INVAL
    assert spa.spa_device_status() == spa.SPA_OK
    assert (out[:3] == 0).all() and (out[3] != 0).any()
    assert int((kp != 7.0).any(-1).sum()) == 1 and int((vp != 7.0).any(-1).sum()) == 1
    kv[2] = 30
    table[0, 1], table[1, 0] = 0, 1
    spa.paged_append(q, k, v, kp, vp, table, cu, kv, w, w, spa.rope_table(29, 64), out=out)
    assert spa.spa_device_status() == spa.SPA_ERR_INVAL
    assert (out[2] == 0).all() and (out[:2] != 0).any()


def test_append_no_tokens(spa):
    table, cu, kv, kp, vp = paged([(0, 20)], 16, 1, 64, torch.bfloat16, 1, fill=7.0)
    q = torch.empty(0, 2, 64, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(64, device=DEV)
    out = spa.paged_append(q, q[:, :1], q[:, 1:], kp, vp, table, cu, kv, w, w, spa.rope_table(32, 64))
    assert out.shape == q.shape and (kp == 7.0).all()


@pytest.mark.parametrize("order", ["token", "head", "expanded", "batch_last"])
def test_gradients_keep_the_layout(spa, order):
    # dq and dk are dense whatever q and k are views of, and in their order of dimensions
    B, H, N, d = 2, 3, 20, 64
    x = torch.randn(B, N, 2 * H, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    q = {"token": lambda: x[:, :, :H].transpose(1, 2), "head": lambda: x[:, :, :H].transpose(1, 2).contiguous(),
         "expanded": lambda: x[:, :, :1].transpose(1, 2).expand(B, H, N, d),
         "batch_last": lambda: x[:, :, :H].permute(1, 2, 0, 3).contiguous().permute(2, 1, 0, 3)}[order]()
    w, table = torch.ones(d, device=DEV), spa.rope_table(N, d)
    dq = torch.randn(B, H, N, d, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    got = spa.qk_norm_rope_backward(dq, dq, q, q, w, w, table)
    want = spa.qk_norm_rope_backward(dq, dq, q.contiguous(), q.contiguous(), w, w, table)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    span = sum((n - 1) * s for n, s in zip(got[0].shape, got[0].stride())) + 1
    assert span == got[0].numel()
    if order == "token":
        assert got[0].transpose(1, 2).is_contiguous()


def test_autograd_takes_values_off_a_vector_border(spa):
    # gradients that arrive as parts of a longer one, and weights that are parts
    # of a flat parameter, start anywhere; so may rows of q and k that are dense
    B, H, N, d = 1, 3, 21, 64
    q, k, wq, wk = make(B, H, 1, N, d, torch.bfloat16, 31, "head")
    table = spa.rope_table(N, d)
    g = torch.Generator().manual_seed(32)
    dq, dk = (torch.randn(t.shape, generator=g).to(torch.bfloat16).to(DEV) for t in (q, k))

    def off(t, by):  # the same values, contiguous, `by` elements behind a border
        flat = t.new_empty(t.numel() + by)
        flat[by:] = t.flatten()
        return flat[by:].view(t.shape)

    want = spa.qk_norm_rope_forward(q, k, wq, wk, table)
    want_g = spa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, table)
    for by in (1, 3):
        leaves = [off(t, by).requires_grad_() for t in (q, k, wq, wk)]
        assert all(t.data_ptr() % 16 for t in leaves)
        out = spa.qk_norm_rope(*leaves, off(table, by))
        got = torch.autograd.grad(out, leaves, (off(dq, by), off(dk, by)))
        for a, b in zip(out + got, want + want_g):
            assert torch.equal(a, b)
    # as it happens: both outputs joined behind something of odd length
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, wq, wk)]
    qn, kn = spa.qk_norm_rope(*leaves, table)
    long = torch.cat((qn.new_zeros(3), qn.flatten(), kn.flatten()))
    got = torch.autograd.grad(long, leaves, torch.cat((dq.new_ones(3), dq.flatten(), dk.flatten())))
    for a, b in zip(got, want_g):
        assert torch.equal(a, b)


def test_the_kernels_gradient_against_differences(spa):
    # the slope that the backward's outputs give along random directions of x
    # and both weights, against central differences of the formula in fp64
    # (step 1e-5: error 1e-6 of the slope's scale); each output may be off by
    # its tolerance above, times the direction's magnitude there
    B, Hq, Hk, N, d, rot, eps = 1, 3, 2, 11, 64, 48, 1e-5
    for il, dtype in ((False, torch.bfloat16), (True, torch.float16)):
        q, k, wq, wk = make(B, Hq, Hk, N, d, dtype, 51)
        g = torch.Generator().manual_seed(52)
        dqo = torch.randn(B, Hq, N, d, generator=g).to(dtype).to(DEV)
        dko = torch.randn(B, Hk, N, d, generator=g).to(dtype).to(DEV)
        table = spa.rope_table(N, rot)
        dq, dk, dwq, dwk = spa.qk_norm_rope_backward(dqo, dko, q, k, wq, wk, table, None, eps, il)
        cs, ok = table.double().cpu(), torch.ones(1, 1, N, 1)
        for dx, dw, dy, x, w in ((dq, dwq, dqo, q, wq), (dk, dwk, dko, k, wk)):
            dx, dw, dy, x, w = (t.detach().double().cpu() for t in (dx, dw, dy, x, w))
            f = lambda x_, w_: (ref_fwd(x_, w_, cs, eps, il)[0] * dy).sum()  # noqa: E731
            _, mag, _, dw_mag = ref_bwd(dy, x, w, cs, eps, il, ok)
            off = HALF[dtype] * dx.abs() * 1.01 + 4e-6 * mag + 2.0 ** -25
            for _ in range(3):
                u, v = torch.randn(x.shape, generator=g).double(), torch.randn(d, generator=g).double()
                h = 1e-5
                diff = (f(x + h * u, w + h * v) - f(x - h * u, w - h * v)) / (2 * h)
                tol = (off * u.abs()).sum() + (1e-5 * dw_mag * v.abs()).sum() + 1e-6 * (1 + diff.abs())
                assert abs((dx * u).sum() + (dw * v).sum() - diff) <= tol
                # a direction of one element each: where no sum hides a wrong sign
                for i in torch.randint(0, x.numel(), (8,), generator=g).tolist():
                    e = torch.zeros(x.numel()).double()
                    e[i] = 1
                    e = e.view(x.shape)
                    diff = (f(x + h * e, w) - f(x - h * e, w)) / (2 * h)
                    assert abs((dx * e).sum() - diff) <= (off * e).sum() + 1e-6 * (1 + diff.abs())


def test_append_beside_refused_tokens(spa):
    # tokens without a place leave the others' rows, keys and values right
    table, cu, kv, kp, vp = paged([(2, 20), (3, 5), (1, 30), (2, 3)], 16, 2, 64, torch.bfloat16, 1, fill=7.0)
    table[0, 1] = kp.shape[0]  # positions 18 and 19 of the first sequence
    q, k, wq, wk = make(1, 4, 2, 8, 64, torch.bfloat16, 3)
    q, k = q[0].transpose(0, 1), k[0].transpose(0, 1)
    v = torch.randn(8, 2, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    rope = spa.rope_table(30, 64)
    out = spa.paged_append(q, k, v, kp, vp, table, cu, kv, wq, wk, rope, 1e-5)
    assert spa.spa_device_status() == spa.SPA_ERR_INVAL
    assert (out[:2] == 0).all()
    pos = [2, 3, 4, 29, 1, 2]
    cs = rope.double().cpu()[pos][:, None]
    check_fwd(out[2:], q[2:].double().cpu(), wq.double().cpu(), cs, 1e-5, False)
    seq = [1, 1, 1, 2, 3, 3]
    page, at = [int(table[s, p // 16]) for s, p in zip(seq, pos)], [p % 16 for p in pos]
    check_fwd(kp[page, :, at], k[2:].double().cpu(), wk.double().cpu(), cs, 1e-5, False)
    assert torch.equal(vp[page, :, at], v[2:])
    assert int((vp != 7.0).flatten(2).any(-1).sum()) <= 6 * 2 and int((vp[:, 0] != 7.0).any(-1).sum()) == 6
