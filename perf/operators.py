"""The operators that stand around the band-sparse attention in a language
model, as cases that can be measured: what each computes in plain torch, the
framework's own calls for it, and its definition in 64 bits.

* ``norm_rope``: RMS norm of every query and key head with a learned weight,
  then the rotary position rotation, from the token-major projections into
  the head-major tensors the attention takes; forward and backward.
* ``append``: the same norm and rotation for the new tokens of several
  sequences, their keys and values written into a paged cache.
* ``attend``: attention of those new tokens (one or many for each sequence)
  over the paged cache, every head over its own band of causal distances.

``own`` chooses between the plain forms (False) and the framework (True).
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest layer of the repository's workloads: launch latency
        {"name": "norm_rope_bwd_b1_h4_n256_d64", "op": "norm_rope_bwd", "B": 1, "Hq": 4, "Hk": 4, "N": 256, "d": 64,
         "rot": 64, "pairs": "halves", "dtype": "bf16", "positions": False},
        # odd length, half of each head rotated, neighbouring pairs, packed documents that restart their positions
        {"name": "norm_rope_fwd_b1_h8_n1001_d64", "op": "norm_rope_fwd", "B": 1, "Hq": 8, "Hk": 8, "N": 1001, "d": 64,
         "rot": 32, "pairs": "neighbours", "dtype": "fp16", "positions": True},
        # the projections of a 7B-like layer on their way into the attention
        {"name": "norm_rope_fwd_b4_h32_n8192_d128", "op": "norm_rope_fwd", "B": 4, "Hq": 32, "Hk": 32, "N": 8192,
         "d": 128, "rot": 128, "pairs": "halves", "dtype": "bf16", "positions": False},
        # the long ragged workload, keys shared by four query heads, on the way back
        {"name": "norm_rope_bwd_b1_h32_n30001_d128", "op": "norm_rope_bwd", "B": 1, "Hq": 32, "Hk": 8, "N": 30001,
         "d": 128, "rot": 128, "pairs": "halves", "dtype": "bf16", "positions": False},
        # one generation step of 64 sequences, in a batch padded to a captured graph's size
        {"name": "append_decode_s64_h32_d128", "op": "append", "seqs": 64, "chunk": 1, "ctx": 4096, "lens": "wide",
         "lens_seed": 1, "pad": 8, "Hq": 32, "Hk": 32, "d": 128, "rot": 128, "pairs": "halves", "dtype": "bf16",
         "page": 64},
        # prompts of several sequences, processed together
        {"name": "append_prompt_s5_h32_d128", "op": "append", "seqs": 5, "chunk": 4096, "ctx": 8192, "lens": "near",
         "lens_seed": 2, "pad": 0, "Hq": 32, "Hk": 8, "d": 128, "rot": 64, "pairs": "halves", "dtype": "fp16",
         "page": 16},
        # one sequence, one token, the odd small workload: launch latency
        {"name": "attend_decode_s1_h8_n1001_d64", "op": "attend", "seqs": 1, "chunk": 1, "ctx": 1001, "lens": "even",
         "lens_seed": 3, "pad": 0, "Hq": 8, "Hk": 8, "d": 64, "bands": "balanced", "width": 0, "dtype": "bf16",
         "page": 16},
        # generation with the long workload's bands (width 1024)
        {"name": "attend_decode_s8_h32_n32768_d128", "op": "attend", "seqs": 8, "chunk": 1, "ctx": 32768,
         "lens": "near", "lens_seed": 4, "pad": 0, "Hq": 32, "Hk": 32, "d": 128, "bands": "balanced", "width": 0,
         "dtype": "bf16", "page": 64},
        # generation over the whole context, keys shared by four query heads
        {"name": "attend_decode_s16_h32_kv8_full", "op": "attend", "seqs": 16, "chunk": 1, "ctx": 32768,
         "lens": "near", "lens_seed": 5, "pad": 0, "Hq": 32, "Hk": 8, "d": 128, "bands": "full", "width": 0,
         "dtype": "bf16", "page": 32},
        # new prompts next to sequences that generate, a sliding window of odd width
        {"name": "attend_mixed_s13_h16_kv4_d64", "op": "attend", "seqs": 13, "chunk": 700, "ctx": 4096,
         "lens": "wide", "lens_seed": 6, "pad": 5, "Hq": 16, "Hk": 4, "d": 64, "bands": "window", "width": 1000,
         "dtype": "fp16", "page": 16},
        # a chunk of a long prompt with the long workload's bands
        {"name": "attend_chunk_s1_h32_n32768_d128", "op": "attend", "seqs": 1, "chunk": 2048, "ctx": 32768,
         "lens": "even", "lens_seed": 7, "pad": 0, "Hq": 32, "Hk": 32, "d": 128, "bands": "balanced", "width": 0,
         "dtype": "bf16", "page": 64},
        # chunks of two long prompts over everything before them: the most arithmetic
        {"name": "attend_chunk_s2_h32_kv8_full", "op": "attend", "seqs": 2, "chunk": 4096, "ctx": 16384,
         "lens": "even", "lens_seed": 8, "pad": 0, "Hq": 32, "Hk": 8, "d": 128, "bands": "full", "width": 0,
         "dtype": "bf16", "page": 128},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def _drawn(rng):
    op = rng.choice(["norm_rope_fwd", "norm_rope_bwd", "append", "append", "attend", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    Hq = Hk * rng.choice([g for g in (1, 1, 2, 3, 4, 6, 8) if Hk * g <= 40])
    case = {"op": op, "Hq": Hq, "Hk": Hk, "d": d, "dtype": rng.choice(["bf16", "fp16"])}
    if op != "attend":
        case |= {"rot": rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d]),
                 "pairs": rng.choice(["halves", "neighbours"])}
    if op.startswith("norm_rope"):
        return case | {"B": _log(rng, 1, 8), "N": _log(rng, 1, 32768), "positions": rng.random() < 0.5}
    chunk = 1 if rng.random() < 0.4 else _log(rng, 1, 4096)
    case |= {"seqs": _log(rng, 1, 64), "chunk": chunk, "ctx": max(chunk, _log(rng, 16, 32768)),
             "lens": rng.choice(["even", "near", "wide"]), "lens_seed": rng.randrange(1 << 30),
             "pad": rng.choice([0, 0, rng.randrange(1, 40)]), "page": rng.choice([16, 32, 64, 128])}
    if op == "attend":
        case |= {"bands": rng.choice(["balanced", "full", "window"]), "width": _log(rng, 1, 4096)}
        if case["bands"] == "balanced":
            case["ctx"] = max(case["ctx"], case["Hq"])
    return case


def draw(rng):
    largest = max((c for c in listed() if c["op"] == "attend"), key=lambda c: work(c)["flops"])
    most = {"flops": work(largest)["flops"], "bytes": max(work(c)["bytes"] for c in listed())}
    while True:
        case = _drawn(rng)
        w = work(case)
        # what the plain form holds at once: padded scores, the gathered cache
        held = 0
        if case["op"] == "attend":
            held = case["seqs"] * case["ctx"] * (case["Hq"] * case["chunk"] + 2 * case["Hk"] * case["d"]) * 4
        if w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"] and held <= 18e9:
            return case


# ------------------------------------------------------------------ sizes
def _lengths(case):
    """New tokens and cached tokens (the new ones included) of each sequence."""
    rng = random.Random(case["lens_seed"])
    new, kept = [], []
    for s in range(case["seqs"]):
        n, c = case["chunk"], case["ctx"]
        if s and case["lens"] == "near":
            n, c = rng.randint((n + 1) // 2, n), rng.randint(max(n, c // 2), c)
        elif s and case["lens"] == "wide":
            n = 1 if rng.random() < 0.5 else _log(rng, 1, n)
            c = max(n, _log(rng, n, c))
        new.append(n)
        kept.append(c)
    return new, kept


def _bands(case):
    """The causal distances [lo, hi) of each query head."""
    H, N = case["Hq"], case["ctx"]
    if case["bands"] == "balanced":
        return [h * N // H for h in range(H)], [(h + 1) * N // H for h in range(H)]
    return [0] * H, [N if case["bands"] == "full" else min(case["width"], N)] * H


def work(case):
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if case["op"].startswith("norm_rope"):
        elems = case["B"] * case["N"] * (Hq + Hk) * d
        passes, flops = (2, 8) if case["op"].endswith("fwd") else (3, 18)
        small = case["N"] * case["rot"] * 4 + 2 * d * 4 * (1 if passes == 2 else 2)
        return {"bytes": passes * elems * 2 + small, "flops": flops * elems}
    new, kept = _lengths(case)
    T = sum(new)
    if case["op"] == "append":
        return {"bytes": 2 * T * (Hq + 2 * Hk) * d * 2 + T * case["rot"] * 4, "flops": 8 * T * (Hq + Hk) * d}
    lo, hi = _bands(case)
    pairs = keys = 0
    for n, c in zip(new, kept):
        pos = np.arange(c - n, c, dtype=np.int64)
        for g in range(Hk):
            spans = []
            for h in range(g * (Hq // Hk), (g + 1) * (Hq // Hk)):
                pairs += int(np.maximum(np.minimum(pos + 1, hi[h]) - lo[h], 0).sum())
                if c - 1 >= lo[h]:
                    spans.append((max(0, c - n - hi[h] + 1), c - lo[h]))
            end = 0
            for a, b in sorted(spans):  # keys that at least one head of the group reads
                keys += max(0, b - max(a, end))
                end = max(end, b)
    return {"bytes": 2 * keys * d * 2 + 2 * T * Hq * d * 2 + 4 * T * Hq, "flops": 4 * d * pairs}


# ------------------------------------------------------------------ inputs
def _table(length, rot):
    """cos and sin of position x 10000^(-2 i / rot), as [length, rot / 2, 2]."""
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float()


def _paged(case, g, dtype):
    new, kept = _lengths(case)
    page, Hk, d = case["page"], case["Hk"], case["d"]
    used = [-(-c // page) for c in kept]
    width, pages = max(used), sum(used) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(kept), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = perm[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    return {"page_table": table, "T": starts[-1] + case["pad"], "used": starts[-1], "max_q": case["chunk"],
            "cu_q": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "kv_len": torch.tensor(kept, dtype=torch.int32, device="cuda"),
            "k_pages": rand(pages, Hk, page, d), "v_pages": rand(pages, Hk, page, d)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, d, Hq, Hk = DTYPES[case["dtype"]], case["d"], case["Hq"], case["Hk"]
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    st = {"op": case["op"], "Hq": Hq, "Hk": Hk}
    if case["op"] != "attend":
        weight = lambda: 1 + 0.2 * torch.randn(d, generator=g, device="cuda")  # noqa: E731
        st |= {"q_weight": weight(), "k_weight": weight(), "neighbours": case["pairs"] == "neighbours"}
    if case["op"].startswith("norm_rope"):
        B, N = case["B"], case["N"]
        qkv = rand(B, N, Hq + 2 * Hk, d)  # the fused projection, token by token
        st |= {"q": qkv[:, :, :Hq].transpose(1, 2), "k": qkv[:, :, Hq:Hq + Hk].transpose(1, 2),
               "table": _table(N, case["rot"]), "positions": None}
        if case["positions"]:  # each row of the batch holds two documents
            cut = torch.randint(0, N, (B, 1), generator=g, device="cuda")
            i = torch.arange(N, device="cuda")[None]
            st["positions"] = torch.where(i < cut, i, i - cut).to(torch.int32)
        if case["op"].endswith("bwd"):
            st |= {"dq_out": rand(B, Hq, N, d), "dk_out": rand(B, Hk, N, d)}
        return st
    st |= _paged(case, g, dtype)
    T = st["T"]
    st["out"] = rand(T, Hq, d)
    if case["op"] == "append":
        qkv = rand(T, Hq + 2 * Hk, d)
        st |= {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:], "table": _table(case["ctx"], case["rot"])}
        return st
    lo, hi = _bands(case)
    st |= {"q": rand(T, Hq, d), "lse": torch.randn(T, Hq, generator=g, device="cuda"), "lo": lo, "hi": hi,
           "N": case["ctx"], "scale": d ** -0.5, "lo_dev": torch.tensor(lo, device="cuda"),
           "hi_dev": torch.tensor(hi, device="cuda")}
    return st


# ------------------------------------------------------------------ plain forms
def _split(x, neighbours):
    return (x[..., 0::2], x[..., 1::2]) if neighbours else x.chunk(2, -1)


def _join(a, b, neighbours):
    return torch.stack((a, b), -1).flatten(-2) if neighbours else torch.cat((a, b), -1)


def _turn(x, cs, neighbours, back=False):
    """The first rot columns of x rotated by the table rows cs (or back)."""
    rot = 2 * cs.shape[-2]
    cos, sin = cs[..., 0], -cs[..., 1] if back else cs[..., 1]
    a, b = _split(x[..., :rot], neighbours)
    return torch.cat((_join(a * cos - b * sin, b * cos + a * sin, neighbours), x[..., rot:]), -1)


def _norm_rope(x, w, cs, neighbours):
    x = x.float()
    return _turn(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w, cs, neighbours)


def _norm_rope_back(dy, x, w, cs, neighbours):
    x, g = x.float(), _turn(dy.float(), cs, neighbours, back=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, gw = x * r, g * w
    return (gw - n * (gw * n).mean(-1, keepdim=True)) * r, (g * n).sum((0, 1, 2))


def _rows(st):
    """Sequence, index within the sequence's new tokens and validity of each token row."""
    t = torch.arange(st["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["cu_q"], t, right=True) - 1
    valid = t < st["cu_q"][-1]
    b = b.clamp(max=st["kv_len"].numel() - 1)
    return b, (t - st["cu_q"][b]).clamp(max=st["max_q"] - 1), valid


def _plain_append(st):
    b, r, valid = _rows(st)
    cu, kv, pages = st["cu_q"], st["kv_len"], st["k_pages"]
    size = pages.shape[2]
    pos = torch.where(valid, kv[b] - (cu[b + 1] - cu[b]) + r, 0).long()
    cs = st["table"][pos][:, None]
    q = _norm_rope(st["q"], st["q_weight"], cs, st["neighbours"]).to(pages.dtype)
    k = _norm_rope(st["k"], st["k_weight"], cs, st["neighbours"]).to(pages.dtype)
    torch.where(valid[:, None, None], q, st["out"], out=st["out"])
    n = st["used"]
    page, at = st["page_table"][b[:n], pos[:n] // size].long(), pos[:n] % size
    st["k_pages"][page, :, at] = k[:n]
    st["v_pages"][page, :, at] = st["v"][:n]
    return {"q": st["out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_attend(st):
    cu, kv, Hq, Hk, mq = st["cu_q"], st["kv_len"], st["Hq"], st["Hk"], st["max_q"]
    B, d = kv.numel(), st["q"].shape[-1]
    r = torch.arange(mq, device="cuda")
    q = st["q"][(cu[:-1, None] + r).clamp(max=st["T"] - 1).long()].float()           # [B, mq, Hq, d]
    q = q.view(B, mq, Hk, Hq // Hk, d).permute(0, 2, 3, 1, 4)                         # [B, Hk, G, mq, d]
    table = st["page_table"].clamp(min=0).long()
    L = table.shape[1] * st["k_pages"].shape[2]
    k = st["k_pages"][table].transpose(1, 2).reshape(B, Hk, 1, L, d).float()
    v = st["v_pages"][table].transpose(1, 2).reshape(B, Hk, 1, L, d).float()
    j = torch.arange(L, device="cuda")
    pos = kv[:, None] - (cu[1:] - cu[:-1])[:, None] + r                                # [B, mq]
    dist = (pos[:, :, None] - j)[:, None, None]                                        # [B, 1, 1, mq, L]
    lo, hi = st["lo_dev"].view(Hk, -1, 1, 1), st["hi_dev"].view(Hk, -1, 1, 1)
    seen = (dist >= lo) & (dist < hi) & (j < kv[:, None])[:, None, None, None]
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"]).masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l.clamp(min=1e-30)
    lse = torch.where(l > 0, m + l.log(), -math.inf)
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, mq, Hq, d), lse.permute(0, 3, 1, 2, 4).reshape(B, mq, Hq)
    b, i, valid = _rows(st)
    torch.where(valid[:, None, None], o[b, i].to(st["out"].dtype), st["out"], out=st["out"])
    torch.where(valid[:, None], lse[b, i], st["lse"], out=st["lse"])
    return {"o": st["out"], "lse": st["lse"]}


def _plain(st):
    if st["op"] == "append":
        return _plain_append(st)
    if st["op"] == "attend":
        return _plain_attend(st)
    dtype, nb = st["q"].dtype, st["neighbours"]
    N = st["q"].shape[2]
    cs = st["table"][:N][None, None] if st["positions"] is None else st["table"][st["positions"].long()][:, None]
    if st["op"] == "norm_rope_fwd":
        return {"q": _norm_rope(st["q"], st["q_weight"], cs, nb).to(dtype),
                "k": _norm_rope(st["k"], st["k_weight"], cs, nb).to(dtype)}
    dq, dwq = _norm_rope_back(st["dq_out"], st["q"], st["q_weight"], cs, nb)
    dk, dwk = _norm_rope_back(st["dk_out"], st["k"], st["k_weight"], cs, nb)
    return {"dq": dq.to(dtype), "dk": dk.to(dtype), "dq_weight": dwq, "dk_weight": dwk}


# ------------------------------------------------------------------ the framework's calls
def _framework(st):
    from head_partitioned_distance_b200 import spa

    if st["op"] == "append":
        spa.paged_append(st["q"], st["k"], st["v"], st["k_pages"], st["v_pages"], st["page_table"], st["cu_q"],
                         st["kv_len"], st["q_weight"], st["k_weight"], st["table"], eps=EPS,
                         interleaved=st["neighbours"], out=st["out"])
        return {"q": st["out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if st["op"] == "attend":
        o, lse = spa.paged_attention(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["cu_q"],
                                     st["kv_len"], st["max_q"], scale=st["scale"], lo=st["lo"], hi=st["hi"],
                                     N=st["N"], out=st["out"], lse=st["lse"])
        return {"o": o, "lse": lse}
    if st["op"] == "norm_rope_fwd":
        q, k = spa.qk_norm_rope_forward(st["q"], st["k"], st["q_weight"], st["k_weight"], st["table"],
                                        positions=st["positions"], eps=EPS, interleaved=st["neighbours"])
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = spa.qk_norm_rope_backward(st["dq_out"], st["dk_out"], st["q"], st["k"], st["q_weight"],
                                                 st["k_weight"], st["table"], positions=st["positions"], eps=EPS,
                                                 interleaved=st["neighbours"])
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_norm_rope(x, w, cs, neighbours):
    """x / sqrt(mean x^2 + eps) * w, then pairs as complex numbers times e^{i angle}."""
    rot = 2 * cs.shape[-2]
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    z = y[..., :rot]
    z = z.unflatten(-1, (rot // 2, 2)) if neighbours else z.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.view_as_complex(cs.contiguous()))
    z = z if neighbours else z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), y[..., rot:]), -1)


def _exact_attend(case, st):
    new, kept = _lengths(case)
    size, G = case["page"], st["Hq"] // st["Hk"]
    out, lse = st["out"].double(), st["lse"].double()
    t0 = 0
    for s, (n, c) in enumerate(zip(new, kept)):
        pages = st["page_table"][s, :-(-c // size)].long()
        pos = torch.arange(c - n, c, device="cuda")
        for h in range(st["Hq"]):
            a, b = max(0, c - n - st["hi"][h] + 1), c - st["lo"][h]
            if b <= a:
                out[t0:t0 + n, h], lse[t0:t0 + n, h] = 0, -math.inf
                continue
            k = st["k_pages"][pages, h // G].reshape(-1, case["d"])[a:b].double()
            v = st["v_pages"][pages, h // G].reshape(-1, case["d"])[a:b].double()
            j = torch.arange(a, b, device="cuda")
            x = st["q"][t0:t0 + n, h].double() @ k.T * st["scale"]
            gap = pos[:, None] - j
            x = torch.where((gap >= st["lo"][h]) & (gap < st["hi"][h]), x, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[t0:t0 + n, h] = z
            out[t0:t0 + n, h] = torch.where(torch.isinf(z)[:, None], 0.0, torch.exp(x - z.clamp(min=-1e300)[:, None])) @ v
        t0 += n
    return {"o": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, st)
    table, nb = st["table"].double(), st["neighbours"]
    wq, wk = st["q_weight"].double(), st["k_weight"].double()
    if case["op"] == "append":
        new, kept = _lengths(case)
        out, kp, vp = st["out"].double(), st["k_pages"].double(), st["v_pages"].double()
        size, t0 = case["page"], 0
        for s, (n, c) in enumerate(zip(new, kept)):
            cs = table[c - n:c, None]
            out[t0:t0 + n] = _exact_norm_rope(st["q"][t0:t0 + n].double(), wq, cs, nb)
            k = _exact_norm_rope(st["k"][t0:t0 + n].double(), wk, cs, nb)
            pos = torch.arange(c - n, c, device="cuda")
            page = st["page_table"][s].long()[pos // size]
            kp[page, :, pos % size] = k
            vp[page, :, pos % size] = st["v"][t0:t0 + n].double()
            t0 += n
        return {"q": out, "k_pages": kp, "v_pages": vp}
    pos = torch.arange(case["N"], device="cuda")[None] if st["positions"] is None else st["positions"].long()
    cs = table[pos][:, None]
    if case["op"] == "norm_rope_fwd":
        return {"q": _exact_norm_rope(st["q"].double(), wq, cs, nb), "k": _exact_norm_rope(st["k"].double(), wk, cs, nb)}
    q, k = st["q"].double().requires_grad_(), st["k"].double().requires_grad_()
    wq.requires_grad_()
    wk.requires_grad_()
    dq, dwq = torch.autograd.grad(_exact_norm_rope(q, wq, cs, nb), (q, wq), st["dq_out"].double())
    dk, dwk = torch.autograd.grad(_exact_norm_rope(k, wk, cs, nb), (k, wk), st["dk_out"].double())
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}
