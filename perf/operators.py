"""Workloads of the full-attention layer that stands next to the KDA layers in a hybrid
model (no position encoding, grouped heads), each as one pass through an operator.

Three operators:

* prompt attention: causal softmax attention over whole prompts, dense or packed
  with cu_seqlens, forward ("fwd") and forward + backward ("train");
* tree attention ("tree"): queries of drafted tokens (a tree given by parent
  indices; one token is the ordinary decode step) over a paged key/value cache;
* cache pages: sequences forked, grown, copied on write, compacted and cut back
  ("beam": a beam-search step; "verify": a step of speculative decoding).

Layouts: q, o [B, T, Hq, d]; k, v [B, T, Hkv, d]; lse fp32 [B, T, Hq] (natural
logarithm); pages [P, Hkv, page, d]; block_table int32 [N, M] (-1: no page); lens
int32 [N]; refs int32 [P] (0: free).

With ``own`` false ``run`` computes with elementary torch operations in fp32; with
``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 1 << 28  # scores held at a time by the plain forms


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest prompt of the test presets: two heads, 64 tokens (latency)
        dict(name="fwd_tiny_fp32", op="fwd", dtype="fp32", B=1, T=64, Hq=2, Hkv=2, d=32),
        # a batch of short chat prompts, packed, odd lengths, small heads
        dict(name="fwd_packed_d64", op="fwd", dtype="bf16", seqs=24, lo=1, hi=700, Hq=16, Hkv=4, d=64),
        # the chunked-prefill workload's batch (B = 4, H = 16, T = 4096, d = 128)
        dict(name="fwd_batch_4096", op="fwd", dtype="bf16", B=4, T=4096, Hq=16, Hkv=16, d=128),
        # one long document, 32 query heads over 8 key/value heads
        dict(name="fwd_long_32768", op="fwd", dtype="bf16", B=1, T=32768, Hq=32, Hkv=8, d=128),
        # a training step's attention on packed documents of ragged lengths
        dict(name="train_packed_d128", op="train", dtype="bf16", seqs=9, lo=33, hi=1900, Hq=16, Hkv=4, d=128),
        # the same in full precision, with small heads and one odd length
        dict(name="train_fp32_d64", op="train", dtype="fp32", B=2, T=777, Hq=8, Hkv=4, d=64),
        # a long training sequence
        dict(name="train_long_16384", op="train", dtype="bf16", B=1, T=16384, Hq=32, Hkv=8, d=128),
        # decode of one short conversation: one token, latency
        dict(name="tree_one_short", op="tree", dtype="bf16", N=1, R=1, lo=900, hi=900, page=16, Hq=32, Hkv=8, d=128),
        # decode of a full batch (256 sequences), one token each
        dict(name="tree_decode_256", op="tree", dtype="bf16", N=256, R=1, lo=500, hi=8192, page=64, Hq=32, Hkv=8, d=128),
        # verification of drafted trees over long contexts
        dict(name="tree_verify_long", op="tree", dtype="bf16", N=16, R=24, ragged=False, lo=1024, hi=65536, page=64, Hq=32, Hkv=8, d=128),
        # a beam-search step: half of the beams go on, twice each, every one writes a token
        dict(name="beam_32x8", op="beam", dtype="bf16", N=256, W=8, lo=300, hi=2000, page=64, Hkv=8, d=128),
        # the cache's part of a speculative step: append the drafts, keep the accepted ones
        dict(name="verify_256x16", op="verify", dtype="bf16", N=256, R=16, lo=300, hi=2000, page=64, Hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, most):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * Hkv <= most])
    return Hkv * G, Hkv


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "train", "tree", "tree", "beam", "verify"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([32, 64, 128, 128])
    if op in ("fwd", "train"):
        Hq, Hkv = _heads(rng, 32)
        most = (16384 if op == "fwd" else 8192) // (4 if dtype == "fp32" else 1)
        case = dict(op=op, dtype=dtype, Hq=Hq, Hkv=Hkv, d=d)
        if rng.random() < 0.5:
            T = _log(rng, 1, most)
            return dict(case, B=rng.choice([1, 2, 3]) if T <= most // 4 else 1, T=T)
        hi = _log(rng, 2, most // 4)
        return dict(case, seqs=rng.randint(1, 12), lo=rng.randint(0, hi // 2), hi=hi)
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        Hq, Hkv = _heads(rng, 32)
        N, R = _log(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 64)])
        hi = _log(rng, 1, 16384 if N <= 16 else 4096)
        return dict(op=op, dtype=dtype, N=N, R=R, ragged=rng.random() < 0.3, lo=rng.randint(0, hi), hi=hi, page=page,
                    Hq=Hq, Hkv=Hkv, d=d)
    hi = _log(rng, 20, 3000)
    case = dict(op=op, dtype=dtype, lo=rng.randint(1, hi), hi=hi, page=page, Hkv=rng.choice([1, 2, 4, 8]), d=d)
    if op == "beam":
        W = rng.choice([2, 4, 8])
        return dict(case, N=W * _log(rng, 1, 16), W=W)
    return dict(case, N=_log(rng, 1, 128), R=rng.randint(1, 32))


def _lengths(case, n):
    """Lengths of the sequences: a property of the case, the same for every seed."""
    r = np.random.RandomState(17)
    x = r.randint(case["lo"], case["hi"] + 1, n)
    if x.sum() == 0:
        x[0] = case["hi"]
    return [int(v) for v in x]


def _spans(case):
    """(start, length) of every sequence of a prompt case, and the tokens in all."""
    if "seqs" not in case:
        return [(b * case["T"], case["T"]) for b in range(case["B"])], case["B"] * case["T"]
    lens = _lengths(case, case["seqs"])
    ends = np.cumsum(lens)
    return [(int(e - n), n) for e, n in zip(ends, lens)], int(ends[-1])


# ------------------------------------------------------------------ inputs
def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + tag)
    return g


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(case, P, g):
    shape = (P, case["Hkv"], case["page"], case["d"])
    return tuple(torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]]) for _ in range(2))


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _table(pages, M, g, P):
    """A table [N, M] whose row n holds pages[n] distinct random pages, and refs [P]."""
    pages = torch.as_tensor(pages, device="cuda")
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(M, device="cuda")
    used = at[None, :] < pages[:, None]
    first = torch.cumsum(pages, 0) - pages
    table = torch.where(used, perm[(first[:, None] + at[None, :]).clamp(max=P - 1)], -1).to(torch.int32)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[perm[:int(pages.sum())].long()] = 1
    return table.contiguous(), refs


def prepare(case, seed):
    g = _gen(seed, 1)
    s = dict(case=case)
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("fwd", "train"):
        spans, total = _spans(case)
        B, T = (1, total) if "seqs" in case else (case["B"], case["T"])
        s["spans"] = spans
        s["cu"] = _i32([0] + [a + n for a, n in spans]) if "seqs" in case else None
        s["q"] = _randn((B, T, case["Hq"], case["d"]), dt, g)
        s["k"] = _randn((B, T, case["Hkv"], case["d"]), dt, g)
        s["v"] = _randn((B, T, case["Hkv"], case["d"]), dt, g)
        if case["op"] == "train":
            s["dO"] = _randn((B, T, case["Hq"], case["d"]), dt, g)
        s["scale"] = case["d"] ** -0.5
        return s
    N, page = case["N"], case["page"]
    if case["op"] == "tree":
        R = case["R"]
        ctx = _lengths(case, N)
        pages = [-(-(c + R) // page) for c in ctx]
        P = sum(pages) + 3
        s["table"], _ = _table(pages, max(pages), g, P)
        s["ctx"] = _i32(ctx)
        s["k_pages"], s["v_pages"] = _pool(case, P, g)
        s["q"] = _randn((N, R, case["Hq"], case["d"]), dt, g)
        # parents: a random tree; each token's parent is the cache's end or an earlier draft
        u = torch.rand((N, R), generator=g, device="cuda")
        at = torch.arange(R, device="cuda")
        s["parents"] = (torch.floor(u * (at + 1)) - 1).to(torch.int32)
        if case.get("ragged"):  # row n of the batch has drafted only 1 + n % R tokens
            s["parents"].masked_fill_(at[None, :] > torch.arange(N, device="cuda")[:, None] % R, -2)
        s["scale"] = case["d"] ** -0.5
        return s
    lens = _lengths(case, N)
    if case["op"] == "beam":
        # no length ends on a page's end, so every shared last page is copied once
        W = case["W"]
        lens = [n + 1 if n % page == 0 else n for n in lens]
        pages = [-(-n // page) for n in lens]
        M, P = max(pages) + 1, sum(pages) + 2 * N
        # half of a group's beams, each taken twice, in a random order
        order = torch.argsort(torch.rand((N // W, W), generator=g, device="cuda"), 1)
        pick = torch.argsort(torch.rand((N // W, W), generator=g, device="cuda"), 1)
        parents = torch.gather(order, 1, pick // 2 if W > 1 else pick)
        s["parents"] = (parents + W * torch.arange(N // W, device="cuda")[:, None]).reshape(-1).to(torch.int32)
        s["add"] = torch.ones(N, dtype=torch.int32, device="cuda")
    else:
        R = case["R"]
        pages = [-(-n // page) for n in lens]
        M, P = -(-(max(lens) + R) // page), sum(-(-(n + R) // page) for n in lens) + N
        s["add"] = torch.full((N,), R, dtype=torch.int32, device="cuda")
        s["k"] = _randn((N, R, case["Hkv"], case["d"]), dt, g)
        s["v"] = _randn((N, R, case["Hkv"], case["d"]), dt, g)
        # row n keeps 1 + n % R of its drafts: an increasing random choice
        keep = 1 + torch.arange(N, device="cuda") % R
        rank = torch.argsort(torch.rand((N, R), generator=g, device="cuda"), 1)
        at = torch.arange(R, device="cuda")[None, :].expand(N, R)
        chosen = torch.where(at < keep[:, None], rank, R).sort(1).values
        s["path"] = torch.where(chosen < R, chosen, -1).to(torch.int32).contiguous()
    s["table"], s["refs"] = _table(pages, M, g, P)
    s["lens"] = _i32(lens)
    s["k_pages"], s["v_pages"] = _pool(case, P, g)
    return s


# ------------------------------------------------------------------ plain forms
def _rows_at_once(heads, keys):
    return max(16, BLOCK // max(1, heads * keys))


def _plain_seq_fwd(q, k, v, scale):
    """Causal attention of one sequence in fp32: q [L, Hq, d], k, v [L, Hkv, d]."""
    L, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    qh = q.reshape(L, Hkv, G, d).permute(1, 2, 0, 3)
    kh, vh = k.permute(1, 2, 0), v.permute(1, 0, 2)
    o = torch.empty_like(qh)
    lse = torch.empty((Hkv, G, L), dtype=torch.float32, device=q.device)
    rows = _rows_at_once(Hq, L)
    for a in range(0, L, rows):
        b = min(L, a + rows)
        s = (qh[:, :, a:b].reshape(Hkv, G * (b - a), d) @ kh[:, :, :b]).mul_(scale).view(Hkv, G, b - a, b)
        later = torch.arange(b, device=q.device)[None, :] > torch.arange(a, b, device=q.device)[:, None]
        s.masked_fill_(later, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = s.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o[:, :, a:b] = (p.view(Hkv, G * (b - a), b) @ vh[:, :b]).view(Hkv, G, b - a, d) / l
        lse[:, :, a:b] = (m + l.log()).squeeze(-1)
    return o.permute(2, 0, 1, 3).reshape(L, Hq, d), lse.permute(2, 0, 1).reshape(L, Hq)


def _plain_seq_bwd(q, k, v, o, lse, dO, scale):
    """Gradients of <dO, o> for one sequence in fp32."""
    L, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    by_head = lambda x: x.reshape(L, Hkv, G, -1).permute(1, 2, 0, 3)  # noqa: E731
    qh, gh = by_head(q), by_head(dO)
    kh, vh = k.permute(1, 0, 2), v.permute(1, 0, 2)
    lh = by_head(lse)
    delta = by_head((dO * o).sum(-1))
    dq = torch.empty_like(qh)
    dk, dv = torch.zeros_like(kh), torch.zeros_like(vh)
    rows = _rows_at_once(2 * Hq, L)
    for a in range(0, L, rows):
        b = min(L, a + rows)
        flat = lambda x: x[:, :, a:b].reshape(Hkv, G * (b - a), -1)  # noqa: E731
        later = torch.arange(b, device=q.device)[None, :] > torch.arange(a, b, device=q.device)[:, None]
        s = (flat(qh) @ kh[:, :b].transpose(1, 2)).mul_(scale).view(Hkv, G, b - a, b).masked_fill_(later, -math.inf)
        p = s.view(Hkv, G * (b - a), b).sub_(flat(lh)).exp_()
        dv[:, :b] += p.transpose(1, 2) @ flat(gh)
        ds = (flat(gh) @ vh[:, :b].transpose(1, 2)).sub_(flat(delta)).mul_(p).mul_(scale)
        dq[:, :, a:b] = (ds @ kh[:, :b]).view(Hkv, G, b - a, d)
        dk[:, :b] += ds.transpose(1, 2) @ flat(qh)
    back = lambda x: x.permute(2, 0, 1, 3).reshape(L, Hq, d)  # noqa: E731
    return back(dq), dk.permute(1, 0, 2), dv.permute(1, 0, 2)


def _plain_prompt(s, train):
    dt = s["q"].dtype
    tok = lambda x: x.reshape((-1,) + x.shape[2:])  # noqa: E731
    q, k, v = (tok(s[n]).float() for n in "qkv")
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    grads = [torch.empty_like(x) for x in (q, k, v)] if train else []
    g = tok(s["dO"]).float() if train else None
    for a, n in s["spans"]:
        w = slice(a, a + n)
        if n:
            o[w], lse[w] = _plain_seq_fwd(q[w], k[w], v[w], s["scale"])
            if train:
                for x, y in zip(grads, _plain_seq_bwd(q[w], k[w], v[w], o[w], lse[w], g[w], s["scale"])):
                    x[w] = y
    out = dict(o=o.to(dt).view_as(s["q"]), lse=lse.view(s["q"].shape[:3]))
    for name, x in zip("qkv", grads):
        out["d" + name] = x.to(dt).view_as(s[name])
    return out


def _tree_mask(parents):
    """visible [N, R, R]: token i attends to draft j. A parent that is neither -1
    nor an earlier draft makes its token and what hangs from it absent."""
    N, R = parents.shape
    at = torch.arange(R, device=parents.device)
    up = (parents[:, :, None] == at) & (at[None, :] < at[:, None])  # a parent comes before its child
    bad = (parents < -1) | (parents >= at)
    seen = up | torch.eye(R, dtype=torch.bool, device=parents.device)
    for _ in range(max(1, (R - 1).bit_length())):
        seen = (seen.float() @ seen.float()) > 0
    absent = (seen & bad[:, None, :]).any(-1)
    return seen & ~absent[:, :, None], absent


def _plain_tree(s):
    case = s["case"]
    q, table, ctx = s["q"], s["table"], s["ctx"]
    N, R, Hq, d = q.shape
    Hkv, page = case["Hkv"], case["page"]
    M = table.shape[1]
    L = M * page
    kv = [x[table.clamp(min=0).long()].float().permute(0, 2, 1, 3, 4).reshape(N, Hkv, L, d)
          for x in (s["k_pages"], s["v_pages"])]
    G = Hq // Hkv
    visible, absent = _tree_mask(s["parents"])
    pos = torch.arange(L, device=q.device)[None, :] - ctx[:, None]  # [N, L]: < 0 cached, 0..R-1 a draft
    draft = torch.gather(visible, 2, pos.clamp(0, R - 1)[:, None, :].expand(N, R, L))
    see = (pos < 0)[:, None, :] | (draft & (pos >= 0)[:, None, :] & (pos < R)[:, None, :])
    see = see & ~absent[:, :, None]
    qh = q.float().reshape(N, R, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(N, Hkv, R * G, d)
    sc = (qh @ kv[0].transpose(2, 3)).mul_(s["scale"]).view(N, Hkv, R, G, L)
    sc.masked_fill_(~see[:, None, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = (sc - m.clamp(min=-1e38)).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(N, Hkv, R * G, L) @ kv[1]).view(N, Hkv, R, G, d) / torch.where(l > 0, l, 1.0)
    lse = (m + l.log()).squeeze(-1)
    return dict(o=o.permute(0, 2, 1, 3, 4).reshape(N, R, Hq, d).to(q.dtype),
                lse=lse.permute(0, 2, 1, 3).reshape(N, R, Hq))


def _plain_fork(refs, table, lens, parents):
    """Row n becomes a copy of row parents[n]; the old rows' holds on their pages end."""
    new, new_lens = table[parents.long()], lens[parents.long()]
    count = lambda t: torch.bincount(t[t >= 0].long(), minlength=refs.numel())  # noqa: E731
    return (refs + count(new) - count(table)).to(torch.int32), new, new_lens


def _plain_reserve(refs, table, lens, add, page):
    """Room for add[n] tokens more in row n: the lowest free pages, row after row; a
    last page that is partly filled and shared is replaced by a copy first."""
    N, M = table.shape
    at = torch.arange(M, device=table.device)
    have, want = (lens + page - 1) // page, (lens + add + page - 1) // page
    last = (have - 1).clamp(min=0)
    tail = table.gather(1, last[:, None].long()).squeeze(1)
    partly = (add > 0) & (lens % page != 0)
    same = (tail[:, None] == tail[None, :]) & partly[:, None] & partly[None, :]
    before = torch.tril(same, -1).sum(1)
    cow = partly & (refs[tail.clamp(min=0).long()] - before > 1)
    count = cow + want - have
    first = torch.cumsum(count, 0) - count
    free = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)  # free pages first, in order
    copies = torch.where(cow[:, None], torch.stack([tail, free[first.clamp(max=free.numel() - 1)]], 1), -1)
    fresh = (at >= have[:, None]) & (at < want[:, None])
    where = (first + cow)[:, None] + at - have[:, None]
    out = torch.where(fresh, free[where.clamp(0, free.numel() - 1)], table)
    out = torch.where(cow[:, None] & (at == last[:, None]), copies[:, 1:], out)
    gone = torch.bincount(torch.where(cow, tail, refs.numel()).long(), minlength=refs.numel() + 1)[:-1]
    rank = torch.arange(refs.numel(), device=refs.device)
    new = torch.zeros_like(refs).scatter_(0, free.long(), (rank < count.sum()).to(torch.int32))
    return (refs - gone + new).to(torch.int32), out.to(torch.int32), (lens + add).to(torch.int32), copies.to(torch.int32)


def _plain_copy(pool, copies):
    real = copies[:, 0] >= 0
    src, dst = copies[:, 0].clamp(min=0).long(), copies[:, 1].clamp(min=0).long()
    # a pair that copies nothing copies the pool's first page onto itself, unless that page is a destination
    spare = torch.where(real.any(), dst[real.to(torch.int8).argmax()], 0)
    src = torch.where(real, src, src[real.to(torch.int8).argmax()])
    pool[torch.where(real, dst, spare)] = pool[src]


def _plain_append(pool, table, at, x):
    N, R = x.shape[:2]
    page = pool.shape[2]
    pos = at[:, None] + torch.arange(R, device=x.device)
    pool[table.gather(1, (pos // page).long()).long(), :, (pos % page).long()] = x


def _plain_compact(pool, table, ctx, path):
    page, M = pool.shape[2], table.shape[1]
    kept = path >= 0
    old = ctx[:, None] + torch.where(kept, path, 0)
    new = ctx[:, None] + torch.arange(path.shape[1], device=path.device)
    place = lambda pos: (table.gather(1, (pos // page).clamp(max=M - 1).long()).long(), (pos % page).long())  # noqa: E731
    (sp, so), (dp, do) = place(old), place(new)
    sp, so = torch.where(kept, sp, dp), torch.where(kept, so, do)
    pool[dp, :, do] = pool[sp, :, so]
    return (ctx + kept.sum(1)).to(torch.int32)


def _plain_release(refs, table, lens, new_lens, page):
    lens = torch.minimum(lens, new_lens)
    over = torch.arange(table.shape[1], device=table.device) >= ((lens + page - 1) // page)[:, None]
    gone = torch.bincount(table[over & (table >= 0)].long(), minlength=refs.numel())
    return (refs - gone).to(torch.int32), torch.where(over, -1, table).to(torch.int32), lens.to(torch.int32)


# ------------------------------------------------------------------ passes
def _lib():
    import gated_delta_rule_132_b200 as kda
    return kda


def _run_prompt(s):
    train = s["case"]["op"] == "train"
    if not own:
        return _plain_prompt(s, train)
    kda = _lib()
    o, lse = kda.kda_attn_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], scale=s["scale"])
    out = dict(o=o, lse=lse)
    if train:
        out.update(kda.kda_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["dO"], cu_seqlens=s["cu"], scale=s["scale"]))
    return out


def _run_tree(s):
    if not own:
        return _plain_tree(s)
    o, lse = _lib().kda_attn_tree(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"],
                                  parents=s["parents"], scale=s["scale"])
    return dict(o=o, lse=lse)


def _run_beam(s):
    page, kp, vp = s["case"]["page"], s["k_pages"], s["v_pages"]
    refs = s["refs"].clone()
    if own:
        kda = _lib()
        table, lens = kda.kda_cache_fork(refs, s["table"], s["lens"], s["parents"])
        copies, status = kda.kda_cache_reserve(refs, table, lens, s["add"], page)
        kda.kda_cache_copy_pages(kp, vp, copies)
    else:
        refs, table, lens = _plain_fork(refs, s["table"], s["lens"], s["parents"])
        refs, table, lens, copies = _plain_reserve(refs, table, lens, s["add"], page)
        _plain_copy(kp, copies)
        _plain_copy(vp, copies)
        status = torch.zeros(1, dtype=torch.int32, device=refs.device)
    return dict(refs=refs, table=table, lens=lens, copies=copies, status=status, k_pages=kp, v_pages=vp)


def _run_verify(s):
    page, kp, vp, ctx = s["case"]["page"], s["k_pages"], s["v_pages"], s["lens"]
    refs, table, lens = s["refs"].clone(), s["table"].clone(), s["lens"].clone()
    if own:
        kda = _lib()
        copies, status = kda.kda_cache_reserve(refs, table, lens, s["add"], page)
        kda.kda_cache_append(kp, vp, table, ctx, s["k"], s["v"])
        kept = kda.kda_cache_compact(kp, vp, table, ctx, s["path"])
        kda.kda_cache_release(refs, table, lens, kept, page)
    else:
        refs, table, lens, copies = _plain_reserve(refs, table, lens, s["add"], page)
        _plain_append(kp, table, ctx, s["k"])
        _plain_append(vp, table, ctx, s["v"])
        kept = _plain_compact(kp, table, ctx, s["path"])
        _plain_compact(vp, table, ctx, s["path"])
        refs, table, lens = _plain_release(refs, table, lens, kept, page)
        status = torch.zeros(1, dtype=torch.int32, device=refs.device)
    return dict(refs=refs, table=table, lens=lens, copies=copies, status=status, k_pages=kp, v_pages=vp)


RUNS = {"fwd": _run_prompt, "train": _run_prompt, "tree": _run_tree, "beam": _run_beam, "verify": _run_verify}


def run(state):
    return RUNS[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] in ("fwd", "train"):
        spans, total = _spans(case)
        Hq = case["Hq"]
        pairs = sum(n * (n + 1) // 2 for _, n in spans)
        size = total * (2 * Hq + 2 * Hkv) * d * es + total * Hq * 4
        if case["op"] == "train":  # dO in, dq, dk, dv out; five products next to the forward's two
            size += total * (2 * Hq + 2 * Hkv) * d * es
        return dict(bytes=size, flops=(14 if case["op"] == "train" else 4) * d * Hq * pairs)
    N, page = case["N"], case["page"]
    lens = _lengths(case, N)
    if case["op"] == "tree":
        R, Hq = case["R"], case["Hq"]
        table = 4 * sum(-(-(n + R) // page) for n in lens)
        real = [1 + i % R if case.get("ragged") else R for i in range(N)]
        size = sum(n + r for n, r in zip(lens, real)) * 2 * Hkv * d * es + 4 * N + table
        size += sum(real) * Hq * d * es + N * R * (Hq * d * es + 4 * Hq + 4)
        return dict(bytes=size, flops=4 * d * Hq * sum(r * (n + r) for n, r in zip(lens, real)))
    row = Hkv * d * es
    pages = sum(-(-n // page) for n in lens)
    if case["op"] == "beam":
        lens = [n + 1 if n % page == 0 else n for n in lens]
        pages = sum(-(-n // page) for n in lens)
        M, P = -(-max(lens) // page) + 1, pages + 2 * N
        copies = N // 2  # of k and of v, each read and written
        return dict(bytes=copies * 2 * 2 * page * row + 4 * (2 * P + 2 * N * M + 6 * N), flops=0)
    R = case["R"]
    kept = sum(1 + n % R for n in range(N))
    P = sum(-(-(n + R) // page) for n in lens) + N
    M = -(-(max(lens) + R) // page)
    # the drafts in and into their pages, the kept rows read and written once more, the tables
    return dict(bytes=2 * row * (2 * N * R + 2 * kept) + 4 * (2 * P + 2 * N * M + N * R + 6 * N), flops=0)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_head(q, k, v, scale, grad=None):
    """One head of one sequence, [L, d] each, in fp64: softmax by the definition, the
    gradients by reverse mode; query rows in slices."""
    L = q.shape[0]
    o, lse = torch.empty_like(q), torch.empty(L, dtype=q.dtype, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    rows = max(1, (1 << 28) // max(L, 1))
    for a in range(0, L, rows):
        b = min(L, a + rows)
        x = [t.clone().requires_grad_(grad is not None) for t in (q[a:b], k[:b], v[:b])]
        s = torch.matmul(x[0] * scale, x[1].t())
        s = s + torch.full((b - a, b), -math.inf, dtype=q.dtype, device=q.device).triu_(a + 1)
        z = torch.logsumexp(s, 1)
        y = torch.matmul(torch.exp(s - z[:, None]), x[2])
        o[a:b], lse[a:b] = y.detach(), z.detach()
        if grad is not None:
            gq, gk, gv = torch.autograd.grad(y, x, grad[a:b])
            dq[a:b] = gq
            dk[:b] += gk
            dv[:b] += gv
    return o, lse, dq, dk, dv


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("beam", "verify"):
        return None  # pages are moved, not computed
    G = case["Hq"] // case["Hkv"]
    if case["op"] == "tree":
        return _exact_tree(s, G)
    train = case["op"] == "train"
    tok = lambda x: x.reshape((-1,) + x.shape[2:])  # noqa: E731
    out = {n: torch.zeros(tok(s[n]).shape, dtype=torch.float64, device="cuda") for n in "qkv"}
    o = torch.zeros_like(out["q"])
    lse = torch.zeros(o.shape[:2], dtype=torch.float64, device="cuda")
    for a, n in s["spans"]:
        w = slice(a, a + n)
        for h in range(case["Hq"] if n else 0):
            x = [tok(s[name])[w, head].double() for name, head in (("q", h), ("k", h // G), ("v", h // G))]
            r = _exact_head(*x, s["scale"], tok(s["dO"])[w, h].double() if train else None)
            o[w, h], lse[w, h] = r[0], r[1]
            out["q"][w, h] = r[2]
            out["k"][w, h // G] += r[3]
            out["v"][w, h // G] += r[4]
    res = dict(o=o.view(s["q"].shape), lse=lse.view(s["q"].shape[:3]))
    if train:
        res.update({"d" + n: out[n].view(s[n].shape) for n in "qkv"})
    return res


def _exact_tree(s, G):
    q, table, ctx = s["q"], s["table"].cpu().numpy(), s["ctx"].cpu().numpy()
    parents = s["parents"].cpu().numpy()
    N, R, Hq, d = q.shape
    page = s["case"]["page"]
    o = torch.zeros((N, R, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((N, R, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for n in range(N):
        c = int(ctx[n])
        rows = torch.as_tensor(table[n][:-(-(c + R) // page)].astype(np.int64), device="cuda")
        k, v = (x[rows].double().permute(1, 0, 2, 3).reshape(x.shape[1], -1, d)[:, :c + R] for x in (s["k_pages"], s["v_pages"]))
        see = np.zeros((R, R), dtype=bool)  # a token sees itself and what its parent sees
        real = [i for i in range(R) if parents[n, i] >= -1]  # a tree's absent tokens have no children here
        for i in real:
            see[i] = see[parents[n, i]] if parents[n, i] >= 0 else False
            see[i, i] = True
        bias = torch.zeros((R, c + R), dtype=torch.float64, device="cuda")
        bias[:, c:] = torch.as_tensor(np.where(see, 0.0, -math.inf), device="cuda")
        for h in range(k.shape[0]):
            x = q[n, real, h * G:(h + 1) * G].double().permute(1, 0, 2) * s["scale"]
            sc = torch.matmul(x, k[h].t()) + bias[real]
            z = torch.logsumexp(sc, -1)
            lse[n, real, h * G:(h + 1) * G] = z.t()
            o[n, real, h * G:(h + 1) * G] = torch.matmul(torch.exp(sc - z[..., None]), v[h]).permute(1, 0, 2)
    return dict(o=o, lse=lse)
