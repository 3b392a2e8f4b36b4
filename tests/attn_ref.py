"""Plain fp64 forms of the full-attention calls, with bounds on what rounding may do to
each result, and a list-based model of the cache's pages.

Rounding model behind the bounds (u: half a step of the results' type; e = 2^-24, fp32):
* a score is a sum of d products in fp32, off by at most E = 2 d e sum|q_i k_i| scale
  (twice d e: the accumulation need not round to nearest); so a probability is off by a
  factor within e^(+-2E), and within (2 n + 64) e more by the exponential, the running
  rescales and the sum over n keys;
* with 16-bit inputs each probability (and score gradient) is rounded once as an operand;
* a result is a sum over n terms in fp32 (2 n e of the sum of magnitudes), rounded once;
* fp32 ends at 2^-126: a smaller probability may become 0. A result is at most 2^18 such
  terms, each times factors of at most 2^12 here, so this can shift it by TINY = 2^-96.
"""
import torch

E32 = 2.0 ** -24
TINY = 2.0 ** -96


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def operand_step(dtype):
    """Half a step of the probabilities' type in the products: none beyond fp32's for fp32."""
    return half_step(torch.bfloat16) if dtype == torch.bfloat16 else E32


def _scores(q, k, see, scale):
    """q [R, d], k [C, d], see [R, C] -> masked scores, and the bound on their error."""
    s = (q @ k.t()) * scale
    err = 2 * q.shape[1] * E32 * scale * (q.abs() @ k.abs().t())
    # keys that are not seen take no part, whatever they hold
    return torch.where(see, s, -torch.inf), torch.where(see, err, 0.0)


def _weighted(w, x, see):
    """sum_c w_rc x_c over the seen keys only (0 * inf stays out)."""
    if torch.isfinite(x).all():
        return w @ x
    out = torch.zeros(w.shape[0], x.shape[1], dtype=w.dtype, device=w.device)
    for r in range(w.shape[0]):
        out[r] = w[r][see[r]] @ x[see[r]]
    return out


def attend(q, k, v, see, scale, dtype):
    """One head: softmax attention in fp64 of q [R, d] over k, v [C, d] where see [R, C].
    Returns o, lse and their bounds; rows that see nothing give 0 and -inf."""
    s, serr = _scores(q, k, see, scale)
    m = s.amax(1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    w = torch.exp(s - m)
    l = w.sum(1, keepdim=True)
    lse = (m + torch.log(l)).squeeze(1)
    p = torch.where(see, w / torch.where(l > 0, l, 1.0), 0.0)
    o, mag = _weighted(p, v, see), _weighted(p, v.abs(), see)
    n = see.sum(1, keepdim=True)
    e = serr.amax(1, keepdim=True)
    rel = 2 * e + (4 * n + 64) * E32
    o_tol = half_step(dtype) * o.abs() + (2 * operand_step(dtype) + 2 * rel) * mag
    lse_tol = (e + (2 * n + 64) * E32).squeeze(1) + 4 * E32 * (m.abs().squeeze(1) + lse.abs())
    return o, lse, o_tol, lse_tol


def attn_fwd(q, k, v, spans, scale):
    """q [T, Hq, d], k, v [T, Hkv, d] (packed), spans [(start, length)]: fp64 results and bounds."""
    dtype, G = q.dtype, q.shape[1] // k.shape[1]
    q, k, v = (x.double() for x in (q, k, v))
    o, o_tol = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    lse_tol = torch.zeros_like(lse)
    for a, n in spans:
        see = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        w = slice(a, a + n)
        for h in range(q.shape[1] if n else 0):
            o[w, h], lse[w, h], o_tol[w, h], lse_tol[w, h] = attend(
                q[w, h], k[w, h // G], v[w, h // G], see, scale, dtype)
    return o, lse, o_tol, lse_tol


def attn_bwd(q, k, v, o, lse, dO, spans, scale):
    """Gradients of <dO, o> by their formulas in fp64, given o and lse; and bounds."""
    dtype, G = q.dtype, q.shape[1] // k.shape[1]
    u, w_step = half_step(dtype), operand_step(dtype)
    q, k, v, o, lse, dO = (x.double() for x in (q, k, v, o, lse, dO))
    d = q.shape[2]
    out = [torch.zeros_like(x) for x in (q, k, v)]
    tol = [torch.zeros_like(x) for x in (q, k, v)]
    for a, n in spans:
        see = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        w = slice(a, a + n)
        for h in range(q.shape[1] if n else 0):
            qh, gh, kh, vh = q[w, h], dO[w, h], k[w, h // G], v[w, h // G]
            s, serr = _scores(qh, kh, see, scale)
            z = lse[w, h][:, None]
            p = torch.where(see, torch.exp(s - z), 0.0)
            delta = (gh * o[w, h]).sum(1, keepdim=True)
            dp = gh @ vh.t()
            ds = p * (dp - delta) * scale
            # errors: p relative, dp and delta absolute
            prel = 2 * serr + (4 * z.abs() + 64) * E32
            dabs = 2 * d * E32 * (gh.abs() @ vh.abs().t() + (gh * o[w, h]).abs().sum(1, keepdim=True))
            eds = scale * p * ((dp.abs() + delta.abs()) * prel + dabs) + 16 * E32 * ds.abs()
            sums = 2 * n * E32
            for i, (part, mag) in enumerate((
                    (ds @ kh, ((w_step + sums) * ds.abs() + eds) @ kh.abs()),
                    (ds.t() @ qh, ((w_step + sums * G) * ds.abs() + eds).t() @ qh.abs()),
                    (p.t() @ gh, ((w_step + sums * G + prel) * p).t() @ gh.abs()))):
                at = h if i == 0 else h // G
                out[i][w, at] += part
                tol[i][w, at] += mag
    # the bounds' own second-order terms are within a hundredth of them
    return out, [u * x.abs() + 1.01 * t for x, t in zip(out, tol)]


def tree_see(parents, ctx, R, M, page, table, P):
    """Positions [0, ctx + R) that each draft of one sequence sees, by walking up the tree."""
    C = min(ctx + R, M * page)
    see = torch.zeros(R, C, dtype=torch.bool)
    for i in range(R):
        j, chain = i, []
        while True:
            chain.append(j)
            up = j - 1 if parents is None else int(parents[j])
            if up == -1:
                break
            if up < -1 or up >= j:
                chain = None
                break
            j = up
        if chain is None:
            continue
        see[i, :min(ctx, C)] = True
        for j in chain:
            if ctx + j < C:
                see[i, ctx + j] = True
    for c in range(0, C, page):
        if not 0 <= int(table[c // page]) < P:
            see[:, c:c + page] = False
    return see


def attn_tree(q, k_pages, v_pages, table, ctx, parents, scale):
    """fp64 tree attention over a paged cache: o, lse and their bounds."""
    N, R, Hq, d = q.shape
    P, Hkv, page, _ = k_pages.shape
    M, G, dev = table.shape[1], Hq // Hkv, q.device
    o = torch.zeros((N, R, Hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((N, R, Hq), -torch.inf, dtype=torch.float64, device=dev)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    for n in range(N):
        c0 = min(max(int(ctx[n]), 0), M * page)
        see = tree_see(None if parents is None else parents[n].tolist(), c0, R, M, page,
                       table[n].tolist(), P).to(dev)
        C = see.shape[1]
        ids = table[n, :-(-C // page)].long()
        ids = torch.where((ids >= 0) & (ids < P), ids, 0)
        k, v = (x[ids].transpose(0, 1).reshape(Hkv, -1, d)[:, :C].double() for x in (k_pages, v_pages))
        for h in range(Hq if C else 0):
            o[n, :, h], lse[n, :, h], o_tol[n, :, h], lse_tol[n, :, h] = attend(
                q[n, :, h].double(), k[h // G], v[h // G], see, scale, q.dtype)
    return o, lse, o_tol, lse_tol


def close(got, want, tol):
    """Every element within its bound; infinities and NaN in the same places."""
    got, want = got.double(), want.double()
    same = torch.where(torch.isfinite(want), (got - want).abs() <= tol + TINY,
                       (got == want) | (got.isnan() & want.isnan()))
    if bool(same.all()):
        return
    bad = (~same).nonzero()
    i = tuple(bad[0].tolist())
    raise AssertionError(f"{bad.shape[0]} of {got.numel()} off, first at {i}: {got[i].item()} "
                         f"for {want[i].item()}, bound {float(tol[i])}")


class Pages:
    """The cache's tables as Python lists."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.page = list(refs), page
        self.table, self.lens = [list(r) for r in table], list(lens)
        self.M = len(self.table[0])

    def count(self, n):
        return -(-n // self.page)

    def _hold(self, row, by):
        for p in row:
            if 0 <= p < len(self.refs):
                self.refs[p] += by

    def fork(self, parents):
        old, lens = self.table, self.lens
        ok = [0 <= a < len(old) for a in parents]
        self.table = [list(old[a]) if g else [-1] * self.M for a, g in zip(parents, ok)]
        self.lens = [lens[a] if g else 0 for a, g in zip(parents, ok)]
        for r in self.table:
            self._hold(r, 1)
        for r in old:
            self._hold(r, -1)

    def reserve(self, add):
        before = (list(self.refs), [list(r) for r in self.table], list(self.lens))
        none = [[-1, -1] for _ in add]
        for n, a in enumerate(add):
            if self.count(self.lens[n] + max(a, 0)) > self.M:
                return none, -1 - n
        copies, missing = [], 0
        # pages free at the call's beginning: one that a copy lets go of waits for the next call
        free = [p for p, r in enumerate(self.refs) if r == 0]

        def take():
            nonlocal missing
            if not free:
                missing += 1
                return None
            self.refs[free[0]] = 1
            return free.pop(0)

        for n, a in enumerate(add):
            a, have = max(a, 0), self.count(self.lens[n])
            pair = [-1, -1]
            if a and self.lens[n] % self.page:
                tail = self.table[n][have - 1]
                if 0 <= tail < len(self.refs) and self.refs[tail] > 1:
                    to = take()
                    pair = [tail, to]
                    self.refs[tail] -= 1
                    self.table[n][have - 1] = to
            for j in range(have, self.count(self.lens[n] + a)):
                self.table[n][j] = take()
            self.lens[n] += a
            copies.append(pair)
        if missing:
            self.refs, self.table, self.lens = before
            return none, missing
        return copies, 0

    def release(self, new_lens):
        for n, want in enumerate(new_lens):
            self.lens[n] = max(0, min(self.lens[n], want))
            keep = self.count(self.lens[n])
            self._hold(self.table[n][keep:], -1)
            self.table[n][keep:] = [-1] * (self.M - keep)
