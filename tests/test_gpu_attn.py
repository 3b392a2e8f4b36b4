"""Prompt attention and its gradients against plain fp64 forms (bounds derived in attn_ref)."""
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def api():
    from gated_delta_rule_132_b200 import attn
    return attn


def inputs(seed, T, Hq, Hkv, d, dtype, B=1, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda h: (torch.randn(B, T, h, d, generator=g, device="cuda") * spread).to(dtype)  # noqa: E731
    return mk(Hq), mk(Hkv), mk(Hkv), mk(Hq)


def spans_of(lens):
    out, a = [], 0
    for n in lens:
        out.append((a, n))
        a += n
    return out


def cu_of(lens):
    return torch.tensor([0] + [a + n for a, n in spans_of(lens)], dtype=torch.int32, device="cuda")


def check(q, k, v, dO, spans, cu, scale=None):
    """Forward and gradients of one call against the plain forms."""
    attn = api()
    s = q.shape[-1] ** -0.5 if scale is None else scale
    o, lse = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, scale=scale)
    flat = [x.reshape((-1,) + x.shape[2:]) for x in (q, k, v, dO)]
    ro, rl, to, tl = R.attn_fwd(*flat[:3], spans, s)
    R.close(o.view_as(flat[0]), ro, to)
    R.close(lse.view(rl.shape), rl, tl)
    g = attn.kda_attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu, scale=scale)
    want, tol = R.attn_bwd(*flat[:3], o.view_as(flat[0]), lse.view(rl.shape), flat[3], spans, s)
    for name, w, t in zip(("dq", "dk", "dv"), want, tol):
        assert g[name].dtype == q.dtype
        R.close(g[name].view_as(w), w, t)
    return o, lse, g


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400])
def test_lengths(T, d, dtype):
    q, k, v, dO = inputs(T, T, 4, 2, d, DT[dtype])
    check(q, k, v, dO, [(0, T)], None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (3, 1, 128), (6, 3, 32), (8, 8, 64), (5, 1, 128), (16, 2, 64)])
def test_heads_and_batch(Hq, Hkv, d, dtype):
    B, T = 3, 150
    q, k, v, dO = inputs(7, T, Hq, Hkv, d, DT[dtype], B)
    check(q, k, v, dO, spans_of([T] * B), None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[1], [0, 5, 0, 0, 300, 1], [128, 256, 64, 1, 127], [700, 13, 13, 260], [1] * 40])
@pytest.mark.parametrize("d", [64, 128])
def test_packed(lens, d, dtype):
    q, k, v, dO = inputs(11, sum(lens), 4, 2, d, DT[dtype])
    check(q, k, v, dO, spans_of(lens), cu_of(lens))


@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences_keep_their_order(d):
    """More sequences than are ranked by length."""
    lens = [(i * 7) % 5 for i in range(2100)]
    q, k, v, dO = inputs(12, sum(lens), 2, 1, d, torch.bfloat16)
    attn = api()
    o, lse = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu_of(lens))
    ro, rl, to, tl = R.attn_fwd(q[0], k[0], v[0], spans_of(lens), d ** -0.5)
    R.close(o[0], ro, to)
    R.close(lse[0], rl, tl)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("count,longest", [(300, 200), (60, 700), (2100, 9)])
def test_many_packed(count, longest, dtype):
    """More tiles than CTAs, of all sizes: every one is worked on once, in either order."""
    g = torch.Generator().manual_seed(count)
    lens = torch.randint(0, longest + 1, (count,), generator=g).tolist()
    q, k, v, dO = inputs(27, sum(lens), 3, 1, 64, DT[dtype])
    check(q, k, v, dO, spans_of(lens), cu_of(lens))


def test_starved_kernels_report_their_wait():
    """A loading warp that copies nothing: the waits run out, the status word says so, and the
    next call on the workspace is clean. Nothing is in flight meanwhile."""
    from gated_delta_rule_132_b200 import kda
    attn = api()
    for Hq, Hkv, T in ((2, 1, 300), (4, 1, 100)):  # a key tile's CTA alone, and a cluster
        q, k, v, dO = inputs(28, T, Hq, Hkv, 128, torch.bfloat16)
        want = attn.kda_attn_fwd(q, k, v)
        grads = attn.kda_attn_bwd(q, k, v, *want, dO)
        for cu in (None, cu_of([T // 3, T - T // 3])):
            ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
            calls = (lambda: attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, workspace=ws),
                     lambda: attn.kda_attn_bwd(q, k, v, *want, dO, cu_seqlens=cu, workspace=ws))
            for call in calls:
                try:
                    kda.kda_debug_set_wait_limit(20000, starve_carry=True)
                    call()
                    status, code = attn.kda_attn_status(ws)
                finally:
                    kda.kda_debug_set_wait_limit(0, starve_carry=False)
                assert status == 6 and code != 0
                call()
                assert attn.kda_attn_status(ws) == (0, 0)
        assert torch.equal(attn.kda_attn_fwd(q, k, v)[0], want[0])
        again = attn.kda_attn_bwd(q, k, v, *want, dO)
        assert all(torch.equal(again[n], grads[n]) for n in grads)


@pytest.mark.parametrize("d", [64, 128])
def test_long_sharp(d):
    """A longer sequence with large scores, whose row maximum moves late, and a scale of one."""
    T = 1500
    q, k, v, dO = inputs(13, T, 2, 1, d, torch.bfloat16)
    ramp = torch.linspace(0.2, 2.5, T, device="cuda")[None, :, None, None]
    k = (k * ramp).to(k.dtype)
    check(q, k, v, dO, [(0, T)], None)
    check((q * 0.3).to(q.dtype), k, v, dO, [(0, T)], None, scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_growing_scores(dtype):
    """Scores that rise along the keys by far more than one rescale step, and fall again."""
    T, d = 600, 64
    q, k, v, dO = inputs(14, T, 1, 1, d, DT[dtype])
    level = torch.cat([torch.linspace(-60, 60, 300), torch.linspace(60, -60, 300)]).to("cuda")
    q[..., 0] = 8.0
    k[0, :, 0, 0] = level.to(k.dtype)
    check(q, k, v, dO, [(0, T)], None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128])
def test_masked_places_do_not_matter(d, bad, dtype):
    """Later tokens, other sequences and tokens outside all of them may hold anything."""
    attn, lens = api(), [40, 150, 60]
    T = 300  # 50 tokens behind the last sequence
    q, k, v, dO = inputs(15, T, 4, 2, d, DT[dtype])
    cu = cu_of(lens)
    spans = spans_of(lens)
    base = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu)
    gb = attn.kda_attn_bwd(q, k, v, *base, dO, cu_seqlens=cu)
    q2, k2, v2, dO2 = (x.clone() for x in (q, k, v, dO))
    for x in (q2, k2, v2, dO2):
        x[0, 250:] = bad
    k2[0, 100], v2[0, 100] = bad, bad  # inside the second sequence [40, 190)
    q2[0, 150, 1] = bad
    o, lse = attn.kda_attn_fwd(q2, k2, v2, cu_seqlens=cu)
    clean = torch.ones(T, dtype=torch.bool, device="cuda")
    clean[100:190] = False
    clean[250:] = False
    ro, rl, to, tl = R.attn_fwd(q[0], k[0], v[0], spans, d ** -0.5)
    R.close(o[0][clean], ro[clean], to[clean])
    R.close(lse[0][clean], rl[clean], tl[clean])
    # gradients: other sequences are untouched, and so is dq before the bad token
    g = attn.kda_attn_bwd(q2, k2, v2, o, lse, dO2, cu_seqlens=cu)
    want, tol = R.attn_bwd(q[0], k[0], v[0], base[0][0], base[1][0], dO[0], spans, d ** -0.5)
    apart = clean.clone()
    apart[40:100] = False
    R.close(g["dq"][0][clean], want[0][clean], tol[0][clean] * 4)
    for name, w, t in zip(("dk", "dv"), want[1:], tol[1:]):
        R.close(g[name][0][apart], w[apart], t[apart])
    assert all(torch.isfinite(x).all() for x in gb["dq"][0, :250].float()[None])


def test_outside_tokens_are_not_written():
    attn = api()
    q, k, v, dO = inputs(16, 200, 2, 1, 64, torch.bfloat16)
    cu = torch.tensor([0, 70, 130], dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    lse = torch.full((1, 200, 2), 7.0, device="cuda")
    attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, o=o, lse=lse)
    assert (o[0, 130:] == 7.0).all() and (lse[0, 130:] == 7.0).all()
    ro, _, to, _ = R.attn_fwd(q[0, :130], k[0, :130], v[0, :130], [(0, 70), (70, 60)], 64 ** -0.5)
    R.close(o[0, :130], ro, to)


@pytest.mark.parametrize("offsets,spans", [
    ([0, 90, 40, 400], [(0, 90), (90, 0), (90, 110)]),   # falls back, and ends behind the tokens
    ([-5, 20, 200], [(0, 20), (20, 180)]),
])
def test_malformed_offsets_stay_inside(offsets, spans):
    attn = api()
    for d in (64, 128):
        q, k, v, dO = inputs(17, 200, 2, 1, d, torch.bfloat16)
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        check(q, k, v, dO, spans, cu)


def test_empty_call():
    attn = api()
    q, k, v, dO = inputs(18, 0, 2, 1, 64, torch.bfloat16)
    o, lse = attn.kda_attn_fwd(q, k, v)
    assert o.shape == q.shape and lse.shape == (1, 0, 2)
    assert attn.kda_attn_bwd(q, k, v, o, lse, dO)["dk"].shape == k.shape


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_runs_are_bit_equal(dtype):
    attn, lens = api(), [300, 77, 513]
    q, k, v, dO = inputs(19, sum(lens), 6, 2, 128, DT[dtype])
    cu = cu_of(lens)
    one = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu)
    g1 = attn.kda_attn_bwd(q, k, v, *one, dO, cu_seqlens=cu)
    for _ in range(3):
        two = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu)
        g2 = attn.kda_attn_bwd(q, k, v, *two, dO, cu_seqlens=cu)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        assert all(torch.equal(g1[n], g2[n]) for n in g1)


@pytest.mark.parametrize("d", [64, 128])
def test_calls_one_after_another_agree(d):
    """Many calls without a pause in between, on two sets of inputs in turn."""
    attn, lens = api(), [900, 33, 1700, 128, 257]
    cu = cu_of(lens)
    sets = [inputs(s, sum(lens), 8, 2, d, torch.bfloat16) for s in (29, 30)]

    def run(x):
        o, lse = attn.kda_attn_fwd(*x[:3], cu_seqlens=cu)
        return [o, lse, *attn.kda_attn_bwd(*x[:3], o, lse, x[3], cu_seqlens=cu).values()]

    want = [run(x) for x in sets]
    for _ in range(20):
        for i, got in enumerate([run(sets[i % 2]) for i in range(10)]):
            assert all(torch.equal(a, b) for a, b in zip(got, want[i % 2]))


def test_no_lse_and_given_buffers():
    from gated_delta_rule_132_b200 import kda
    import ctypes
    attn = api()
    q, k, v, _ = inputs(20, 130, 2, 1, 64, torch.bfloat16)
    want, _ = attn.kda_attn_fwd(q, k, v)
    o = torch.empty_like(q)
    need = kda.lib().kda_attn_fwd_workspace_size(1, 130, 2, 1, 64, 0, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = kda.lib().kda_attn_fwd(kda._p(q), kda._p(k), kda._p(v), 1, None, 0, 1, 130, 2, 1, 64, 0.125,
                                kda._p(o), None, kda._p(ws), need,
                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    ws2 = torch.empty(need, dtype=torch.uint8, device="cuda")
    attn.kda_attn_fwd(q, k, v, workspace=ws2, o=o)
    assert attn.kda_attn_status(ws2) == (0, 0)


def test_another_stream():
    attn = api()
    q, k, v, dO = inputs(21, 500, 4, 2, 128, torch.bfloat16)
    want = attn.kda_attn_fwd(q, k, v)
    gw = attn.kda_attn_bwd(q, k, v, *want, dO)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(4):
        o, lse = attn.kda_attn_fwd(q, k, v, stream=s)
        g = attn.kda_attn_bwd(q, k, v, o, lse, dO, stream=s)
        junk = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(4)]
        s.synchronize()
        assert torch.equal(o, want[0]) and all(torch.equal(g[n], gw[n]) for n in g)
        del junk


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_captured_and_replayed(dtype, packed):
    """Two graphs, each with the workspaces it allocated, replayed with new inputs in turn."""
    attn, lens = api(), [130, 1, 250]
    cu = cu_of(lens) if packed else None
    graphs = []
    for seed in (22, 23):
        x = inputs(seed, 381, 4, 2, 64, DT[dtype])
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            attn.kda_attn_fwd(*x[:3], cu_seqlens=cu)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = attn.kda_attn_fwd(*x[:3], cu_seqlens=cu)
            grads = attn.kda_attn_bwd(*x[:3], o, lse, x[3], cu_seqlens=cu)
        graphs.append((g, x, o, lse, grads))
    fresh = inputs(24, 381, 4, 2, 64, DT[dtype])
    for a, b in zip(graphs[0][1], fresh):
        a.copy_(b)
    for _ in range(2):
        for g, *_ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, x, o, lse, grads in graphs:
        want = attn.kda_attn_fwd(*x[:3], cu_seqlens=cu)
        gw = attn.kda_attn_bwd(*x[:3], *want, x[3], cu_seqlens=cu)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert all(torch.equal(grads[n], gw[n]) for n in gw)


def test_refusals():
    attn = api()
    q, k, v, dO = inputs(25, 32, 4, 2, 64, torch.bfloat16)
    from gated_delta_rule_132_b200.kda import KdaError
    with pytest.raises(ValueError, match="contiguous"):
        attn.kda_attn_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)
    with pytest.raises(TypeError):
        attn.kda_attn_fwd(q, k.float(), v)
    with pytest.raises(ValueError):
        attn.kda_attn_fwd(q, k, v[:, :16])
    with pytest.raises(KdaError):
        attn.kda_attn_fwd(q, k, v, scale=0.0)
    with pytest.raises(KdaError):
        attn.kda_attn_fwd(q[:, :, :3].contiguous(), k, v)
    with pytest.raises(KdaError):
        attn.kda_attn_fwd(q, k, v, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(KdaError):  # two batch rows and offsets
        attn.kda_attn_fwd(*(x.expand(2, -1, -1, -1).contiguous() for x in (q, k, v)), cu_seqlens=cu_of([32, 32]))
    flat = torch.zeros(q.numel() + 4, dtype=q.dtype, device="cuda")
    with pytest.raises(KdaError, match="ALIGNMENT"):
        attn.kda_attn_fwd(flat[4:].view_as(q), k, v)
    o, lse = attn.kda_attn_fwd(q, k, v)
    with pytest.raises(ValueError):
        attn.kda_attn_bwd(q, k, v, o, lse[:, :16].contiguous(), dO)
    with pytest.raises(TypeError):
        attn.kda_attn_bwd(q, k, v, o, lse, dO.float())


@pytest.mark.slow
@pytest.mark.parametrize("Hq,Hkv,T", [(2, 1, 9000), (1, 1, 20011)])
def test_long(Hq, Hkv, T):
    q, k, v, dO = inputs(26, T, Hq, Hkv, 128, torch.bfloat16)
    check(q, k, v, dO, [(0, T)], None)
