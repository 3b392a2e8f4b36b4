"""The full-attention calls without a GPU: refusals, workspace sizes, and the plain
forms that the GPU tests compare with."""
import ctypes

import pytest
import torch

import attn_ref as R


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_132_b200 import attn, build
    build.build()
    return attn._lib()


def at(addr=0x10000):
    return ctypes.c_void_p(addr)


BIG = 1 << 40


def fwd(L, **kw):
    a = dict(q=at(), k=at(), v=at(), dt=1, cu=None, n=0, B=1, T=64, Hq=4, Hkv=2, d=128, scale=0.1,
             o=at(), lse=at(), ws=at(), size=BIG, stream=None)
    a.update(kw)
    return L.kda_attn_fwd(*a.values())


def bwd(L, **kw):
    a = dict(q=at(), k=at(), v=at(), o=at(), lse=at(), dO=at(), dt=1, cu=None, n=0, B=1, T=64, Hq=4,
             Hkv=2, d=128, scale=0.1, gq=at(), gk=at(), gv=at(), ws=at(), size=BIG, stream=None)
    a.update(kw)
    return L.kda_attn_bwd(*a.values())


def tree(L, **kw):
    a = dict(q=at(), k=at(), v=at(), dt=1, table=at(), ctx=at(), parents=at(), N=2, R=3, Hq=4, Hkv=2,
             d=128, P=8, M=4, page=16, scale=0.1, o=at(), lse=at(), ws=at(), size=BIG, stream=None)
    a.update(kw)
    return L.kda_attn_tree(*a.values())


# Nothing below may reach a device: the pointers are made up.
COMMON = [(dict(q=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(Hq=0), 1), (dict(Hkv=3), 1),
          (dict(d=96), 2), (dict(d=0), 1), (dict(dt=7), 2), (dict(q=at(0x10008)), 3), (dict(k=at(0x10002)), 3),
          (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
          (dict(scale=float("inf")), 1), (dict(Hq=131072, Hkv=1), 2)]
PROMPT = COMMON + [(dict(B=0), 1), (dict(T=-1), 1), (dict(cu=at(), n=0), 1), (dict(cu=at(), n=2, B=2), 1),
                   (dict(ws=None), 4), (dict(size=16), 4), (dict(cu=at(0x10002), n=2), 3),
                   (dict(B=1 << 16, T=1 << 16), 2), (dict(T=1 << 30, Hq=64, Hkv=64), 2),
                   (dict(T=0, q=None, o=None), 0)]


@pytest.mark.parametrize("kw,status", PROMPT + [(dict(lse=at(0x10008)), 3)])
def test_fwd_refuses(L, kw, status):
    assert fwd(L, **kw) == status


@pytest.mark.parametrize("kw,status", PROMPT + [(dict(lse=None), 1), (dict(dO=None), 1), (dict(gk=None), 1),
                                                (dict(gq=at(0x10004)), 3), (dict(dO=at(0x10004)), 3)])
def test_bwd_refuses(L, kw, status):
    assert bwd(L, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(N=0), 1), (dict(R=-1), 1), (dict(R=65), 2), (dict(M=0), 1), (dict(P=0), 1), (dict(page=0), 2),
    (dict(page=24), 2), (dict(page=2048), 2), (dict(M=1 << 28, page=16), 2), (dict(table=None), 1),
    (dict(ctx=None), 1), (dict(parents=at(0x10002)), 3), (dict(lse=at(0x10002)), 3), (dict(R=0, q=None), 0)])
def test_tree_refuses(L, kw, status):
    assert tree(L, **kw) == status


def call(L, name, defaults, **kw):
    a = dict(defaults)
    a.update(kw)
    return getattr(L, name)(*a.values())


FORK = dict(refs=at(), table=at(), lens=at(0x90000), parents=at(), N_in=4, N_out=4, M=8, P=16,
            new=at(0x20000), new_lens=at(0x30000), stream=None)
RESERVE = dict(refs=at(), table=at(), lens=at(), add=at(), N=4, M=8, P=16, page=16, copies=at(),
               status=at(), ws=at(), size=BIG, stream=None)
RELEASE = dict(refs=at(), table=at(), lens=at(), new=at(), N=4, M=8, P=16, page=16, stream=None)
APPEND = dict(k=at(), v=at(), dt=1, table=at(), start=at(), kn=at(), vn=at(), cu=None, n=0, B=2, T=3,
              Hkv=2, d=64, P=16, M=8, page=16, stream=None)
COMPACT = dict(k=at(), v=at(), dt=1, table=at(), ctx=at(), path=at(), N=4, R=5, Hkv=2, d=64, P=16, M=8,
               page=16, new=at(), stream=None)
COPY = dict(k=at(), v=at(), dt=1, copies=at(), C=4, Hkv=2, d=64, P=16, page=16, stream=None)


@pytest.mark.parametrize("name,defaults,kw,status", [
    ("kda_cache_fork", FORK, dict(refs=None), 1), ("kda_cache_fork", FORK, dict(N_in=0), 1),
    ("kda_cache_fork", FORK, dict(N_out=0), 1), ("kda_cache_fork", FORK, dict(P=0), 1),
    ("kda_cache_fork", FORK, dict(parents=at(0x10002)), 3),
    ("kda_cache_fork", FORK, dict(new=at(0x10000)), 1),          # in place
    ("kda_cache_fork", FORK, dict(new=at(0x10000 + 4 * 31)), 1),  # the last entry shared
    ("kda_cache_fork", FORK, dict(new_lens=at(0x90000)), 1),
    ("kda_cache_fork", FORK, dict(N_in=1 << 16, M=1 << 16), 2),
    ("kda_cache_reserve", RESERVE, dict(add=None), 1), ("kda_cache_reserve", RESERVE, dict(page=12), 2),
    ("kda_cache_reserve", RESERVE, dict(ws=None), 4), ("kda_cache_reserve", RESERVE, dict(size=8), 4),
    ("kda_cache_reserve", RESERVE, dict(M=0), 1), ("kda_cache_reserve", RESERVE, dict(ws=at(0x10008)), 3),
    ("kda_cache_release", RELEASE, dict(lens=None), 1), ("kda_cache_release", RELEASE, dict(N=0), 1),
    ("kda_cache_release", RELEASE, dict(page=0), 2), ("kda_cache_release", RELEASE, dict(new=at(0x10001)), 3),
    ("kda_cache_append", APPEND, dict(k=None), 1), ("kda_cache_append", APPEND, dict(kn=None), 1),
    ("kda_cache_append", APPEND, dict(kn=at(0x10008)), 3), ("kda_cache_append", APPEND, dict(d=48), 2),
    ("kda_cache_append", APPEND, dict(T=-1), 1), ("kda_cache_append", APPEND, dict(cu=at(), n=3), 1),
    ("kda_cache_append", APPEND, dict(T=0, kn=None), 0), ("kda_cache_append", APPEND, dict(dt=2), 2),
    ("kda_cache_compact", COMPACT, dict(path=None), 1), ("kda_cache_compact", COMPACT, dict(R=0), 1),
    ("kda_cache_compact", COMPACT, dict(R=1025), 2), ("kda_cache_compact", COMPACT, dict(v=at(0x10004)), 3),
    ("kda_cache_copy_pages", COPY, dict(copies=None), 1), ("kda_cache_copy_pages", COPY, dict(C=-1), 1),
    ("kda_cache_copy_pages", COPY, dict(C=16385), 2), ("kda_cache_copy_pages", COPY, dict(C=0), 0),
    ("kda_cache_copy_pages", COPY, dict(page=3), 2),
])
def test_cache_refuses(L, name, defaults, kw, status):
    assert call(L, name, defaults, **kw) == status


def test_workspace_sizes(L):
    for fn in (L.kda_attn_fwd_workspace_size, L.kda_attn_bwd_workspace_size):
        assert 256 <= fn(1, 1, 2, 1, 32, 0, 0) < fn(1, 100000, 2, 1, 32, 5, 0)
        assert fn(1, 100, 2, 1, 96, 0, 0) == 0 and fn(1, 100, 3, 2, 64, 0, 0) == 0
        assert fn(2, 100, 2, 1, 64, 0, 5) == 0
    # the backward keeps one number per token and head
    assert L.kda_attn_bwd_workspace_size(1, 4096, 8, 8, 128, 0, 1) >= 4096 * 8 * 4
    assert L.kda_attn_tree_workspace_size(4, 65, 8, 8, 128, 10, 16, 1) == 0
    assert L.kda_cache_reserve_workspace_size(4, 8, 100) >= 1200
    assert L.kda_cache_reserve_workspace_size(0, 8, 100) == 0


def test_binding_refuses():
    from gated_delta_rule_132_b200 import attn
    x = torch.zeros(1, 4, 2, 32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.kda_attn_fwd(x, x, x)
    with pytest.raises(TypeError):
        attn.kda_attn_fwd(x.half(), x.half(), x.half())
    with pytest.raises(ValueError):
        attn.kda_attn_fwd(x[0], x[0], x[0])


def small(seed, spans, Hq, Hkv, d):
    g = torch.Generator().manual_seed(seed)
    T = sum(n for _, n in spans)
    mk = lambda h: torch.randn(T, h, d, generator=g, dtype=torch.float64)  # noqa: E731
    return mk(Hq), mk(Hkv), mk(Hkv), mk(Hq)


def test_plain_gradients_are_the_differences():
    """The formulas of the backward against central differences of the forward (fp64)."""
    spans, scale = [(0, 3), (3, 0), (3, 4)], 0.6
    q, k, v, dO = small(3, spans, 4, 2, 2)

    def loss(q, k, v):
        return float((R.attn_fwd(q, k, v, spans, scale)[0] * dO).sum())

    o, lse = R.attn_fwd(q, k, v, spans, scale)[:2]
    grads = R.attn_bwd(q, k, v, o, lse, dO, spans, scale)[0]
    h = 1e-5
    for i, x in enumerate((q, k, v)):
        flat = x.view(-1)
        for j in range(flat.numel()):
            keep = float(flat[j])
            flat[j] = keep + h
            hi = loss(q, k, v)
            flat[j] = keep - h
            lo = loss(q, k, v)
            flat[j] = keep
            assert abs((hi - lo) / (2 * h) - float(grads[i].view(-1)[j])) < 1e-8


def test_plain_masked_places_do_not_matter():
    spans = [(0, 5), (5, 4)]
    q, k, v, _ = small(4, spans, 2, 1, 4)
    o, lse = R.attn_fwd(q, k, v, spans, 0.5)[:2]
    k[3], v[3] = float("nan"), float("inf")
    o2, lse2 = R.attn_fwd(q, k, v, spans, 0.5)[:2]
    for keep in (slice(0, 3), slice(5, 9)):
        assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert not torch.isfinite(o2[3:5]).any()


def test_plain_tree_chain_is_causal():
    """A chain over a cache is the last rows of causal attention over the whole."""
    N, c, n, d, page = 1, 5, 3, 4, 4
    q, k, v, _ = small(5, [(0, c + n)], 2, 1, d)
    kp, vp = (torch.zeros(3, 1, page, d, dtype=torch.float64) for _ in range(2))
    for pool, x in ((kp, k), (vp, v)):
        for t in range(c + n):
            pool[[2, 0][t // page], 0, t % page] = x[t, 0]
    table = torch.tensor([[2, 0, -1]], dtype=torch.int32)
    o, lse = R.attn_tree(q[None, c:], kp, vp, table, torch.tensor([c]), None, 0.5)[:2]
    ref, zref = R.attn_fwd(q, k, v, [(0, c + n)], 0.5)[:2]
    assert torch.allclose(o[0], ref[c:], atol=1e-12) and torch.allclose(lse[0], zref[c:], atol=1e-12)


def test_pages_model():
    p = R.Pages([1, 1, 0, 0, 0], [[0, 1, -1], [-1, -1, -1]], [5, 0], 4)
    p.fork([0, 0])
    assert p.refs == [2, 2, 0, 0, 0] and p.lens == [5, 5]
    copies, status = p.reserve([4, 1])  # the first copies the shared page, the last holder keeps it
    assert status == 0 and copies == [[1, 2], [-1, -1]]
    assert p.table == [[0, 2, 3], [0, 1, -1]] and p.refs == [2, 1, 1, 1, 0] and p.lens == [9, 6]
    assert p.reserve([3, 3])[1] == 0 and p.table[1] == [0, 1, 4]
    assert p.reserve([1, 0])[1] == -1
    p.release([4, 0])
    assert p.refs == [1, 0, 0, 0, 0] and p.table == [[0, -1, -1], [-1, -1, -1]]
