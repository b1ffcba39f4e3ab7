"""Paged caches on the GPU against the fp64 oracle.

Tolerances. Attention: the oracle's own bounds for 32-bit arithmetic over the same inputs.
Append: one rounding to the storage type (bf16 2^-8, fp32 2^-24 of the value) plus 32-bit
arithmetic: norm, weight and rotation are some 30 roundings of 2^-24 of |r_a| + |r_b|, and the
angle's error (2^-20 + |angle| 2^-43) turns the pair by as much of the same sum. Moves, tables
and copied rows are exact.
"""

import numpy as np
import pytest
import torch

import oracle.paged_oracle as pg
from helpers import ensure_built
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def api():
    from kv_cache_eviction_snapkv_gb300 import api as a
    return a


def status():
    return api().kvsel_device_status()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen).to(dtype).to(DEV)


class Cache:
    """Random pages of sequences of the given lengths. layout: "dense", "kv" (K and V pages
    interleaved) or "layers" (the layers of a page side by side). What no sequence holds (rows
    past the ends, unused pages) is NaN; table entries past the ends are out of range."""

    def __init__(self, lens, ps, layers, Hkv, D, dtype, seed=0, layout="dense", spare=3):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.ps = list(lens), ps
        need = [-(-n // ps) for n in lens]
        self.P = sum(need) + spare
        W = max(need + [0]) + 1
        order = torch.randperm(self.P, generator=gen).tolist()
        table, live, at = [], torch.zeros((self.P, ps), dtype=torch.bool), 0
        for n, w in zip(lens, need):
            own = order[at:at + w]
            at += w
            table.append(own + [self.P + 7] * (W - w))
            for j in range(n):
                live[own[j // ps], j % ps] = True
        self.table = ints(table)
        live = live[None, :, :, None, None]
        pools = [torch.where(live, torch.randn((layers, self.P, ps, Hkv, D), generator=gen),
                             float("nan")).to(dtype) for _ in range(2)]
        if layout == "kv":
            both = torch.stack(pools, dim=2).to(DEV)
            self.K, self.V = both[:, :, 0], both[:, :, 1]
        elif layout == "layers":
            self.K, self.V = (p.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for p in pools)
        else:
            self.K, self.V = (p.to(DEV) for p in pools)
        self.dlens = ints(self.lens)


def check_attention(c, q, out, lse):
    o, z, ob, zb = pg.attention(f64(q), f64(c.K), f64(c.V), c.table.cpu().numpy(), c.lens)
    got, gz = f64(out), f64(lse)
    assert np.array_equal(np.isneginf(gz), np.isneginf(z))
    live = ~np.isneginf(z)
    assert (np.abs(got - o) <= ob).all(), float((np.abs(got - o) / np.maximum(ob, 1e-30)).max())
    assert (np.abs(gz[live] - z[live]) <= zb[live]).all()
    assert not got[~live].any()


ATTENTION = [
    # dtype, D, H, Hkv, page, layers, layout, lens
    (BF16, 128, 8, 2, 16, 2, "dense", [1, 0, 15, 16, 17, 63, 64, 65, 300]),
    (BF16, 128, 3, 3, 1, 1, "dense", [1, 2, 31, 33]),
    (BF16, 64, 12, 1, 8, 1, "kv", [0, 500, 129, 7]),
    (BF16, 64, 20, 1, 32, 2, "layers", [257, 64]),
    (BF16, 128, 48, 2, 64, 1, "dense", [1, 1000, 64]),
    (BF16, 128, 5, 1, 128, 1, "kv", [5000]),
    (BF16, 128, 2, 1, 256, 3, "dense", [0, 0, 3]),
    (BF16, 128, 64, 1, 16, 1, "dense", [3000, 17]),
    (BF16, 128, 1, 1, 16, 1, "kv", [20000]),
    (F32, 64, 6, 3, 16, 2, "dense", [1, 0, 15, 16, 17, 63, 64, 65, 300]),
    (F32, 128, 4, 4, 2, 1, "layers", [129, 1000, 1]),
    (F32, 128, 17, 1, 32, 1, "kv", [33, 0, 2049]),
    (F32, 64, 9, 1, 8, 1, "dense", [4000]),
]


@pytest.mark.parametrize("dtype,D,H,Hkv,ps,layers,layout,lens", ATTENTION)
def test_attention(dtype, D, H, Hkv, ps, layers, layout, lens):
    c = Cache(lens, ps, layers, Hkv, D, dtype, seed=len(lens) + D, layout=layout)
    gen = torch.Generator().manual_seed(7)
    q = normal(gen, dtype, layers, len(lens), H, D) * 2
    out, lse = Guarded(q.shape, F32), Guarded(q.shape[:3], F32)
    api().kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens, out.t, lse.t)
    assert status() == 0
    assert out.intact() and lse.intact()
    check_attention(c, q, out.t, lse.t)
    again, _ = api().kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens, want_lse=False)
    assert torch.equal(again, out.t)


def test_attention_large_scores_and_many_sequences():
    """Scores of several hundred (one row takes the whole weight), and a batch that is longer
    than the blocks of the launch."""
    c = Cache([3 + i % 90 for i in range(700)], 16, 1, 1, 64, BF16, seed=3)
    gen = torch.Generator().manual_seed(8)
    q = normal(gen, BF16, 1, 700, 2, 64)
    q[:, ::5] *= 100
    out, lse = api().kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens)
    assert status() == 0
    check_attention(c, q, out, lse)


def test_attention_of_the_most_sequences():
    """8192 sequences, most of them empty or of a few rows, and layers."""
    c = Cache([(i * 7) % 5 if i % 3 else 0 for i in range(8192)], 2, 2, 1, 64, F32, seed=13)
    q = normal(torch.Generator().manual_seed(14), F32, 2, 8192, 1, 64)
    out, lse = api().kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens)
    assert status() == 0
    check_attention(c, q, out, lse)
    with pytest.raises(api().KvselError) as e:
        api().kvsel_paged_attention(torch.zeros((2, 8193, 1, 64), device=DEV), c.K, c.V,
                                    torch.zeros((8193, 1), dtype=torch.int32, device=DEV),
                                    torch.zeros(8193, dtype=torch.int32, device=DEV))
    assert e.value.status == api().KVSEL_ERR_UNSUPPORTED


def test_calls_on_nothing():
    """No sequences, no tokens, no pages: nothing is done, and update frees every page."""
    a = api()
    c = Cache([20, 5], 16, 1, 2, 64, BF16, seed=15)
    none = ints([])
    empty = torch.zeros((0, c.table.shape[1]), dtype=torch.int32, device=DEV)
    out, lse = a.kvsel_paged_attention(torch.zeros((1, 0, 4, 64), dtype=BF16, device=DEV), c.K, c.V, empty,
                                       none)
    assert out.shape == (1, 0, 4, 64) and lse.shape == (1, 0, 4)
    q = a.kvsel_paged_append(torch.zeros((0, 4, 64), dtype=BF16, device=DEV), None, None, c.K, c.V, None)
    assert q.shape == (0, 4, 64)
    t, ref, free = a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, none, parents=none)
    assert t.shape[0] == 0 and not ref.any() and free.item() == c.P
    t, ref, free = a.kvsel_pages_update(c.K, c.V, empty, none, ints([17, 0, 1]), parents=ints([-1, -1, -1]))
    assert t[:, :2].tolist() == [[0, 1], [-1, -1], [2, -1]] and free.item() == c.P - 3
    nothing = torch.zeros((1, 0, 16, 2, 64), dtype=BF16, device=DEV)
    assert status() == 0
    out, lse = a.kvsel_paged_attention(torch.ones((1, 1, 2, 64), dtype=BF16, device=DEV), nothing, nothing,
                                       ints([[0]]), ints([3]))
    assert status() == a.KVSEL_ERR_BAD_INDEX
    assert not out.any() and bool(torch.isneginf(lse).all())
    t, ref, free = a.kvsel_pages_update(nothing, nothing, ints([[-1]]), ints([0]), ints([3]))
    assert status() == a.KVSEL_ERR_NO_PAGES
    assert t.tolist() == [[-1]] and free.item() == -1
    pos = a.kvsel_paged_compact(c.K, c.V, c.table, c.dlens, torch.zeros((1, 0, 2), dtype=torch.int32,
                                                                        device=DEV), ints([0, 0, 0]), 4)
    assert pos.shape == (1, 0, 2) and status() == 0


def test_attention_agrees_with_the_packed_call():
    """A packed cache is a pool of one-row pages; both calls read it alike."""
    gen = torch.Generator().manual_seed(9)
    K, V = (normal(gen, BF16, 2, 900, 2, 128) for _ in range(2))
    q = normal(gen, BF16, 2, 1, 8, 128)
    o1, l1 = api().kvsel_decode_attention(q, K, V, [0, 900])
    table = torch.arange(900, dtype=torch.int32, device=DEV)[None]
    o2, l2 = api().kvsel_paged_attention(q, K.unsqueeze(2), V.unsqueeze(2), table, ints([900]))
    assert status() == 0
    torch.testing.assert_close(o2, o1, rtol=1e-4, atol=2e-5)
    torch.testing.assert_close(l2, l1, rtol=0, atol=1e-4)


def test_attention_bad_lengths_pages_and_values():
    a = api()
    c = Cache([40, 20], 16, 1, 1, 64, BF16, seed=5)
    q = normal(torch.Generator().manual_seed(1), BF16, 1, 2, 2, 64)
    good, _ = a.kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens)
    assert status() == 0
    bad = c.table.clone()
    bad[0, 1] = c.P                                   # one page out of range: its rows are left out
    out, _ = a.kvsel_paged_attention(q, c.K, c.V, bad, c.dlens)
    assert status() == a.KVSEL_ERR_BAD_INDEX
    assert torch.equal(out[:, 1], good[:, 1])
    keep = [j for j in range(40) if j // 16 != 1]
    rows = [pg.rows_of(f64(t)[0], c.table[0].cpu().numpy(), 40)[keep, 0] for t in (c.K, c.V)]
    import oracle.decode_oracle as dec
    for h in range(2):
        ref, _ = dec.decode_attention(f64(q)[0, 0, h], *rows)
        np.testing.assert_allclose(f64(out)[0, 0, h], ref, rtol=1e-4, atol=2e-5)
    out, lse = a.kvsel_paged_attention(q, c.K, c.V, c.table, ints([-5, 20]))
    assert status() == a.KVSEL_ERR_BAD_INDEX
    # other lengths cut the rows into other runs, so sequence 1's sums differ by their rounding:
    # the bound for any order of 32-bit sums holds, equal bits are promised for equal arguments only
    o, _, ob, _ = pg.attention(f64(q), f64(c.K), f64(c.V), c.table.cpu().numpy(), [0, 20])
    assert not out[:, 0].any() and (np.abs(f64(out) - o) <= ob).all()
    a.kvsel_paged_attention(q, c.K, c.V, c.table, ints([40, 1 << 30]))   # held to the table's rows
    assert status() == a.KVSEL_ERR_BAD_INDEX
    c.K[0, c.table[1, 0], 3] = float("inf")
    out, _ = a.kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens)
    assert status() == a.KVSEL_ERR_NONFINITE
    assert torch.equal(out[:, 0], good[:, 0])
    assert status() == 0


def test_attention_replays_with_new_lengths_on_another_stream():
    c = Cache([100, 130], 16, 2, 2, 128, BF16, seed=6)
    q = normal(torch.Generator().manual_seed(2), BF16, 2, 2, 4, 128)
    out, lse = (torch.empty(s, device=DEV) for s in (q.shape, q.shape[:3]))
    args = (q, c.K, c.V, c.table, c.dlens, out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api().kvsel_paged_attention(*args)
    side.synchronize()
    graphs = []
    for _ in range(2):                                # two graphs over the same tensors
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            api().kvsel_paged_attention(*args)
        graphs.append(g)
    for lens in ([100, 130], [1, 77], [0, 128]):
        c.lens = lens
        c.dlens.copy_(ints(lens))
        for g in graphs:
            out.fill_(float("nan"))
            g.replay()
            assert status() == 0
            check_attention(c, q, out, lse)
    out2, lse2 = api().kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens, stream=side)
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dtype,D,H,Hkv", [(BF16, 128, 24, 1), (F32, 64, 6, 2), (F32, 128, 9, 1)])
def test_workspaces_of_the_least_size(dtype, D, H, Hkv):
    """Both calls stay within the bytes that they ask for, whatever lies in them before, and a
    byte less is refused; q on a 16-byte boundary only."""
    import ctypes
    from kv_cache_eviction_snapkv_gb300 import _native
    a = api()
    c = Cache([5000, 3, 0, 64, 1200], 16, 2, Hkv, D, dtype, seed=40, spare=900)
    pool = _native.KvselPages(2, c.P, 16, Hkv, D, 0 if dtype == BF16 else 1, 0, 0, c.K.data_ptr(),
                              c.V.data_ptr())
    lib = _native.lib()
    n = lib.kvsel_paged_attention_bytes(ctypes.byref(pool), 5, H)
    ws = Guarded((n,), torch.uint8)
    flat = torch.empty(2 * 5 * H * D + 8, dtype=dtype, device=DEV)
    q = flat[16 // flat.element_size():][:2 * 5 * H * D].view(2, 5, H, D)
    q.copy_(normal(torch.Generator().manual_seed(41), dtype, 2, 5, H, D))
    for fill in (0, 255):
        ws.t.fill_(fill)
        out, lse = a.kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens, workspace=ws.t)
        assert status() == 0 and ws.intact()
        check_attention(c, q, out, lse)
    with pytest.raises(a.KvselError):
        a.kvsel_paged_attention(q, c.K, c.V, c.table, c.dlens, workspace=ws.t[:n - 1])
    m = lib.kvsel_pages_update_bytes(ctypes.byref(pool), 7)
    ws = Guarded((m,), torch.uint8)
    new, parents = [5001, 5001, 4, 0, 65, 1201, 30], [0, 0, 1, 2, 3, 4, 0]
    table, ref, free, _ = pg.update(c.table.tolist(), c.lens, parents, new, c.P, 16)
    for fill in (0, 255):
        ws.t.fill_(fill)
        t, r, f = a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, ints(new), parents=ints(parents),
                                       workspace=ws.t)
        assert status() == 0 and ws.intact()
        assert t.tolist() == table and r.tolist() == ref and f.item() == free
    with pytest.raises(a.KvselError):
        a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, ints(new), parents=ints(parents),
                             workspace=ws.t[:m - 1])


def test_calls_on_two_streams_at_once():
    """Each call has a workspace of its own: many of them in flight on two streams give what
    they give alone."""
    a = api()
    caches = [Cache([4000 + 300 * i, 77, 0, 900], 16, 1, 2, 128, BF16, seed=20 + i) for i in range(2)]
    qs = [normal(torch.Generator().manual_seed(30 + i), BF16, 1, 4, 8, 128) for i in range(2)]
    grown = [ints([n + 1 for n in c.lens]) for c in caches]
    parents = ints([0, 1, 1, 3])

    def calls(i, stream):
        c = caches[i]
        out, lse = a.kvsel_paged_attention(qs[i], c.K, c.V, c.table, c.dlens, stream=stream)
        return (out, lse, *a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, grown[i], parents=parents,
                                                stream=stream))

    alone = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [calls(k % 2, streams[k % 2]) for k in range(40)]
    torch.cuda.synchronize()
    assert status() == 0
    for k, r in enumerate(got):
        for x, y in zip(r, alone[k % 2]):
            assert torch.equal(x, y)


# ---------------------------------------------------------------------------

def append_reference(x, w, eps, pos, inv_freq, interleaved, scale, dtype):
    """(value, bound) of [L, N, heads, D] rows."""
    r = x if w is None else np.stack([pg.norm(x[l], w[l], eps) for l in range(x.shape[0])])
    y, s = r.copy(), np.abs(r)
    if inv_freq is not None:
        ang = pos[:, None] * inv_freq[None]
        half = ang.shape[1]
        y = np.stack([pg.rotate(r[l], ang, interleaved, scale) for l in range(x.shape[0])])
        a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
        both = (np.abs(r[..., a]) + np.abs(r[..., b])) * abs(scale)
        turn = (2.0 ** -20 + np.abs(ang) * 2.0 ** -43)[:, None]
        s = s * (30 * pg.U32)
        s[..., a] = s[..., b] = both * (30 * pg.U32 + turn)
    else:
        s = s * (30 * pg.U32)
    step = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    return y, s + (np.abs(y) + s) * step + 1e-38


APPEND = [
    # dtype, D, H, Hkv, page, layers, tokens, rot, interleaved, norm, far
    (BF16, 128, 8, 2, 16, 2, 5, 128, False, True, 100000),
    (BF16, 128, 1, 1, 1, 1, 1, 16, True, True, 3),
    (BF16, 64, 3, 1, 8, 1, 301, 48, False, False, 1 << 24),
    (BF16, 64, 4, 4, 64, 3, 33, 64, True, True, 5000),
    (BF16, 128, 33, 3, 32, 1, 130, 0, False, True, 1),
    (F32, 64, 12, 4, 16, 2, 77, 32, True, False, 1000000),
    (F32, 128, 6, 2, 8, 1, 9, 128, False, True, (1 << 31) - 1),
    (F32, 128, 2, 1, 4, 1, 1000, 96, False, True, 40000),
]


@pytest.mark.parametrize("dtype,D,H,Hkv,ps,layers,N,rot,inter,norm,far", APPEND)
@pytest.mark.parametrize("fused", [False, True])
def test_append(dtype, D, H, Hkv, ps, layers, N, rot, inter, norm, far, fused):
    a = api()
    gen = torch.Generator().manual_seed(N + D)
    S = min(3, N)
    c = Cache([N + 20] * S, ps, layers, Hkv, D, dtype, seed=N)
    if fused:
        qkv = normal(gen, dtype, layers, N, H + 2 * Hkv, D)
        q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    else:
        q, k, v = (normal(gen, dtype, layers, N, h, D) for h in (H, Hkv, Hkv))
    seqs = torch.randint(0, S, (N,), generator=gen).to(torch.int32)
    pos_in = torch.arange(N).to(torch.int32) + 3
    pos_in[::7] = -1                                   # padding tokens
    positions = torch.randint(0, far, (N,), generator=gen).to(torch.int32)
    if far > 2:
        positions[-1] = far - 1
    w = [(1 + 0.3 * torch.randn((layers, D), generator=gen)).to(dtype).to(DEV) if norm else None
         for _ in range(2)]
    freq, scale = a.kvsel_rope_frequencies(rot) if rot else (torch.empty(0), 1.0)
    scale = 1.0 if not rot else 1.25
    q_out = Guarded(q.shape, dtype)
    K0, V0 = c.K.clone(), c.V.clone()
    got = a.kvsel_paged_append(q, k, v, c.K, c.V, pos_in.to(DEV), positions=positions.to(DEV),
                               table=c.table, seqs=seqs.to(DEV), q_weight=w[0], k_weight=w[1],
                               inv_freq=freq.to(DEV), interleaved=inter, scale=scale, q_out=q_out.t)
    assert status() == 0 and got is q_out.t and q_out.intact()
    p64, f = positions.double().numpy(), freq.double().numpy() if rot else None
    ref = lambda t, i: append_reference(f64(t), None if w[i] is None else f64(w[i]), 1e-6, p64, f,  # noqa: E731
                                        inter, scale, dtype)
    y, bound = ref(q, 0)
    assert (np.abs(f64(q_out.t) - y) <= bound).all()
    y, bound = ref(k, 1)
    live = [n for n in range(N) if pos_in[n] >= 0]
    page = c.table.cpu()[seqs[live].long(), (pos_in[live] // ps).long()].long()
    slot = (pos_in[live] % ps).long()
    assert (np.abs(f64(c.K.cpu()[:, page, slot]) - y[:, live]) <= bound[:, live]).all()
    assert torch.equal(c.V.cpu()[:, page, slot], v.cpu()[:, live])
    # every other row of the pool is as it was
    same = torch.ones(c.K.shape[1:3], dtype=torch.bool)
    same[page, slot] = False
    for now, old in ((c.K, K0), (c.V, V0)):
        x, z = now.cpu()[:, same], old.cpu()[:, same]
        assert torch.equal(x.view(torch.uint8), z.view(torch.uint8))


def test_append_parts_alone_and_in_place():
    """Queries in place; keys and values alone; a packed cache without a table; token n of
    sequence n without `seqs`."""
    a = api()
    gen = torch.Generator().manual_seed(4)
    q, k, v = (normal(gen, BF16, 5, h, 64) for h in (6, 2, 2))
    freq = a.kvsel_rope_frequencies(64)[0].to(DEV)
    pos = ints([9, 2, 100, 7, 0])
    K, V = (torch.zeros((40, 1, 2, 64), dtype=BF16, device=DEV) for _ in range(2))
    at = ints([39, 0, 17, -1, 5])
    whole = a.kvsel_paged_append(q, k, v, K, V, at, positions=pos, inv_freq=freq)
    assert status() == 0
    K2, V2 = torch.zeros_like(K), torch.zeros_like(V)
    assert a.kvsel_paged_append(None, k, v, K2, V2, at, positions=pos, inv_freq=freq) is None
    own = q.clone()
    a.kvsel_paged_append(own, None, None, K, V, None, positions=pos, inv_freq=freq, q_out=own)
    assert status() == 0
    assert torch.equal(own, whole) and torch.equal(K2, K) and torch.equal(V2, V)
    assert torch.equal(V[[39, 0, 17, 5], 0], v[[0, 1, 2, 4]])
    P, W = torch.zeros((20, 4, 2, 64), dtype=BF16, device=DEV), torch.zeros((20, 4, 2, 64), dtype=BF16, device=DEV)
    table = torch.randperm(20, generator=gen).to(torch.int32).to(DEV).view(5, 4)
    a.kvsel_paged_append(q, k, v, P, W, ints([0, 5, 15, -1, 8]), positions=pos, table=table, inv_freq=freq)
    assert status() == 0
    t = table.cpu().tolist()
    for n, (col, r) in {0: (0, 0), 1: (1, 1), 2: (3, 3), 4: (2, 0)}.items():
        assert torch.equal(W[t[n][col], r], v[n])
    assert int((W != 0).any(-1).sum()) == 8
    for bad in (dict(cache_pos=ints([16, 0, 0, -1, 0])), dict(table=table + 20),
                dict(seqs=ints([5, 0, 1, 2, 3])), dict(seqs=ints([-1, 0, 1, 2, 3]))):
        kw = dict(cache_pos=ints([0, 1, 2, -1, 3]), table=table, seqs=None)
        kw.update(bad)
        p2, w2 = torch.zeros_like(P), torch.zeros_like(W)
        got = a.kvsel_paged_append(q, k, v, p2, w2, kw["cache_pos"], positions=pos, table=kw["table"],
                                   seqs=kw["seqs"], inv_freq=freq)
        assert status() == a.KVSEL_ERR_BAD_INDEX
        assert torch.equal(got, whole)
    p2 = torch.zeros_like(K)
    a.kvsel_paged_append(q, k, v, p2, torch.zeros_like(K), ints([40, 0, 1, 2, 3]), positions=pos, inv_freq=freq)
    assert status() == a.KVSEL_ERR_BAD_INDEX and not p2[4:].any()


# ---------------------------------------------------------------------------

def run_compact(c, want, dtype, ref=None, max_keep=None):
    """want[layer][b][h]: kept rows. Calls the operator; returns slot_pos."""
    layers, S, Hkv = len(want), len(want[0]), len(want[0][0])
    offs = [0]
    for b in range(S):
        offs.append(offs[-1] + len(want[0][b][0]))
    idx = torch.zeros((layers, offs[-1], Hkv), dtype=torch.int32)
    for l in range(layers):
        for b in range(S):
            for h in range(Hkv):
                idx[l, offs[b]:offs[b + 1], h] = torch.tensor(want[l][b][h], dtype=torch.int32)
    most = max(offs[b + 1] - offs[b] for b in range(S)) if max_keep is None else max_keep
    pos = Guarded(idx.shape, torch.int32)
    api().kvsel_paged_compact(c.K, c.V, c.table, c.dlens, idx.to(DEV), ints(offs), most, ref=ref,
                              slot_pos=pos.t)
    assert pos.intact()
    return pos.t.cpu(), offs


COMPACT = [
    # dtype, D, Hkv, page, layers, layout, lens, kept
    (BF16, 128, 2, 16, 2, "dense", [100, 17, 1, 64], [40, 17, 1, 33]),
    (BF16, 64, 3, 1, 1, "kv", [50, 0, 9], [49, 0, 0]),
    (F32, 64, 1, 8, 3, "layers", [700, 3], [256, 2]),
    (F32, 128, 2, 64, 1, "dense", [3000], [1033]),
    (BF16, 128, 8, 32, 1, "dense", [21000], [16500]),
    (BF16, 64, 1, 16, 1, "dense", [33001], [32768]),
]


@pytest.mark.parametrize("dtype,D,Hkv,ps,layers,layout,lens,kept", COMPACT)
def test_compact(dtype, D, Hkv, ps, layers, layout, lens, kept):
    c = Cache(lens, ps, layers, Hkv, D, dtype, seed=sum(lens), layout=layout)
    rng = np.random.default_rng(sum(kept))
    want = [[[rng.permutation(n)[:m].tolist() for _ in range(Hkv)] for n, m in zip(lens, kept)]
            for _ in range(layers)]
    K0, V0 = c.K.cpu(), c.V.cpu()
    pos, offs = run_compact(c, want, dtype, ref=torch.ones(c.P, dtype=torch.int32, device=DEV))
    assert status() == 0
    table = c.table.cpu().long()
    Ke, Ve = K0.clone(), V0.clone()
    for l in range(layers):
        for b, n in enumerate(lens):
            for h in range(Hkv):
                take = pg.compact(want[l][b][h], n)
                assert pos[l, offs[b]:offs[b + 1], h].tolist() == take
                t, s = torch.tensor(take, dtype=torch.long), torch.arange(len(take))
                for new, old in ((Ke, K0), (Ve, V0)):
                    new[l, table[b, s // ps], s % ps, h] = old[l, table[b, t // ps], t % ps, h]
    for got, ref in ((c.K.cpu(), Ke), (c.V.cpu(), Ve)):
        assert torch.equal(got.contiguous().view(torch.uint8), ref.contiguous().view(torch.uint8))


def test_compact_refusals_leave_the_rows():
    a = api()
    want = [[[[5, 30, 2], [1, 2, 3]], [[9, 8], [0, 11]]]]

    def fresh():
        return Cache([40, 12], 16, 1, 2, 64, F32, seed=8)

    c = fresh()
    base_k = c.K.clone()
    shared = torch.ones(c.P, dtype=torch.int32, device=DEV)
    shared[c.table[0, 0].long()] = 2
    run_compact(c, want, F32, ref=shared)
    assert status() == a.KVSEL_ERR_SHARED_PAGE
    first = c.table[0, :3].long()
    same = lambda x, y: torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))  # noqa: E731
    assert same(c.K[:, first], base_k[:, first])
    second = c.table[1, :1].long()
    assert not same(c.K[:, second], base_k[:, second])
    for change in ("twice", "range", "negative", "most", "length", "page"):
        c = fresh()
        w = [[[list(x) for x in b] for b in want[0]]]
        kw = {}
        if change == "twice":
            w[0][0][0] = [2, 30, 2]
        elif change == "range":
            w[0][0][0] = [2, 40, 1]
        elif change == "negative":
            w[0][0][0] = [2, -1, 1]
        elif change == "most":
            kw["max_keep"] = 2
        elif change == "length":
            c.dlens = ints([2, 12])
        else:
            c.table[0, 0] = -1
        run_compact(c, w, F32, **kw)
        assert status() == a.KVSEL_ERR_BAD_INDEX, change
        rows = torch.ones_like(base_k, dtype=torch.bool)
        rows[:, second] = False
        if change in ("twice", "range", "negative"):
            rows[..., 1, :] = False                    # the other head's list is fine
        assert same(c.K[rows], base_k[rows]), change
        assert not same(c.K[:, second], base_k[:, second]), change


# ---------------------------------------------------------------------------

def check_update(c, parents, new, status_want=0):
    table, ref, free, copies = pg.update(c.table.tolist(), c.lens, parents, new, c.P, c.ps)
    K0, V0 = c.K.cpu(), c.V.cpu()
    W = c.table.shape[1]
    out = Guarded((len(new), W), torch.int32)
    r = Guarded((c.P,), torch.int32)
    t, rr, f = api().kvsel_pages_update(c.K, c.V, c.table, c.dlens, ints(new),
                                        parents=None if parents is None else ints(parents),
                                        table_out=out.t, ref=r.t)
    assert status() == status_want
    assert out.intact() and r.intact()
    assert t.tolist() == table and rr.tolist() == ref and f.item() == free
    for src, dst, n in copies:
        K0[:, dst, :n] = K0[:, src, :n]
        V0[:, dst, :n] = V0[:, src, :n]
    for got, want in ((c.K.cpu(), K0), (c.V.cpu(), V0)):
        assert torch.equal(got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))
    c.table, c.lens, c.dlens = t, list(new), ints(new)
    return ref


@pytest.mark.parametrize("dtype,D,Hkv,ps,layers,layout", [
    (BF16, 64, 2, 4, 2, "dense"), (F32, 128, 1, 1, 1, "kv"), (BF16, 128, 3, 16, 3, "layers")])
def test_update_steps(dtype, D, Hkv, ps, layers, layout):
    c = Cache([30, 0, 13, 16], ps, layers, Hkv, D, dtype, seed=2, layout=layout, spare=200)
    cap = c.table.shape[1] * ps
    rng = np.random.default_rng(ps)
    check_update(c, None, [min(cap, n + 1) for n in c.lens])
    check_update(c, [0, 0, 0, 2, 2, -1, 3, 0], [c.lens[0]] * 3 + [5, 9, 3, 16, 7])
    for _ in range(12):
        n = int(rng.integers(1, 12))
        parents = [int(rng.integers(-1, len(c.lens))) for _ in range(n)]
        new = [int(rng.integers(0, min(cap, (c.lens[p] if p >= 0 else 0) + 5) + 1)) for p in parents]
        check_update(c, parents, new)
    check_update(c, [-1], [0])


def test_update_many_sequences_and_pages():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 400, size=1500)]
    c = Cache(lens, 16, 1, 1, 64, BF16, seed=3, spare=9000)
    parents = [int(x) for x in rng.integers(-1, 1500, size=1700)]
    new = [min(400, lens[p] + 1 if p >= 0 else 40) for p in parents]
    args = (c.K, c.V, c.table, c.dlens, ints(new), ints(parents))
    ref = check_update(c, parents, new)
    odd = torch.empty(c.P + 1, dtype=torch.int32, device=DEV)[1:]      # not on a 16-byte boundary
    _, got, _ = api().kvsel_pages_update(*args, ref=odd)
    assert status() == 0 and got is odd and got.tolist() == ref


def test_update_more_sequences_and_pages_than_shared_memory_holds():
    """3000 sequences in a pool of 260000 one-row pages, and 300 columns a table."""
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 60, size=2999)] + [299]
    c = Cache(lens, 1, 1, 1, 64, BF16, seed=3, spare=260000 - sum(lens))
    assert c.P == 260000
    parents = [int(x) for x in rng.integers(-1, 3000, size=3000)]
    check_update(c, parents, [min(300, lens[p] + 2) if p >= 0 else 1 for p in parents])
    c = Cache(lens, 2, 1, 1, 64, BF16, seed=4, spare=5000)
    check_update(c, parents, [min(300, lens[p] + 1) if p >= 0 else 3 for p in parents])


def test_update_shortfall_and_bad_arguments():
    a = api()
    c = Cache([20, 40], 16, 1, 1, 64, BF16, seed=4, spare=1)
    check_update(c, [0, 1, 1], [33, 40, 41], a.KVSEL_ERR_NO_PAGES)
    c = Cache([20, 40], 16, 1, 1, 64, BF16, seed=4, spare=1)
    for parents, new in (([2, 1], [20, 40]), ([0, -2], [20, 40]), ([0, 1], [20, -1]),
                         ([0, 1], [20, 16 * c.table.shape[1] + 1])):
        t, ref, _ = a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, ints(new), parents=ints(parents))
        assert status() == a.KVSEL_ERR_BAD_INDEX
        ok = [b for b in range(2) if 0 <= parents[b] < 2 and 0 <= new[b] <= 16 * c.table.shape[1]]
        for b in range(2):
            want = -(-new[b] // 16) if b in ok else 0
            assert t[b, :want].tolist() == c.table[b, :want].tolist() and (t[b, want:] == -1).all()
        assert ref.sum().item() == sum(-(-new[b] // 16) for b in ok)
    bad = c.table.clone()
    bad[1, 0] = -3
    t, _, _ = a.kvsel_pages_update(c.K, c.V, bad, c.dlens, c.dlens)
    assert status() == a.KVSEL_ERR_BAD_INDEX
    assert t[1].tolist()[0] == -1 and t[1].tolist()[1:3] == c.table[1].tolist()[1:3]


# ---------------------------------------------------------------------------

def test_a_served_request_from_prompt_to_samples():
    """Two prompts are rotated and written into pages and, packed, selected from; their caches
    are cut in place and their tail pages freed; each is forked into samples, and the samples
    append tokens and attend for three steps. Checked against fp64 rows kept per sequence."""
    a = api()
    gen = torch.Generator().manual_seed(11)
    L, H, Hkv, D, ps, W, C = 2, 4, 2, 64, 16, 8, 70
    lens = [333, 60]
    offs = [0, 333, 393]
    T = offs[-1]
    q, k, v = (normal(gen, BF16, L, T, h, D) for h in (H, Hkv, Hkv))
    qw, kw = (normal(gen, BF16, L, D) * 0.1 + 1 for _ in range(2))
    freq, scale = a.kvsel_rope_frequencies(D, 10000.0, a.KVSEL_ROPE_PARTS, 4.0, 256)
    rope = dict(q_weight=qw, k_weight=kw, inv_freq=freq.to(DEV), scale=scale)
    positions = ints(list(range(333)) + list(range(60)))
    # packed: the scoring reads it
    Kp, Vp = (torch.empty((L, T, 1, Hkv, D), dtype=BF16, device=DEV) for _ in range(2))
    flat = torch.arange(T, dtype=torch.int32, device=DEV)
    qr = a.kvsel_paged_append(q, k, v, Kp, Vp, flat, positions=positions, **rope)
    # paged: tables first
    P, width = 64, 24
    K, V = (torch.zeros((L, P, ps, Hkv, D), dtype=BF16, device=DEV) for _ in range(2))
    empty = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    table, ref, free = a.kvsel_pages_update(K, V, empty, ints([0, 0]), ints(lens))
    seqs = ints([0] * 333 + [1] * 60)
    assert torch.equal(a.kvsel_paged_append(q, k, v, K, V, positions, positions=positions, table=table,
                                            seqs=seqs, **rope), qr)
    assert free.item() == P - 21 - 4 and status() == 0
    # selection on the packed cache, cut of the pages
    win = torch.cat([qr[:, offs[b + 1] - W:offs[b + 1]] for b in range(2)], dim=1).contiguous()
    idx, out_k, out_v = a.kvsel_snapkv_grouped(win, Kp.squeeze(2), Vp.squeeze(2), offs, W, C, 0, 7)
    kept = [min(n, C) for n in lens]
    keep_offsets = ints([0, kept[0], sum(kept)])
    a.kvsel_paged_compact(K, V, table, ints(lens), idx, keep_offsets, C, ref=ref)
    table, ref, free = a.kvsel_pages_update(K, V, table, ints(lens), ints(kept))
    assert free.item() == P - 5 - 4 and status() == 0
    # what each sequence holds, in fp64: the selection's own gathered rows, in any order
    rows = [[f64(t[:, o:o + n]) for t in (out_k, out_v)] for o, n in ((0, C), (C, 60))]
    parents, logical, phys = [0, 0, 0, 1, 1], [333] * 3 + [60] * 2, [70] * 3 + [60] * 2
    rows = [[x.copy() for x in rows[p]] for p in parents]
    have = ints(kept)
    for step in range(3):
        table, ref, free = a.kvsel_pages_update(K, V, table, have, ints([n + 1 for n in phys]),
                                                parents=ints(parents))
        qn, kn, vn = (normal(gen, BF16, L, 5, h, D) for h in (H, Hkv, Hkv))
        qn = a.kvsel_paged_append(qn, kn, vn, K, V, ints(phys), positions=ints(logical), table=table, **rope)
        phys, logical = [n + 1 for n in phys], [n + 1 for n in logical]
        have = ints(phys)
        out, lse = a.kvsel_paged_attention(qn, K, V, table, have)
        assert status() == 0
        t = table.cpu().numpy()
        Kc, Vc = f64(K), f64(V)
        for b in range(5):
            j = phys[b] - 1                                  # the row just written
            new = [x[:, t[b, j // ps], j % ps] for x in (Kc, Vc)]
            np.testing.assert_array_equal(new[1], f64(vn)[:, b])
            rows[b] = [np.concatenate([r, n[:, None]], axis=1) for r, n in zip(rows[b], new)]
            for l in range(L):                                # the same set of rows, any order
                for x, pool in zip(rows[b], (Kc, Vc)):
                    got = pg.rows_of(pool[l], t[b], phys[b])
                    for h in range(Hkv):
                        key = lambda z: z[np.lexsort(z.T)]  # noqa: E731
                        np.testing.assert_array_equal(key(got[:, h]), key(x[l, :, h]))
        o, z, ob, zb = pg.attention(f64(qn), Kc, Vc, t, phys)
        assert (np.abs(f64(out) - o) <= ob).all() and (np.abs(f64(lse) - z) <= zb).all()
        # the samples of a prompt change places, and one ends for another
        parents = [2, 0, 0, 4, 3]
        rows = [[x.copy() for x in rows[p]] for p in parents]
        phys, logical = [phys[p] for p in parents], [logical[p] for p in parents]
    held = [x for row in table.cpu().tolist() for x in row if x >= 0]
    assert ref.tolist() == [held.count(x) for x in range(P)]


def test_updates_and_cuts_replay_from_a_graph():
    """Captured bookkeeping, append, attention and cut: replayed with new lengths, and two
    graphs with workspaces of their own."""
    a = api()
    c = Cache([37, 90], 16, 1, 2, 64, F32, seed=12, spare=20)
    new, parents = ints([38, 91]), ints([0, 1])
    rng = np.random.default_rng(1)
    idx = torch.stack([torch.tensor(rng.permutation(37)[:20]), torch.tensor(rng.permutation(37)[:20])],
                      dim=1).to(torch.int32)
    idx2 = torch.stack([torch.tensor(rng.permutation(90)[:41]) for _ in range(2)], dim=1).to(torch.int32)
    keep = torch.cat([idx, idx2])[None].to(DEV)
    offs = ints([0, 20, 61])
    K0, V0 = c.K.clone(), c.V.clone()

    def both():
        t, ref, free = a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, new, parents=parents)
        pos = a.kvsel_paged_compact(c.K, c.V, c.table, c.dlens, keep, offs, 41, ref=ref)
        return t, ref, free, pos

    eager = both()
    assert status() == 0
    after = c.K.clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both())
        graphs.append(g)
    for g, o in zip(graphs, outs):
        c.K.copy_(K0), c.V.copy_(V0)
        g.replay()
        assert status() == 0
        for x, y in zip(o, eager):
            assert torch.equal(x, y)
        assert torch.equal(torch.nan_to_num(c.K), torch.nan_to_num(after))
    parents.copy_(ints([1, 1]))
    new.copy_(ints([91, 92]))
    c.K.copy_(K0), c.V.copy_(V0)
    for g, o in zip(graphs, outs):
        g.replay()
        table, ref, free, _ = pg.update(c.table.tolist(), c.lens, [1, 1], [91, 92], c.P, 16)
        assert o[0].tolist() == table and o[1].tolist() == ref and o[2].item() == free
        assert status() == a.KVSEL_ERR_SHARED_PAGE        # both go on from sequence 1: it cannot be cut


def test_pages_beyond_four_gigabytes():
    """Every call on the last pages of a 5 GB pool against the same call on a small one."""
    a = api()
    P, ps, Hkv, D = 80000, 16, 16, 128
    gen = torch.Generator().manual_seed(50)
    K, V = (torch.zeros((P, ps, Hkv, D), dtype=BF16, device=DEV) for _ in range(2))
    assert K.nbytes > 4 << 30
    far = [P - 1, P - 7, P - 3]
    rows = [normal(gen, BF16, 3, ps, Hkv, D) for _ in range(2)]
    K[far], V[far] = rows
    k, v = torch.zeros((12, ps, Hkv, D), dtype=BF16, device=DEV), torch.zeros((12, ps, Hkv, D), dtype=BF16,
                                                                               device=DEV)
    near = [11, 5, 9]
    k[near], v[near] = rows
    q = normal(gen, BF16, 1, 32, D)
    new = [normal(gen, BF16, 1, h, D) for h in (32, Hkv, Hkv)]
    idx = torch.stack([torch.randperm(40, generator=gen)[:20] for _ in range(Hkv)], dim=1).to(torch.int32).to(DEV)
    got = []
    for pool, pages in (((K, V), far), ((k, v), near)):
        table = ints([pages + [-1]])
        r = [a.kvsel_paged_append(*new, *pool, ints([40]), table=table)]
        r += a.kvsel_paged_attention(q, *pool, table, ints([41]))
        r.append(a.kvsel_paged_compact(*pool, table, ints([40]), idx, ints([0, 20]), 20))
        r += [x[pages].clone() for x in pool]
        t, ref, free = a.kvsel_pages_update(*pool, table, ints([20]), ints([21, 21]), parents=ints([0, 0]))
        assert status() == 0
        assert t.tolist() == [pages[:2] + [-1, -1], [pages[0], 0, -1, -1]]
        assert free.item() == pool[0].shape[0] - 3
        r += [x[0, :4].clone() for x in pool]          # the copied rows
        got.append(r)
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert bool(got[0][-1].any())


def test_binding_checks():
    a = api()
    c = Cache([20], 16, 2, 2, 64, BF16, seed=1)
    q = torch.zeros((2, 1, 4, 64), dtype=BF16, device=DEV)
    for bad in (lambda: a.kvsel_paged_attention(q.float(), c.K, c.V, c.table, c.dlens),
                lambda: a.kvsel_paged_attention(q[:1], c.K, c.V, c.table, c.dlens),
                lambda: a.kvsel_paged_attention(q, c.K, c.V[:, :, :, :1], c.table, c.dlens),
                lambda: a.kvsel_paged_attention(q, c.K.transpose(2, 3), c.V.transpose(2, 3), c.table, c.dlens),
                lambda: a.kvsel_paged_attention(q, c.K, c.V, c.table.long(), c.dlens),
                lambda: a.kvsel_paged_attention(q, c.K, c.V, c.table.cpu(), c.dlens),
                lambda: a.kvsel_paged_attention(q.transpose(2, 3), c.K, c.V, c.table, c.dlens),
                lambda: a.kvsel_paged_attention(q, c.K.half(), c.V.half(), c.table, c.dlens),
                lambda: a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, c.dlens, ref=c.dlens),
                lambda: a.kvsel_paged_append(q, None, q, c.K, c.V, c.dlens)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(a.KvselError):
        a.kvsel_paged_attention(q[:, :, :3].contiguous(), c.K, c.V, c.table, c.dlens)
    small = torch.empty(1, dtype=torch.uint8, device=DEV)
    with pytest.raises(a.KvselError):
        a.kvsel_pages_update(c.K, c.V, c.table, c.dlens, c.dlens, workspace=small)
    assert status() == 0
