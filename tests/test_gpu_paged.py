"""The paged-cache calls on the GPU against 64-bit references: norms and
rotation, append, decode, prefill, and a run of them as a server makes it."""
import random

import pytest
import torch

import block_sparse_long_qsa_b200 as qsa
import paged_util as U

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
HEADS = [(24, 2, 256), (7, 7, 128), (28, 4, 128), (16, 16, 64), (40, 1, 64), (64, 1, 128), (17, 1, 256)]


def randn(g, dt, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float32).to(dt).cuda()


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def ok(ws):
    torch.cuda.synchronize()
    return qsa.qsa_check_device_error(ws)


# ------------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("T", [1, 2, 5, 67])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("heads,rope", [((24, 2, 256), 64), ((7, 7, 128), 128), ((16, 16, 64), 32), ((40, 1, 64), 64),
                                        ((24, 2, 256), 256), ((28, 4, 128), 16), ((3, 3, 128), 0)])
def test_norm_rope(heads, rope, dt, T):
    hq, hk, D = heads
    g = gen(T)
    p = qsa.layer_params(hq, hk, D, dtype=dt, rope_dim=rope)
    qkv = randn(g, dt, T, hq + 2 * hk, D)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    qw, kw = randn(g, dt, D), randn(g, dt, D)
    qo, ko = torch.empty(T, hq, D, dtype=dt, device="cuda"), torch.empty(T, hk, D, dtype=dt, device="cuda")
    qsa.qsa_norm_rope(p, T, 1000003, q, k, qw, kw, qo, ko)
    pos = 1000003 + torch.arange(T, device="cuda")[None]
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        U.check_norm_rope(got, *U.norm_rope64(p, x, w, pos), dt)


def test_norm_rope_and_append_of_many_tokens():
    """Enough tokens for a warp a token, ragged."""
    T, hq, hk, D, page = 3300, 6, 2, 128, 16
    p = qsa.layer_params(hq, hk, D)
    g = gen(13)
    qkv = randn(g, BF, T, hq + 2 * hk, D)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    qw, kw = randn(g, BF, D), randn(g, BF, D)
    qo, ko = torch.empty(T, hq, D, dtype=BF, device="cuda"), torch.empty(T, hk, D, dtype=BF, device="cuda")
    qsa.qsa_norm_rope(p, T, 5, q, k, qw, kw, qo, ko)
    pos = 5 + torch.arange(T, device="cuda")[None]
    U.check_norm_rope(qo, *U.norm_rope64(p, q, qw, pos), BF)
    U.check_norm_rope(ko, *U.norm_rope64(p, k, kw, pos), BF)
    cached, new = [5, 0, -1, 900], [1000, 1, 299, 1990]
    cache = U.Cache(p, [max(c, 0) + n for c, n in zip(cached, new)], page, BF, "cuda", "head")
    cu = torch.tensor([0, 1000, 1001, 1300, 3290], dtype=torch.int32, device="cuda")
    cl = torch.tensor(cached, dtype=torch.int32, device="cuda")
    ws = qsa.paged_workspace(p, 4, T)
    qo.fill_(5)
    qsa.qsa_paged_append(p, cache.kv, 4, T, cu, cl, k, v, ws, q=q, q_out=qo, q_weight=qw, k_weight=kw)
    assert ok(ws) == 0
    for b in (0, 1, 3):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        at = cached[b] + torch.arange(new[b], device="cuda")
        pg, sl = cache.slots(b, at)
        U.check_norm_rope(qo[rows], *U.norm_rope64(p, q[rows], qw, at[None]), BF)
        U.check_norm_rope(cache.k[pg, sl], *U.norm_rope64(p, k[rows], kw, at[None]), BF)
        assert torch.equal(cache.v[pg, sl], v[rows])
    assert bool((qo[1001:1300] == 5).all()) and bool((qo[3290:] == 5).all())


@pytest.mark.parametrize("rope,section", [(64, (11, 11, 10)), (64, (16, 8, 8)), (128, (24, 20, 20)), (32, (16, 0, 0)), (64, (21, 0, 11)), (128, (22, 22, 20))])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_three_axes(rope, section, interleaved):
    T, hq, hk, D = 33, 4, 2, 128
    g = gen(3)
    p = qsa.layer_params(hq, hk, D, rope_dim=rope, rope_axes=3, rope_section=section, rope_interleaved=interleaved)
    q, k, qw = randn(g, BF, T, hq, D), randn(g, BF, T, hk, D), randn(g, BF, D)
    pos = torch.randint(0, 1 << 21, (3, T), generator=g, dtype=torch.int32).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    qsa.qsa_norm_rope(p, T, 0, q, k, qw, None, qo, ko, positions=pos)
    U.check_norm_rope(qo, *U.norm_rope64(p, q, qw, pos), BF)
    U.check_norm_rope(ko, *U.norm_rope64(p, k, None, pos), BF)         # no weight: no norm
    one = qsa.layer_params(hq, hk, D, rope_dim=rope)                   # a text token: one position on all axes
    same = torch.arange(T, dtype=torch.int32, device="cuda").expand(3, T).contiguous()
    a, b = torch.empty_like(q), torch.empty_like(q)
    qsa.qsa_norm_rope(p, T, 0, q, None, qw, None, a, None, positions=same)
    qsa.qsa_norm_rope(one, T, 0, q, None, qw, None, b, None)
    assert torch.equal(a, b)


@pytest.mark.parametrize("centred", [0, 1])
@pytest.mark.parametrize("pos0", [0, (1 << 31) - 10])
def test_norm_rope_yarn_and_far_positions(pos0, centred):
    T, hq, hk, D = 9, 6, 2, 256
    g = gen(5)
    p = qsa.layer_params(hq, hk, D, rope_dim=64, yarn_factor=4.0, norm_zero_centred=centred, norm_eps=1e-3)
    k, kw = randn(g, BF, T, hk, D) * 1e-2, randn(g, BF, D)
    ko = torch.empty_like(k)
    qsa.qsa_norm_rope(p, T, pos0, None, k, None, kw, None, ko)
    pos = (pos0 + torch.arange(T, device="cuda"))[None]
    U.check_norm_rope(ko, *U.norm_rope64(p, k, kw, pos), BF)


def test_norm_rope_in_place_and_rows_behind():
    T, hq, hk, D = 11, 24, 2, 256
    g = gen(6)
    p = qsa.layer_params(hq, hk, D)
    q, k, w = randn(g, BF, T + 3, hq, D), randn(g, BF, T + 3, hk, D), randn(g, BF, D)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    qsa.qsa_norm_rope(p, T, 7, q, k, w, w, qo, ko)
    q2, k2 = q.clone(), k.clone()
    qsa.qsa_norm_rope(p, T, 7, q2, k2, w, w, q2, k2)
    assert torch.equal(q2[:T], qo[:T]) and torch.equal(k2[:T], ko[:T])
    assert torch.equal(q2[T:], q[T:]) and torch.equal(k2[T:], k[T:])
    qsa.qsa_norm_rope(p, 0, 7, q2, k2, w, w, q2, k2)                   # nothing to do
    zero = torch.zeros(1, hq, D, dtype=BF, device="cuda")
    qsa.qsa_norm_rope(p, 1, 7, zero, None, w, None, zero, None)        # eps keeps a zero row finite
    assert torch.equal(zero, torch.zeros_like(zero))


# ------------------------------------------------------------------------ append
@pytest.mark.parametrize("layout", ["token", "head", "beside"])
@pytest.mark.parametrize("page", [1, 3, 16, 48])
@pytest.mark.parametrize("heads,dt", [((24, 2, 256), BF), ((7, 7, 128), FP), ((40, 1, 64), BF)])
def test_append(heads, dt, page, layout):
    hq, hk, D = heads
    g = gen(page)
    p = qsa.layer_params(hq, hk, D, dtype=dt, rope_dim=32)
    cached, new = [0, 17, -1, 5, 40, 1], [3, 1, 4, 0, 33, 1]          # a padding and an empty sequence among them
    lens = [max(c, 0) + n for c, n in zip(cached, new)]
    cache = U.Cache(p, lens, page, dt, "cuda", layout)
    B, T = len(new), sum(new) + 3                                      # three rows behind the last sequence
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    cl = torch.tensor(cached, dtype=torch.int32, device="cuda")
    qkv = randn(g, dt, T, hq + 2 * hk, D)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    qw, kw = randn(g, dt, D), randn(g, dt, D)
    qo = torch.full((T, hq, D), 5.0, dtype=dt, device="cuda")
    ws = qsa.paged_workspace(p, B, T)
    qsa.qsa_paged_append(p, cache.kv, B, T, cu, cl, k, v, ws, q=q, q_out=qo, q_weight=qw, k_weight=kw)
    assert ok(ws) == 0
    written = torch.zeros(cache.k.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(B):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        if cached[b] < 0:
            assert bool((qo[rows] == 5).all())
            continue
        at = cached[b] + torch.arange(new[b], device="cuda")
        U.check_norm_rope(qo[rows], *U.norm_rope64(p, q[rows], qw, at[None]), dt)
        pg, sl = cache.slots(b, at)
        U.check_norm_rope(cache.k[pg, sl], *U.norm_rope64(p, k[rows], kw, at[None]), dt)
        assert torch.equal(cache.v[pg, sl], v[rows])
        written[pg, sl] = True
    assert bool((qo[T - 3:] == 5).all())
    assert bool(cache.k[~written].isnan().all()) and bool(cache.v[~written].isnan().all())


@pytest.mark.parametrize("layout", ["head", "beside"])
@pytest.mark.parametrize("T", [5, 3100])
@pytest.mark.parametrize("same", ["tensor", "start"])
def test_append_where_queries_and_keys_are_one_tensor(same, T, layout):
    """A shared projection (as many query as KV heads, or fewer KV heads from the
    same first element) with a weight each, into caches whose heads do not lie
    side by side; nothing behind q_out is written."""
    hq, hk, D, page = (4, 4, 128, 16) if same == "tensor" else (6, 2, 128, 16)
    p = qsa.layer_params(hq, hk, D)
    g = gen(T)
    cache = U.Cache(p, [7 + T], page, BF, "cuda", layout)
    x, v, qw, kw = randn(g, BF, T, hq, D), randn(g, BF, T, hk, D), randn(g, BF, D), randn(g, BF, D)
    qo = torch.full((3 * T, hq, D), 5.0, dtype=BF, device="cuda")
    cu, cl = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([0, T], [7]))
    ws = qsa.paged_workspace(p, 1, T)
    qsa.qsa_paged_append(p, cache.kv, 1, T, cu, cl, x[:, :hk], v, ws, q=x, q_out=qo, q_weight=qw, k_weight=kw)
    assert ok(ws) == 0
    at = 7 + torch.arange(T, device="cuda")
    U.check_norm_rope(qo[:T], *U.norm_rope64(p, x, qw, at[None]), BF)
    pg, sl = cache.slots(0, at)
    U.check_norm_rope(cache.k[pg, sl], *U.norm_rope64(p, x[:, :hk], kw, at[None]), BF)
    assert torch.equal(cache.v[pg, sl], v) and bool((qo[T:] == 5).all())


def test_append_one_token_each_without_queries():
    hq, hk, D, B = 8, 4, 128, 70
    p = qsa.layer_params(hq, hk, D, rope_axes=3)
    cached = [(b * 37) % 100 for b in range(B)]
    cache = U.Cache(p, [c + 1 for c in cached], 16, BF, "cuda")
    g = gen(9)
    k, v, kw = randn(g, BF, B, hk, D), randn(g, BF, B, hk, D), randn(g, BF, D)
    pos = torch.randint(0, 5000, (3, B), generator=g, dtype=torch.int32).cuda()
    ws = qsa.paged_workspace(p, B, B)
    cl = torch.tensor(cached, dtype=torch.int32, device="cuda")
    qsa.qsa_paged_append(p, cache.kv, B, B, None, cl, k, v, ws, k_weight=kw, positions=pos)
    assert ok(ws) == 0
    want, size = U.norm_rope64(p, k, kw, pos)
    for b in range(B):
        pg, sl = cache.slots(b, torch.tensor([cached[b]], device="cuda"))
        U.check_norm_rope(cache.k[pg, sl], want[b:b + 1], size[b:b + 1], BF)
        assert torch.equal(cache.v[pg, sl], v[b:b + 1])


def test_append_bad_pages_are_left_out_and_reported():
    p = qsa.layer_params(4, 2, 64, rope_dim=0)
    cache = U.Cache(p, [8, 8, 8], 4, BF, "cuda")
    cache.table[0, 1] = cache.k.shape[0]                               # one past the pool
    cache.table[1, 1] = -1
    g = gen(1)
    k, v = randn(g, BF, 12, 2, 64), randn(g, BF, 12, 2, 64)
    cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")
    ws = qsa.paged_workspace(p, 3, 12)
    for cl, good in [([2, 2, 2], [(0, 2), (1, 2), (2, 4)]), ([100, 0, 0], [(1, 4), (2, 4)])]:
        cache.k.fill_(float("nan"))
        cache.v.fill_(float("nan"))
        qsa.qsa_paged_append(p, cache.kv, 3, 12, cu, torch.tensor(cl, dtype=torch.int32, device="cuda"), k, v, ws)
        assert ok(ws) == 7                                             # QSA_ERR_DEVICE_BOUNDS, then cleared
        assert ok(ws) == 0
        assert int((~cache.k[..., 0].isnan()).sum()) == 2 * sum(n for _, n in good)
        for b, n in good:
            at = torch.arange(cl[b], cl[b] + n, device="cuda")
            pg, sl = cache.slots(b, at)
            assert torch.equal(cache.k[pg, sl], k[4 * b:4 * b + n]) and torch.equal(cache.v[pg, sl], v[4 * b:4 * b + n])


# --------------------------------------------------------------------- attention
def batch(p, cached, new, page, dt, layout="token", seed=0, spread=1.0):
    """A cache that holds all tokens' keys and values, and the new tokens' queries."""
    g = gen(seed)
    needed = [U.needed_pages(p, c, c + n - 1, page) if c >= 0 and n else [] for c, n in zip(cached, new)]
    lens = [max(c, 0) + n for c, n in zip(cached, new)]
    cache = U.Cache(p, lens, page, dt, "cuda", layout, seed, needed=needed)
    for b, need in enumerate(needed):
        for j in need:
            lo, hi = j * page, min((j + 1) * page, lens[b])
            cache.fill(b, lo, hi, spread * randn(g, dt, hi - lo, p.n_kv_heads, p.head_dim),
                       randn(g, dt, hi - lo, p.n_kv_heads, p.head_dim))
    q = randn(g, dt, sum(new), p.n_q_heads, p.head_dim)
    cl = torch.tensor(cached, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    return cache, q, cl, cu


def check_batch(p, cache, cached, new, q, out, lse, dt, tokens=None):
    row = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        for i in range(n):
            if c >= 0 and (tokens is None or i in tokens(n)):
                keys = U.visible(p, c + i).cuda()
                k, v = cache.rows(b, keys)
                U.check_row(out[row + i], None if lse is None else lse[row + i], U.attend64(p, q[row + i], k, v), dt)
        row += n


def run_decode(p, cache, q, cl, ws=None):
    B = q.shape[0]
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, dtype=torch.float32, device="cuda")
    ws = qsa.paged_workspace(p, B, B) if ws is None else ws
    qsa.qsa_paged_decode(p, cache.kv, B, cl, q, out, ws, lse=lse)
    return out, lse, ws


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dt,page,layout", [(BF, 16, "token"), (FP, 48, "head"), (BF, 1, "beside")])
def test_decode(heads, dt, page, layout):
    p = qsa.layer_params(*heads, dtype=dt)
    cached = [0, 1, 14, 15, 16, 63, 64, 200, 1025, -1, 511]
    cache, q, cl, _ = batch(p, cached, [1] * len(cached), page, dt, layout)
    out, lse, ws = run_decode(p, cache, q, cl)
    assert ok(ws) == 0
    check_batch(p, cache, cached, [1] * len(cached), q, out, lse, dt)
    assert bool((out[9] == 9).all()) and bool((lse[9] == 9).all())     # padding: left as it was


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 64), (100, 300), (4096, 4)])
@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128), (16, 16, 64)])
def test_decode_window(heads, window, sinks):
    """Pages that hold no visible key have no entry in the table."""
    p = qsa.layer_params(*heads, window=window, n_sinks=sinks)
    cached = [0, 1, window - 1, window, window + 1, window + sinks, window + sinks + 1, 3 * window + 517, 5000]
    cache, q, cl, _ = batch(p, cached, [1] * len(cached), 16, BF, seed=window)
    out, lse, ws = run_decode(p, cache, q, cl)
    assert ok(ws) == 0
    check_batch(p, cache, cached, [1] * len(cached), q, out, lse, BF)


@pytest.mark.parametrize("heads", [(24, 2, 256), (7, 7, 128)])
def test_decode_one_long_sequence_and_many_short(heads):
    """Both ends of the split: one sequence over all SMs, and many to an SM."""
    p = qsa.layer_params(*heads)
    for cached in ([20011], [(b * 29) % 83 for b in range(300)], [9000] + [3] * 40 + [-1] * 5 + [700]):
        cache, q, cl, _ = batch(p, cached, [1] * len(cached), 64, BF)
        out, lse, ws = run_decode(p, cache, q, cl)
        assert ok(ws) == 0
        check_batch(p, cache, cached, [1] * len(cached), q, out, lse, BF)
        again, lse2, _ = run_decode(p, cache, q, cl, ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)      # sums in one order


@pytest.mark.parametrize("dt", [BF, FP])
def test_decode_large_scores(dt):
    """Scores of some hundreds: the running maximum rises along the way."""
    p = qsa.layer_params(24, 2, 256, dtype=dt, softmax_scale=1.0)
    cached = [2000, 77]
    cache, q, cl, _ = batch(p, cached, [1, 1], 16, dt, spread=4.0)
    out, lse, ws = run_decode(p, cache, q, cl)
    assert ok(ws) == 0
    check_batch(p, cache, cached, [1, 1], q, out, lse, dt)


def test_decode_bad_pages_are_masked_and_reported():
    p = qsa.layer_params(24, 2, 256)
    cached = [100, 100, 30, 5]
    cache, q, cl, _ = batch(p, cached, [1] * 4, 16, BF)
    bad = cache.table.clone()
    cache.table[0, 2] = 1 << 30                                        # keys 32 .. 47 of sequence 0
    cache.table[2] = -1                                                # all of sequence 2
    out, lse, ws = run_decode(p, cache, q, cl)
    assert ok(ws) == 7 and ok(ws) == 0
    cache.table.copy_(bad)
    keys = torch.cat([torch.arange(32), torch.arange(48, 101)]).cuda()
    U.check_row(out[0], lse[0], U.attend64(p, q[0], *cache.rows(0, keys)), BF)
    assert bool((out[2] == 0).all()) and bool((lse[2] == -float("inf")).all())
    for b in (1, 3):
        U.check_row(out[b], lse[b], U.attend64(p, q[b], *cache.rows(b, U.visible(p, cached[b]).cuda())), BF)
    # a length past the table: what the table holds
    cl2 = torch.tensor([100, 10 ** 6, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out, lse, ws = run_decode(p, cache, q, cl2)
    assert ok(ws) == 7
    U.check_row(out[0], lse[0], U.attend64(p, q[0], *cache.rows(0, U.visible(p, 100).cuda())), BF)


def test_decode_captured_follows_lengths():
    """A graph of append and decode replayed at growing lengths, a sequence leaving on the way."""
    hq, hk, D, B, page = 24, 2, 256, 5, 16
    p = qsa.layer_params(hq, hk, D)
    cache = U.Cache(p, [400] * B, page, BF, "cuda")
    g = gen(2)
    start = [0, 15, 16, 200, 333]
    for b, n in enumerate(start):
        cache.fill(b, 0, n, randn(g, BF, n, hk, D), randn(g, BF, n, hk, D))
    cl = torch.tensor(start, dtype=torch.int32, device="cuda")
    q, k, v = randn(g, BF, B, hq, D), randn(g, BF, B, hk, D), randn(g, BF, B, hk, D)
    qo, out = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(B, hq, device="cuda")
    ws = qsa.paged_workspace(p, B, B)

    def step(s):
        qsa.qsa_paged_append(p, cache.kv, B, B, None, cl, k, v, ws, q=q, q_out=qo, stream=s)
        qsa.qsa_paged_decode(p, cache.kv, B, cl, qo, out, ws, lse=lse, stream=s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = cl.clone()
    cl.fill_(-1)                                                       # warm up on nothing
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    cl.copy_(keep)
    for i in range(20):
        for t in (q, k, v):
            t.copy_(randn(g, BF, *t.shape))
        graph.replay()
        lens = cl.tolist()
        check_batch(p, cache, lens, [1] * B, qo, out, lse, BF)
        cl += (cl >= 0).int()
        if i == 9:
            cl[3] = -1
    assert ok(ws) == 0


def test_offsets_past_32_bits():
    """Pages and rows more than 2^31 elements into the pool."""
    hq, hk, D, page = 24, 2, 256, 64
    p = qsa.layer_params(hq, hk, D)
    n_pages = (1 << 31) // (page * hk * D) + 9                         # 4.3 GB of keys, as much of values
    k = torch.empty(n_pages, page, hk, D, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    ids = [n_pages - 1, 0, n_pages - 2]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    g = gen(4)
    n = 3 * page
    kn, vn, q = randn(g, BF, n, hk, D), randn(g, BF, n, hk, D), randn(g, BF, n, hq, D)
    kv = qsa.PagedKV(k, v, table)
    ws = qsa.paged_workspace(p, 1, n)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cl = torch.zeros(1, dtype=torch.int32, device="cuda")
    plain = qsa.layer_params(hq, hk, D, rope_dim=0)
    qsa.qsa_paged_append(plain, kv, 1, n, cu, cl, kn, vn, ws)
    assert torch.equal(k[ids].flatten(0, 1), kn) and torch.equal(v[ids].flatten(0, 1), vn)
    out, lse = torch.zeros_like(q), torch.zeros(n, hq, device="cuda")
    qsa.qsa_paged_prefill(p, kv, 1, n, cu, cl, q, out, ws, lse=lse)
    for i in (0, 63, 64, 130, n - 1):
        U.check_row(out[i], lse[i], U.attend64(p, q[i], kn[:i + 1].double(), vn[:i + 1].double()), BF)
    o1, l1 = torch.zeros(1, hq, D, dtype=BF, device="cuda"), torch.zeros(1, hq, device="cuda")
    qsa.qsa_paged_decode(p, kv, 1, torch.tensor([n - 1], dtype=torch.int32, device="cuda"), q[n - 1:], o1, ws, lse=l1)
    U.check_row(o1[0], l1[0], U.attend64(p, q[n - 1], kn.double(), vn.double()), BF)
    assert ok(ws) == 0


def run_prefill(p, cache, q, cl, cu, ws=None):
    B, T = cl.shape[0], q.shape[0]
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, dtype=torch.float32, device="cuda")
    ws = qsa.paged_workspace(p, B, T) if ws is None else ws
    qsa.qsa_paged_prefill(p, cache.kv, B, T, cu, cl, q, out, ws, lse=lse)
    return out, lse, ws


def some(n):
    return {0, 1, 9, 10, 11, n // 3, n // 2, n - 2, n - 1}


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dt,page,layout", [(BF, 16, "token"), (FP, 48, "head"), (BF, 1, "beside"), (FP, 128, "token")])
def test_prefill(heads, dt, page, layout):
    p = qsa.layer_params(*heads, dtype=dt)
    cached, new = [0, 3, 130, -1, 0, 1000, 127], [1, 200, 5, 7, 0, 40, 131]
    cache, q, cl, cu = batch(p, cached, new, page, dt, layout)
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    check_batch(p, cache, cached, new, q, out, lse, dt, some)
    pad = slice(int(cu[3]), int(cu[4]))
    assert bool((out[pad] == 9).all()) and bool((lse[pad] == 9).all())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 64), (100, 300), (1000, 4)])
@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128), (16, 16, 64)])
def test_prefill_window(heads, window, sinks):
    p = qsa.layer_params(*heads, window=window, n_sinks=sinks)
    cached, new = [0, 2 * window + 77, window, 0], [300, 130, 1, 2 * window + 9 if window < 500 else 3]
    cache, q, cl, cu = batch(p, cached, new, 16, BF, seed=window)
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    check_batch(p, cache, cached, new, q, out, lse, BF, some)


def hide(p, cache, cached, new):
    """NaN in every slot of the sequences' pages that no token of the call sees."""
    for b, (c, n) in enumerate(zip(cached, new)):
        if c < 0 or n == 0:
            continue
        seen = torch.zeros(cache.table.shape[1] * cache.page, dtype=torch.bool)
        for i in range(n):
            seen[U.visible(p, c + i)] = True
        pages = (cache.table[b] >= 0).cpu().nonzero().flatten()
        keys = (pages[:, None] * cache.page + torch.arange(cache.page)).flatten()
        pg, sl = cache.slots(b, keys[~seen[keys]].cuda())
        cache.k[pg, sl] = float("nan")
        cache.v[pg, sl] = float("nan")


@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128), (16, 16, 64)])
@pytest.mark.parametrize("page,layout", [(16, "token"), (48, "beside"), (64, "head"), (64, "beside"), (24, "token")])
@pytest.mark.parametrize("window,sinks", [(70, 0), (70, 5), (300, 17), (1000, 100)])
def test_slots_that_no_token_sees_may_hold_anything(heads, page, layout, window, sinks):
    """Pages of which the window or the sinks leave a part: the other slots are NaN."""
    p = qsa.layer_params(*heads, window=window, n_sinks=sinks)
    for cached, new in (([window + 333, 0, 50, 5003], [200, 131, 70, 30]), ([window + 333, 9, 5003], [3, 2, 1])):
        cache, q, cl, cu = batch(p, cached, new, page, BF, layout, seed=window)
        hide(p, cache, cached, new)
        out, lse, ws = run_prefill(p, cache, q, cl, cu)
        assert ok(ws) == 0
        check_batch(p, cache, cached, new, q, out, lse, BF, some)
        assert bool(out.isfinite().all())
    one = [1] * len(cached)
    cache, q, cl, _ = batch(p, cached, one, page, BF, layout, seed=window + 1)
    hide(p, cache, cached, one)
    out, lse, ws = run_decode(p, cache, q, cl)
    assert ok(ws) == 0
    check_batch(p, cache, cached, one, q, out, lse, BF)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dt,page", [(BF, 16), (FP, 48), (BF, 64)])
def test_prefill_keys_and_values_side_by_side(heads, dt, page):
    """Keys and values of a page side by side with a gap behind each row, in page
    sizes that go through tensor maps."""
    p = qsa.layer_params(*heads, dtype=dt)
    for cached, new in (([0, 3, 130, -1, 0, 1000, 127], [1, 200, 5, 7, 0, 40, 131]), ([3000, 20], [9, 2])):
        cache, q, cl, cu = batch(p, cached, new, page, dt, "beside")
        out, lse, ws = run_prefill(p, cache, q, cl, cu)
        assert ok(ws) == 0
        check_batch(p, cache, cached, new, q, out, lse, dt, some)


@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128)])
@pytest.mark.parametrize("window,sinks", [(100, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0)])
def test_window_and_sinks_of_any_size(heads, window, sinks):
    """The largest windows and sinks leave every key."""
    p = qsa.layer_params(*heads, window=window, n_sinks=sinks)
    cached, new = [700, 0, 130], [5, 300, 1]
    cache, q, cl, cu = batch(qsa.layer_params(*heads), cached, new, 64, BF)
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    check_batch(qsa.layer_params(*heads), cache, cached, new, q, out, lse, BF, some)
    out, lse, ws = run_decode(p, cache, q[:3].contiguous(), cl, ws)
    assert ok(ws) == 0
    check_batch(qsa.layer_params(*heads), cache, cached, [1] * 3, q[:3], out, lse, BF)


@pytest.mark.parametrize("heads,n", [((7, 7, 128), 300), ((16, 16, 64), 20), ((24, 2, 256), 60), ((24, 2, 256), 5)])
@pytest.mark.parametrize("window", [8, 2 ** 31 - 100, 2 ** 31 - 1])
@pytest.mark.parametrize("page", [64, 24])
def test_positions_past_31_bits(heads, n, window, page):
    """Positions that pass 2^31 lie past the table and are reported; their rows see
    the sinks and what a window of that size leaves of the table's keys."""
    p = qsa.layer_params(*heads, window=window, n_sinks=90)
    cache, q, _, cu = batch(qsa.layer_params(*heads), [2 * page - 1], [1], page, BF)
    g = gen(n)
    q = randn(g, BF, n, *heads[::2])
    kv = qsa.PagedKV(cache.k, cache.v, cache.table[:, :2])
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    far = 2 ** 31 - 1 - 3
    cl = torch.tensor([far], dtype=torch.int32, device="cuda")
    out, lse, ws = torch.empty_like(q), torch.empty(n, heads[0], device="cuda"), qsa.paged_workspace(p, 1, n)
    qsa.qsa_paged_prefill(p, kv, 1, n, cu, cl, q, out, ws, lse=lse)
    assert ok(ws) == 7
    for i in some(n):
        if i < n:
            keys = torch.arange(2 * page)
            keys = keys[(keys > far + i - window) | (keys < 90)].cuda()
            U.check_row(out[i], lse[i], U.attend64(p, q[i], *cache.rows(0, keys)), BF)


@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128)])
def test_offsets_past_the_tokens(heads):
    """Offsets beyond T count as T: nothing behind row T is read or written."""
    p = qsa.layer_params(*heads, rope_dim=0)
    hq, hk, D = heads
    cached, new = [40, 0], [30, 50]
    cache, q, cl, cu = batch(p, cached, new, 16, BF)
    wide = cu.clone()
    wide[2] = 5000
    out = torch.full((100, hq, D), 9.0, dtype=BF, device="cuda")
    lse = torch.full((100, hq), 9.0, device="cuda")
    ws = qsa.paged_workspace(p, 2, 80)
    k, v = (cache.rows(1, torch.arange(50).cuda())[i].to(BF) for i in (0, 1))
    k, v = (torch.cat([torch.zeros(30, hk, D, dtype=BF, device="cuda"), x]) for x in (k, v))
    cl2 = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    qsa.qsa_paged_append(p, cache.kv, 2, 80, wide, cl2, k, v, ws)
    qsa.qsa_paged_prefill(p, cache.kv, 2, 80, wide, cl, q, out, ws, lse=lse)
    assert ok(ws) == 0
    check_batch(p, cache, cached, new, q, out, lse, BF)
    assert bool((out[80:] == 9).all()) and bool((lse[80:] == 9).all())


def test_two_graphs_with_one_workspace():
    """Graphs of a chunk cut over the CTAs and of a decode that share a workspace, replayed in turn."""
    p = qsa.layer_params(24, 2, 256)
    cache, q, cl, cu = batch(p, [9000, 20], [9, 40], 16, BF)
    d_cache, d_q, d_cl, _ = batch(p, [5000, 3, 800], [1] * 3, 16, BF, seed=5)
    ws = qsa.paged_workspace(p, 3, q.shape[0])
    want, want_l, _ = run_prefill(p, cache, q, cl, cu, ws)
    d_want, d_want_l, _ = run_decode(p, d_cache, d_q, d_cl, ws)
    check_batch(p, cache, [9000, 20], [9, 40], q, want, want_l, BF)
    out, lse, d_out, d_lse = (torch.zeros_like(x) for x in (want, want_l, d_want, d_want_l))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        qsa.qsa_paged_prefill(p, cache.kv, 2, q.shape[0], cu, cl, q, out, ws, lse=lse)
    with torch.cuda.graph(graphs[1]):
        qsa.qsa_paged_decode(p, d_cache.kv, 3, d_cl, d_q, d_out, ws, lse=d_lse)
    for i in (0, 1, 1, 0, 0, 1):
        for t in (out, lse, d_out, d_lse):
            t.zero_()
        graphs[i].replay()
        graphs[1 - i].replay()
        assert torch.equal(out, want) and torch.equal(lse, want_l)
        assert torch.equal(d_out, d_want) and torch.equal(d_lse, d_want_l)
    assert ok(ws) == 0


def test_prefill_long_prefix_few_rows():
    """A short chunk over a long prefix."""
    p = qsa.layer_params(24, 2, 256)
    for cached, new in (([20011], [5]), ([9000, 12, 7001], [37, 3, 1])):
        cache, q, cl, cu = batch(p, cached, new, 64, BF)
        out, lse, ws = run_prefill(p, cache, q, cl, cu)
        assert ok(ws) == 0
        check_batch(p, cache, cached, new, q, out, lse, BF)
        again, lse2, _ = run_prefill(p, cache, q, cl, cu, ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def check_weights(q, k, v, scale, got, got_lse, dt, shift):
    """A row of queries [H][D] over keys and values [n][Hk][D], all visible, whose
    weights span more than the element type: each weight has an error of half a
    step, or, below the type's normal numbers, of half the smallest one, 2^-25 in
    fp16, of weights that the kernels hold 2^shift times as large (relative to the
    largest, whose sum is at least that); scores, sums and result as in check_row."""
    H, D = q.shape
    per = H // k.shape[1]
    k, v = k.repeat_interleave(per, 1), v.repeat_interleave(per, 1)
    s = torch.einsum("hd,nhd->hn", q.double(), k) * scale
    w = (s - s.logsumexp(1, keepdim=True)).exp()
    delta = 2 * D * 2.0 ** -24 * scale * torch.einsum("hd,nhd->hn", q.double().abs(), k.abs())   # of each score
    want = torch.einsum("hn,nhd->hd", w, v)
    shared = (w * delta).sum(1)                                        # of the sum, relative
    size = torch.einsum("hn,nhd->hd", w * (U.half_step(dt) + 2 * delta + 2 * shared[:, None] + (k.shape[0] + 64) * 2.0 ** -23), v.abs())
    low = 2.0 ** (-25 - shift) * v.abs().sum(0) + 2.0 ** -25 if dt == FP else 0.0
    err = (got.double() - want).abs()
    tol = U.half_step(dt) * want.abs() + size + low
    assert bool((err <= tol).all()), (float((err / want.abs()).max()), float((err - tol).max()))
    # log-sum-exp: the sum's relative error, the score of its maximum, log2 and the product
    lse = s.logsumexp(1)
    assert bool(((got_lse.double() - lse).abs() <= shared + delta.amax(1) + (k.shape[0] + 64) * 2.0 ** -23 + 2.0 ** -22 * (lse.abs() + 20)).all())


@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128), (16, 16, 64)])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("gap", [6.0, 13.0, 18.0])
def test_first_key_that_outweighs_the_others(heads, dt, gap):
    """A first key whose score lies `gap` above all others and whose value is zero,
    as models learn them: the result is the others' small weights alone."""
    hq, hk, D = heads
    p = qsa.layer_params(*heads, dtype=dt)
    n, g = 700, gen(int(gap))
    cache = U.Cache(p, [n] * 3, 16, dt, "cuda")
    u = torch.sign(torch.randn(D, generator=g)).cuda()
    for b in range(3):
        k, v = 0.05 * randn(g, dt, n, hk, D), 1 + 0.2 * randn(g, dt, n, hk, D)
        k[0], v[0] = (gap / D ** 0.5 * u).to(dt), 0
        cache.fill(b, 0, n, k, v)
    new = [9, 200, 1]                           # the last tokens of each sequence
    q = (u + 0.01 * randn(g, dt, sum(new), hq, D)).to(dt)
    cl, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n - m for m in new], [0, 9, 209, 210]))
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    last = torch.tensor([8, 208, 209], device="cuda")
    end = torch.full((3,), n - 1, dtype=torch.int32, device="cuda")
    d_out, d_lse, _ = run_decode(p, cache, q[last].contiguous(), end, ws)
    assert ok(ws) == 0
    for row, b, m in ((0, 0, n - 8), (8, 0, n), (9, 1, n - 199), (150, 1, n - 58), (208, 1, n), (209, 2, n)):
        k, v = cache.rows(b, torch.arange(m).cuda())
        check_weights(q[row], k, v, D ** -0.5, out[row], lse[row], dt, 7)
    for b in range(3):
        k, v = cache.rows(b, torch.arange(n).cuda())
        check_weights(q[last[b]], k, v, D ** -0.5, d_out[b], d_lse[b], dt, 15)


@pytest.mark.parametrize("dt", [BF, FP])
def test_prefill_large_scores(dt):
    p = qsa.layer_params(24, 2, 256, dtype=dt, softmax_scale=1.0)
    cached, new = [700, 0], [60, 300]
    cache, q, cl, cu = batch(p, cached, new, 16, dt, spread=4.0)
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    check_batch(p, cache, cached, new, q, out, lse, dt, some)


@pytest.mark.parametrize("heads", [(24, 2, 256), (33, 3, 128), (7, 7, 128), (17, 1, 64), (16, 16, 64)])
@pytest.mark.parametrize("cached,new", [([14882], [1]), ([9000], [300]), ([0], [2100]), ([19, 0, 2879, 1836, 0], [168, 22, 300, 16, 124])])
def test_prefill_gives_the_same_bits_every_time(heads, cached, new):
    """Row maxima that rise along the way, many times over: every run gives the same
    bits, and the rows are right.  (An O that is rescaled or read while products
    are still being added to it comes out differently now and then.)"""
    p = qsa.layer_params(*heads, softmax_scale=1.0)
    cache, q, cl, cu = batch(p, cached, new, 32, BF, seed=len(new))
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    check_batch(p, cache, cached, new, q, out, lse, BF, some)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        again, lse2, _ = run_prefill(p, cache, q, cl, cu, ws)
        wrong += (again != out).sum() + (lse2 != lse).sum()
    assert int(wrong) == 0 and ok(ws) == 0


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(seed):
    """Head layouts, pages, windows and lengths of any mix: some rows of each sequence
    against 64 bits, the same bits twice, rows behind and of padding left alone."""
    r = random.Random(seed)
    D, per, hk = r.choice([64, 128, 256]), r.choice([1, 2, 3, 7, 12, 16, 17, 33, 64]), r.choice([1, 2, 3, 8])
    hk, dt = min(hk, max(1, 128 // per)), r.choice([BF, FP])
    page = r.choice([1, 8, 16, 16, 32, 48, 64, 80, r.randint(1, 200)])
    p = qsa.layer_params(per * hk, hk, D, dtype=dt, window=r.choice([0, 0, r.randint(1, 40), r.randint(1, 2000)]),
                         n_sinks=r.choice([0, 4, r.randint(0, 200)]), softmax_scale=r.choice([0.0, 1.0]))
    B = r.choice([1, 1, 3, 12, 60])
    cached = [r.choice([-1, 0, r.randint(0, 300), r.randint(0, 3000 if B < 20 else 500)]) for _ in range(B)]
    new = [r.choice([0, 1, r.randint(0, 40), r.randint(0, 400 if B < 20 else 50)]) for _ in range(B)]
    cached[r.randrange(B)], new[r.randrange(B)] = r.choice([0, 9001]), r.choice([1, 5, 1500])
    layout, behind = r.choice(["token", "head", "beside"]), r.choice([0, 50])
    cache, q, cl, cu = batch(p, cached, new, page, dt, layout, seed)
    T = q.shape[0]
    q = torch.cat([q, torch.zeros(behind, *q.shape[1:], dtype=dt, device="cuda")])
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    check_batch(p, cache, cached, new, q, out, lse, dt, lambda n: {0, n - 1, r.randrange(n)})
    again, lse2, _ = run_prefill(p, cache, q, cl, cu, ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    row = 0
    for c, n in zip(cached, new):
        assert c >= 0 or bool((out[row:row + n] == 9).all())
        row += n
    assert row == T and bool((out[T:] == 9).all())
    cache, q, cl, _ = batch(p, cached, [1] * B, page, dt, layout, seed + 1000)
    out, lse, ws = run_decode(p, cache, q, cl)
    assert ok(ws) == 0
    check_batch(p, cache, cached, [1] * B, q, out, lse, dt)


def test_prefill_bad_pages_and_rows_behind():
    p = qsa.layer_params(24, 2, 256)
    cached, new = [50, 0, 30], [20, 40, 10]
    cache, q, cl, cu = batch(p, cached, new, 16, BF)
    good = cache.table.clone()
    cache.table[0, 1] = 1 << 29                                        # keys 16 .. 31 of sequence 0
    cache.table[2] = -3
    q2 = torch.cat([q, q[:6]])                                         # six rows behind the last sequence
    out, lse, ws = run_prefill(p, cache, q2, cl, cu)
    assert ok(ws) == 7 and ok(ws) == 0
    cache.table.copy_(good)
    for i in range(20):
        keys = torch.cat([torch.arange(16), torch.arange(32, 51 + i)]).cuda()
        U.check_row(out[i], lse[i], U.attend64(p, q[i], *cache.rows(0, keys)), BF)
    check_batch(p, cache, [-1, 0, -1], new, q, out, lse, BF)
    assert bool((out[60:70] == 0).all()) and bool((lse[60:70] == -float("inf")).all())
    assert bool((out[70:] == 9).all()) and bool((lse[70:] == 9).all())


def test_prefill_of_one_token_each_is_a_decode():
    p = qsa.layer_params(24, 2, 256, window=64, n_sinks=4)
    cached = [0, 5, 63, 64, 200, 1000]
    cache, q, cl, cu = batch(p, cached, [1] * 6, 16, BF)
    a, la, _ = run_decode(p, cache, q, cl)
    b, lb, _ = run_prefill(p, cache, q, cl, cu)
    assert float((a.double() - b.double()).abs().max()) < 2e-2 and float((la - lb).abs().max()) < 1e-4


@pytest.mark.parametrize("heads,cached,new", [
    ((24, 2, 256), [5000], [600]),                      # pairs of CTAs, tiles cut over them
    ((24, 2, 256), [0, 777], [3001, 40]),               # pairs, whole items
    ((24, 2, 256), [3000, 0, 20, 9001], [9, 1, 4, 2]),  # single CTAs, cut: few rows
    ((28, 4, 128), [0], [2501]),                        # single CTAs, whole items
    ((28, 4, 128), [4000, 0], [30, 300]),
    ((16, 16, 64), [100], [1300]),
    ((16, 16, 64), [8000], [3]),
    ((64, 1, 128), [33], [700]),
    ((24, 2, 256), [9000], [11]),                       # a pair with few rows in its second half, many pieces
    ((24, 2, 256), [100] * 47 + [12000], [21] * 48),    # pairs, more items than pairs, one of them long
    ((24, 2, 256), [50] * 100 + [15000, -1], [2] * 102),    # single CTAs, likewise, a padding sequence
    ((32, 8, 128), [0, 40] * 20 + [9000], [3] * 41),    # 656 items: no cut
    ((32, 8, 128), [0, 40] * 10 + [9000], [3, 1] * 10 + [1]),
    ((24, 2, 256), [0] * 30, [3, 70, 120] * 10)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
def test_prefill_ways_to_deal_the_tiles(heads, cached, new, window, sinks):
    """Each kernel and each way to deal the tiles to the CTAs, twice with the same bits."""
    p = qsa.layer_params(*heads, window=window, n_sinks=sinks)
    cache, q, cl, cu = batch(p, cached, new, 32, BF, seed=len(new))
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    check_batch(p, cache, cached, new, q, out, lse, BF, some)
    again, lse2, _ = run_prefill(p, cache, q, cl, cu, ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128)])
def test_window_past_the_table_leaves_zero_rows(heads):
    """Rows whose keys all lie past the table: zero, lse -inf, reported."""
    p = qsa.layer_params(*heads, window=8)
    cache, q, cl, cu = batch(p, [40], [4], 16, BF)
    far = torch.tensor([4096], dtype=torch.int32, device="cuda")
    out, lse, ws = run_prefill(p, cache, q, far, cu)
    assert ok(ws) == 7
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    out, lse, ws = run_decode(p, cache, q[:1].contiguous(), far, ws)
    assert ok(ws) == 7
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


def test_prefill_captured_follows_lengths():
    """A graph of append and prefill replayed with other lengths, offsets and pages."""
    hq, hk, D, B, T = 24, 2, 256, 3, 64
    p = qsa.layer_params(hq, hk, D)
    g = gen(3)
    cache = U.Cache(p, [500] * B, 16, BF, "cuda")
    for b in range(B):
        cache.fill(b, 0, 500, randn(g, BF, 500, hk, D), randn(g, BF, 500, hk, D))
    cl = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    q, k, v = randn(g, BF, T, hq, D), randn(g, BF, T, hk, D), randn(g, BF, T, hk, D)
    qo, out, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(T, hq, device="cuda")
    ws = qsa.paged_workspace(p, B, T)

    def step():
        qsa.qsa_paged_append(p, cache.kv, B, T, cu, cl, k, v, ws, q=q, q_out=qo)
        qsa.qsa_paged_prefill(p, cache.kv, B, T, cu, cl, qo, out, ws, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                          # warm up on nothing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for cached, new in (([0, 300, 17], [30, 1, 33]), ([400, -1, 0], [5, 20, 0]), ([1, 2, 3], [64, 0, 0])):
        for t in (q, k, v):
            t.copy_(randn(g, BF, *t.shape))
        out.fill_(9)
        cl.copy_(torch.tensor(cached))
        cu.copy_(torch.tensor([0] + list(torch.tensor(new).cumsum(0))))
        graph.replay()
        check_batch(p, cache, cached, new, qo, out, lse, BF)
        assert bool((out[sum(new):] == 9).all())
    assert ok(ws) == 0


def test_two_streams_with_a_workspace_each():
    """A decode and a prefill at the same time give what they give alone."""
    p = qsa.layer_params(24, 2, 256)
    cached, new = [3000, 700, 20], [50, 9, 300]
    cache, q, cl, cu = batch(p, cached, new, 16, BF)
    d_cache, d_q, d_cl, _ = batch(p, [9000, 100, 2000, 5] * 8, [1] * 32, 16, BF, seed=5)
    want, want_l, ws1 = run_prefill(p, cache, q, cl, cu)
    d_want, d_want_l, ws2 = run_decode(p, d_cache, d_q, d_cl)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        out, lse, d_out, d_lse = (torch.zeros_like(x) for x in (want, want_l, d_want, d_want_l))
        torch.cuda.synchronize()
        qsa.qsa_paged_prefill(p, cache.kv, 3, q.shape[0], cu, cl, q, out, ws1, lse=lse, stream=s1)
        qsa.qsa_paged_decode(p, d_cache.kv, 32, d_cl, d_q, d_out, ws2, lse=d_lse, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_l)
        assert torch.equal(d_out, d_want) and torch.equal(d_lse, d_want_l)
    assert ok(ws1) == 0 and ok(ws2) == 0


def test_shared_pages():
    """Sequences that share the pages of a common prefix."""
    p = qsa.layer_params(24, 2, 256)
    cached, new = [200, 200], [3, 40]
    cache, q, cl, cu = batch(p, cached, new, 16, BF)
    cache.table[1, :12] = cache.table[0, :12]           # 192 tokens in common
    out, lse, ws = run_prefill(p, cache, q, cl, cu)
    check_batch(p, cache, cached, new, q, out, lse, BF)
    out, lse, ws = run_decode(p, cache, q[:2].contiguous(), cl, ws)
    check_batch(p, cache, cached, [1, 1], q[:2], out, lse, BF)
    assert ok(ws) == 0


@pytest.mark.parametrize("heads", [(24, 2, 256), (28, 4, 128)])
@pytest.mark.parametrize("new", [[5], [400]])
def test_wait_that_runs_out_is_reported(heads, new):
    """Debug build: no CTA signals its first tile of scores; the waits run
    out (20 ms), the call ends with QSA_ERR_DEVICE_TIMEOUT, and the next is right."""
    from block_sparse_long_qsa_b200 import _build
    _build.build(debug=True)
    p = qsa.layer_params(*heads)
    cache, q, cl, cu = batch(p, [300], new, 64, BF)
    want, want_l, ws = run_prefill(p, cache, q, cl, cu)
    assert ok(ws) == 0
    prev = qsa.use_library(qsa.LIB_DEBUG_PATH)
    try:
        qsa.qsa_debug_inject(qsa.INJECT_PAGED_STALL)
        run_prefill(p, cache, q, cl, cu, ws)
        assert ok(ws) == 6
        out, lse, _ = run_prefill(p, cache, q, cl, cu, ws)
        assert ok(ws) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_l)
    finally:
        qsa.use_library(prev or qsa.LIB_PATH)


# ---------------------------------------------------------------- a run of them
def test_dense_layer_equals_qsa_prefill():
    """While the budget covers every block, QSA is dense causal attention: the
    paged calls give what qsa_prefill gives on the same tokens."""
    T = 1000
    g = gen(8)
    q, k, v = randn(g, BF, T, 24, 256), randn(g, BF, T, 2, 256), randn(g, BF, T, 2, 256)
    w = torch.softmax(torch.randn(T, 4, generator=g), -1).to(BF).cuda()
    r = qsa.prefill(q, k, v, randn(g, BF, T, 4, 128), w, randn(g, BF, T, 128), budget=512)
    p = qsa.layer_params()
    cache = U.Cache(p, [T], 64, BF, "cuda")
    ws = qsa.paged_workspace(p, 1, T)
    cu, cl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [0]))
    qo, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(T, 24, device="cuda")
    qsa.qsa_paged_append(p, cache.kv, 1, T, cu, cl, k, v, ws, q=q, q_out=qo)
    qsa.qsa_paged_prefill(p, cache.kv, 1, T, cu, cl, qo, out, ws, lse=lse)
    assert ok(ws) == 0 and qsa.qsa_check_device_error(r["ws"]) == 0
    want = r["out"].view(BF).double()
    diff = out.double() - want
    assert float(diff.abs().max()) < 2e-2 and float(diff.norm() / want.norm()) < 5e-3
    assert float((lse - r["lse"]).abs().max()) < 2e-2


def test_norms_feed_qsa_prefill():
    """With rope_dim 0 the normed queries and keys go into qsa_prefill, which rotates them."""
    T = 500
    g = gen(10)
    qkv = randn(g, BF, T, 28, 256)
    qw, kw = 0.1 * randn(g, BF, 256), 0.1 * randn(g, BF, 256)
    qn, kn = torch.empty(T, 24, 256, dtype=BF, device="cuda"), torch.empty(T, 2, 256, dtype=BF, device="cuda")
    qsa.qsa_norm_rope(qsa.layer_params(rope_dim=0), T, 0, qkv[:, :24], qkv[:, 24:26], qw, kw, qn, kn)
    w = torch.softmax(torch.randn(T, 4, generator=g), -1).to(BF).cuda()
    r = qsa.prefill(qn, kn, qkv[:, 26:].contiguous(), randn(g, BF, T, 4, 128), w, randn(g, BF, T, 128), budget=512)
    p = qsa.layer_params()
    pos = torch.arange(T, device="cuda")[None]
    qr, _ = U.norm_rope64(p, qkv[:, :24], qw, pos)
    kr, _ = U.norm_rope64(p, qkv[:, 24:26], kw, pos)
    torch.cuda.synchronize()
    # The calls round the normed and the rotated operands (two half steps of 2^-8
    # each for q and k): scores of about 1 move by 2^-6, outputs of about 1 by that
    # times their spread, and one rounding: below 3e-2.
    for i in (0, 1, 7, 250, 499):
        want, *_ = U.attend64(p, qr[i], kr[:i + 1], qkv[:i + 1, 26:].double())
        assert float((r["out"][i].view(BF).double() - want).abs().max()) < 3e-2


@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_serving_run(window, sinks):
    """Prompts in chunks, then decode steps, norms and three-axis positions on the
    way, against attention over everything in 64 bits."""
    hq, hk, D, page = 12, 2, 128, 16
    p = qsa.layer_params(hq, hk, D, rope_dim=64, rope_axes=3, window=window, n_sinks=sinks)
    prompt, steps = [70, 5, 133], 6
    B = len(prompt)
    total = [n + steps for n in prompt]
    cache = U.Cache(p, total, page, BF, "cuda")
    g = gen(12)
    qkv = [randn(g, BF, n, hq + 2 * hk, D) for n in total]
    qw, kw = 0.2 * randn(g, BF, D), 0.2 * randn(g, BF, D)
    pos = [torch.stack([torch.arange(n), torch.arange(n) // 3, torch.arange(n) % 7]).int().cuda() for n in total]
    ws = qsa.paged_workspace(p, B, sum(total))
    got = [torch.empty(n, hq, D, dtype=BF, device="cuda") for n in total]
    done = [0] * B

    def step(new):
        x = torch.cat([qkv[b][done[b]:done[b] + n] for b, n in enumerate(new)])
        ps = torch.cat([pos[b][:, done[b]:done[b] + n] for b, n in enumerate(new)], 1).contiguous()
        T = x.shape[0]
        cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
        cl = torch.tensor(done, dtype=torch.int32, device="cuda")
        qo = torch.empty(T, hq, D, dtype=BF, device="cuda")
        out = torch.empty_like(qo)
        qsa.qsa_paged_append(p, cache.kv, B, T, cu, cl, x[:, hq:hq + hk], x[:, hq + hk:], ws, q=x[:, :hq], q_out=qo,
                             q_weight=qw, k_weight=kw, positions=ps)
        if max(new) == 1:
            qsa.qsa_paged_decode(p, cache.kv, B, cl, qo, out, ws)
        else:
            qsa.qsa_paged_prefill(p, cache.kv, B, T, cu, cl, qo, out, ws)
        row = 0
        for b, n in enumerate(new):
            got[b][done[b]:done[b] + n] = out[row:row + n]
            done[b] += n
            row += n

    step([50, 5, 64])
    step([20, 0, 69])
    for _ in range(steps):
        step([1] * B)
    assert ok(ws) == 0
    for b in range(B):
        x = qkv[b]
        # the rounded queries and keys that the calls hand on (where a value lies on
        # a border of rounding they may differ by a step, 2^-7: as above)
        qr = U.norm_rope64(p, x[:, :hq], qw, pos[b])[0].to(BF)
        kr = U.norm_rope64(p, x[:, hq:hq + hk], kw, pos[b])[0].to(BF).double()
        for i in {0, 4, 49, 50, total[b] - steps - 1, total[b] - steps, total[b] - 1}:
            if i < total[b]:
                keys = U.visible(p, i).cuda()
                want, *_ = U.attend64(p, qr[i], kr[keys], x[keys][:, hq + hk:].double())
                assert float((got[b][i].double() - want).abs().max()) < 3e-2, (b, i)
