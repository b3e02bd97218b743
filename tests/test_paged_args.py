"""Argument checks of the paged-cache calls (no GPU: everything is refused on
the host before a launch), and the host arithmetic the kernels rely on."""
import ctypes
import math
import random

import pytest
import torch

import block_sparse_long_qsa_b200 as qsa
from block_sparse_long_qsa_b200 import _build

A = 1 << 20          # a 16-byte aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return qsa.load()


def kv_struct(**kw):
    c = qsa.qsa_paged_kv(A, 2 * A, 100, 16, 8, 16 * 512, 512, 256, 3 * A, 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BIG = 1 << 40


def call(name, p, kv=None, ws_bytes=BIG, **kw):
    L, P = qsa.load(), ctypes.byref(p)
    K = ctypes.byref(kv if kv is not None else kv_struct())
    d = dict(B=2, T=2, pos0=0, positions=None, cu=A, cl=A, q=A, q_ld=24 * 256, k=A, k_ld=512, v=A, v_ld=512, qw=A, kw=A,
             q_out=A, k_out=A, out=A, lse=A, ws=A)
    d.update(kw)
    g = d.get
    if name == "norm_rope":
        return L.qsa_norm_rope(P, g("T"), g("pos0"), g("positions"), g("q"), g("q_ld"), g("k"), g("k_ld"), g("qw"), g("kw"),
                               g("q_out"), g("k_out"), None)
    if name == "append":
        return L.qsa_paged_append(P, K, g("B"), g("T"), g("cu"), g("cl"), g("positions"), g("q"), g("q_ld"), g("k"),
                                  g("k_ld"), g("v"), g("v_ld"), g("qw"), g("kw"), g("q_out"), g("ws"), ws_bytes, None)
    if name == "decode":
        return L.qsa_paged_decode(P, K, g("B"), g("cl"), g("q"), g("out"), g("lse"), g("ws"), ws_bytes, None)
    return L.qsa_paged_prefill(P, K, g("B"), g("T"), g("cu"), g("cl"), g("q"), g("out"), g("lse"), g("ws"), ws_bytes, None)


CALLS = ["norm_rope", "append", "decode", "prefill"]
INVALID, UNSUPPORTED, MISALIGNED, SMALL = 1, 2, 3, 4


@pytest.mark.parametrize("name", CALLS)
def test_layer_checks(name):
    for kw, want in [(dict(head_dim=96), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED), (dict(n_kv_heads=7), INVALID),
                     (dict(n_q_heads=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_kv_heads=-2), INVALID),
                     (dict(n_q_heads=130), UNSUPPORTED), (dict(n_q_heads=2048, n_kv_heads=1024), UNSUPPORTED),
                     (dict(rope_dim=-16), INVALID), (dict(rope_dim=24), UNSUPPORTED), (dict(rope_dim=272), UNSUPPORTED),
                     (dict(rope_axes=2), UNSUPPORTED), (dict(rope_axes=3, rope_interleaved=2), INVALID),
                     (dict(rope_theta=1.0), INVALID), (dict(rope_theta=float("nan")), INVALID),
                     (dict(yarn_factor=-1.0), INVALID), (dict(yarn_factor=4.0, yarn_beta_fast=0.5), INVALID),
                     (dict(norm_eps=0.0), INVALID), (dict(norm_eps=float("inf")), INVALID),
                     (dict(norm_zero_centred=2), INVALID), (dict(softmax_scale=-1.0), INVALID),
                     (dict(softmax_scale=float("nan")), INVALID), (dict(window=-1), INVALID), (dict(n_sinks=-1), INVALID),
                     (dict(dtype=2), UNSUPPORTED)]:
        p = qsa.layer_params()
        for k, v in kw.items():
            setattr(p, k, v)
        assert call(name, p) == want, (kw, want)
    for sec in [(11, 11, 11), (-1, 17, 16), (0, 16, 17), (10, 10, 11)]:
        p = qsa.layer_params(rope_axes=3, rope_section=sec)
        assert call(name, p) == INVALID, sec


def test_sections():
    """Any three counts that sum to rope_dim / 2, interleaved or not."""
    n = ctypes.c_size_t()
    for sec in [(11, 11, 10), (32, 0, 0), (20, 12, 0), (0, 0, 32), (21, 0, 11)]:
        p = qsa.layer_params(rope_axes=3, rope_section=sec)
        for p.rope_interleaved in (0, 1):
            assert qsa.load().qsa_paged_workspace_size(ctypes.byref(p), 1, 1, ctypes.byref(n)) == 0


@pytest.mark.parametrize("name", ["append", "decode", "prefill"])
def test_cache_checks(name):
    p = qsa.layer_params()
    for kw, want in [(dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID), (dict(page_table=None), INVALID),
                     (dict(k_pages=A + 8), MISALIGNED), (dict(v_pages=A + 2), MISALIGNED), (dict(n_pages=0), INVALID),
                     (dict(n_pages=1 << 31), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(page_size=65537), UNSUPPORTED),
                     (dict(max_pages=0), INVALID), (dict(table_ld=7), INVALID), (dict(page_stride=8), INVALID),
                     (dict(token_stride=255), INVALID), (dict(token_stride=260), INVALID), (dict(head_stride=-256), INVALID)]:
        assert call(name, p, kv_struct(**kw)) == want, kw
    assert call(name, p, B=0) == INVALID
    assert call(name, p, B=4097, T=4097) == UNSUPPORTED
    assert call(name, p, ws_bytes=100) == SMALL
    assert call(name, p, ws=None) == INVALID
    assert call(name, p, ws=A + 8) == MISALIGNED
    assert call(name, p, cl=None) == INVALID


def test_call_checks():
    p = qsa.layer_params()
    assert call("norm_rope", p, q=None) == INVALID                     # q_out without q
    assert call("norm_rope", p, k_out=None) == INVALID
    assert call("norm_rope", p, q=None, q_out=None, k=None, k_out=None) == INVALID
    assert call("norm_rope", p, T=-1) == INVALID
    assert call("norm_rope", p, T=1 << 31) == UNSUPPORTED
    assert call("norm_rope", p, pos0=-1) == INVALID
    assert call("norm_rope", p, q_ld=24 * 256 - 8) == INVALID
    assert call("norm_rope", p, k_ld=516) == INVALID
    assert call("norm_rope", p, qw=A + 4) == MISALIGNED
    assert call("append", p, k=None) == INVALID
    assert call("append", p, v=None) == INVALID
    assert call("append", p, q_out=None) == INVALID
    assert call("append", p, cu=None, T=3) == INVALID                  # one token per sequence
    assert call("append", p, v_ld=504) == INVALID
    assert call("append", p, v=A + 2) == MISALIGNED
    assert call("append", p, T=1 << 24) == UNSUPPORTED
    assert call("decode", p, q=None) == INVALID
    assert call("decode", p, out=A + 8) == MISALIGNED
    assert call("decode", p, kv_struct(max_pages=1 << 20, table_ld=1 << 20, page_size=65536), B=65) == UNSUPPORTED
    assert call("prefill", p, cu=None) == INVALID
    assert call("prefill", p, T=-1) == INVALID
    assert call("prefill", p, T=1 << 24) == UNSUPPORTED
    with pytest.raises(qsa.QSAError):
        qsa.qsa_paged_workspace_size(p, 0, 4)
    with pytest.raises(qsa.QSAError):
        qsa.qsa_paged_workspace_size(p, 1, -1)


def test_binding_refuses_tensors_that_do_not_fit():
    p = qsa.layer_params(4, 2, 64)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = bf(5, 16, 2, 64)
    with pytest.raises(ValueError, match="alike"):
        qsa.PagedKV(pool, bf(5, 16, 2, 32), i32(2, 3))
    with pytest.raises(ValueError, match="int32"):
        qsa.PagedKV(pool, pool, i32(2, 3).long())
    with pytest.raises(ValueError, match="16-bit"):
        qsa.PagedKV(pool.float(), pool.float(), i32(2, 3))
    with pytest.raises(ValueError, match="contiguous"):
        qsa.PagedKV(pool.transpose(2, 3), pool.transpose(2, 3), i32(2, 3))
    kv = qsa.PagedKV(pool, bf(5, 16, 2, 64), i32(2, 3))
    ws = torch.zeros(1 << 24, dtype=torch.uint8)
    q, out = bf(2, 4, 64), bf(2, 4, 64)
    for bad in [dict(q=bf(2, 4, 32)), dict(q=bf(1, 4, 64)), dict(q=q.half()), dict(out=out.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(lse=torch.zeros(2, 4, dtype=torch.float64)), dict(cache_len=i32(1)), dict(cache_len=i32(2).long()),
                dict(ws=None)]:
        kw = dict(cache_len=i32(2), q=q, out=out, ws=ws, lse=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            qsa.qsa_paged_decode(p, kv, 2, **kw)
    with pytest.raises(ValueError, match="pages hold"):
        qsa.qsa_paged_decode(qsa.layer_params(4, 1, 64), kv, 2, i32(2), q, out, ws)
    with pytest.raises(ValueError, match="rows for"):
        qsa.qsa_paged_decode(p, kv, 3, i32(3), bf(3, 4, 64), bf(3, 4, 64), ws)
    with pytest.raises(ValueError, match="dtype"):
        qsa.qsa_paged_decode(qsa.layer_params(4, 2, 64, dtype=torch.float16), kv, 2, i32(2), q, out, ws)
    with pytest.raises(ValueError, match="CUDA"):                      # all right, but on the host
        qsa.qsa_paged_decode(p, kv, 2, i32(2), q, out, ws)
    with pytest.raises(ValueError, match="positions"):
        qsa.qsa_norm_rope(p, 2, 0, q, None, None, None, out, None, positions=i32(3, 2))
    with pytest.raises(ValueError, match="heads of a row"):
        qsa.qsa_norm_rope(p, 2, 0, bf(2, 64, 4).transpose(1, 2), None, None, None, out, None)
    with pytest.raises(TypeError):
        qsa.layer_params(no_such_field=1)


def test_struct_sizes_match_header(tmp_path):
    """The ctypes structs have the header's sizes and field offsets."""
    import os
    import subprocess
    src = tmp_path / "s.c"
    names = {"qsa_layer_params": qsa.qsa_layer_params, "qsa_paged_kv": qsa.qsa_paged_kv}
    lines = []
    for n, c in names.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % n)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (n, f) for f, *_ in c._fields_]
    src.write_text('#include <stdio.h>\n#include "qsa.h"\nint main(void) {%s return 0;}' % "".join(lines))
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", _build.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for c in names.values():
        want.append(ctypes.sizeof(c))
        want += [getattr(c, f).offset for f, *_ in c._fields_]
    assert got == want and os.path.exists(exe)


def test_page_division():
    """j / page_size by the multiplier and shift that the host hands the kernels,
    over the page sizes and the borders of the pages, up to 2^31 - 1."""
    r = random.Random(1)
    for size in list(range(1, 200)) + [544, 1000, 4095, 4096, 4097, 65535, 65536] + [r.randint(1, 65536) for _ in range(50)]:
        sh = 0
        while (1 << sh) < size:
            sh += 1
        mul = ((1 << 32) * ((1 << sh) - size)) // size + 1
        assert mul < 1 << 32
        top = (1 << 31) - 1
        js = [0, 1, size - 1, size, size + 1, top, top // size * size, top // size * size - 1]
        js += [k * size + d for k in (r.randint(0, top // size) for _ in range(200)) for d in (-1, 0)]
        for j in js:
            if 0 <= j <= top:
                q = (((mul * j) >> 32) + j)
                assert q < 1 << 32 and q >> sh == j // size, (size, j)


def test_tile_slots_hold_every_tile():
    """The prefill grid: sequence b's tiles fit between its first slot,
    cu[b] per / rows + b, and the next one's."""
    r = random.Random(2)
    for _ in range(300):
        B, per, rows = r.randint(1, 40), r.randint(1, 64), r.choice([64, 128])
        new = [r.choice([0, 0, 1, 2, r.randint(0, 300)]) for _ in range(B)]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        first = [cu[b] * per // rows + b for b in range(B + 1)]
        for b in range(B):
            assert first[b] + -(-new[b] * per // rows) <= first[b + 1]
        assert first[B] <= -(-cu[B] * per // rows) + B


def test_decode_split_covers_every_unit_once():
    """The decode split: units of all items end to end, cut evenly over the CTAs;
    each item is either one CTA's or pieces that the join finds again."""
    r = random.Random(3)
    for _ in range(200):
        B, HM, G = r.randint(1, 30), r.choice([1, 2, 3, 16]), r.choice([1, 7, 148, 160])
        units = [r.choice([0, 0, 1, 2, r.randint(0, 400)]) for _ in range(B)]
        items = [(b, hm, u) for b, u in enumerate(units) for hm in range(HM) if u]
        start, total = {}, 0
        for b, hm, u in items:
            start[b, hm] = total
            total += u
        n_cta = min(G, total)
        if total == 0:
            continue
        base, more = total // n_cta, total % n_cta
        pieces, rec, whole = {}, {}, set()
        for c in range(n_cta):
            ua = base * c + min(c, more)
            ub = ua + base + (1 if c < more else 0)
            assert ua < ub and (c or ua == 0) and (c < n_cta - 1 or ub == total)
            for b, hm, u in items:
                s, e = start[b, hm], start[b, hm] + u
                lo, hi = max(s, ua), min(e, ub)
                if lo >= hi:
                    continue
                if hi - lo == u:
                    whole.add((b, hm))
                    continue
                slot = 2 * c + (1 if s >= ua else 0)
                assert slot not in pieces and slot < 2 * G
                pieces[slot] = (b, hm, lo - s, hi - s)
                if s >= ua:
                    assert c not in rec
                    x = e - 1                       # the CTA of the item's last unit
                    rec[c] = (b, hm, x // (base + 1) if x < more * (base + 1) else more + (x - more * (base + 1)) // base)
        for c, (b, hm, last) in rec.items():
            at = 0
            for i in range(last - c + 1):
                pb, phm, lo, hi = pieces.pop(2 * (c + i) + (1 if i == 0 else 0))
                assert (pb, phm, lo) == (b, hm, at)
                at = hi
            assert at == units[b]
            assert (b, hm) not in whole
            whole.add((b, hm))
        assert not pieces and len(whole) == len(items)


# (rope_dim, theta, original length, beta_fast, beta_slow): both crossings of the
# betas among the pairs, before them, behind them, on either side
YARN = [(64, 1e7, 262144.0, 32.0, 1.0), (128, 1e6, 4096.0, 32.0, 1.0), (64, 10.0, 262144.0, 32.0, 1.0), (16, 1.5, 1e6, 32.0, 1.0),
        (64, 1e4, 4.0, 32.0, 1.0), (32, 1e4, 1.0, 2.0, 1.0), (64, 10.0, 128.0, 32.0, 1.0), (64, 1e4, 300.0, 60.0, 0.01),
        (256, 1e7, 6.0, 32.0, 1.0), (64, 1e4, 6.3, 32.0, 1.0)]


@pytest.mark.parametrize("rope_dim,theta,length,fast,slow", YARN)
def test_yarn_keeps_and_divides_by_the_count_of_turns(rope_dim, theta, length, fast, slow):
    """A pair that turns at least beta_fast times over the original length keeps its
    frequency, one of at most beta_slow turns has it divided, others lie between."""
    _build.build(debug=True)
    L = ctypes.CDLL(_build.LIB_DEBUG)
    p = qsa.layer_params(head_dim=256, rope_dim=rope_dim, rope_theta=theta, yarn_factor=4.0, yarn_original_max=length,
                         yarn_beta_fast=fast, yarn_beta_slow=slow)
    f = (ctypes.c_double * (rope_dim // 2))()
    assert L.qsa_debug_rope_frequencies(ctypes.byref(p), f) == 0
    for i, got in enumerate(f):
        plain = theta ** (-2 * i / rope_dim)
        turns = length * plain / (2 * math.pi)
        if turns >= fast:
            assert got == pytest.approx(plain, rel=1e-12), i
        elif turns <= slow:
            assert got == pytest.approx(plain / 4, rel=1e-12), i
        else:
            assert plain / 4 * (1 - 1e-12) <= got <= plain * (1 + 1e-12), i


# ------------------------------ the kernels' own index arithmetic, on the host
@pytest.fixture(scope="module")
def debug():
    _build.build(debug=True)
    L = ctypes.CDLL(_build.LIB_DEBUG)
    i32, i64, u32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
    L.qsa_debug_page_of.argtypes, L.qsa_debug_page_of.restype = [i32, u32], u32
    for f in (L.qsa_debug_cut_begin, L.qsa_debug_cut_owner):
        f.argtypes, f.restype = [i64, i64, i64], i64
    L.qsa_debug_first_tile_slot.argtypes, L.qsa_debug_first_tile_slot.restype = [i32, i32, i32, u32, u32], i32
    return L


def test_page_of(debug):
    """At the borders of pages, up to 2^31 - 1."""
    r = random.Random(1)
    top = (1 << 31) - 1
    for size in list(range(1, 200)) + [544, 1000, 4095, 4096, 4097, 65535, 65536] + [r.randint(1, 65536) for _ in range(50)]:
        js = [0, 1, size - 1, size, size + 1, top, top // size * size, top // size * size - 1]
        js += [k * size + d for k in (r.randint(0, top // size) for _ in range(100)) for d in (-1, 0)]
        for j in js:
            if 0 <= j <= top:
                assert debug.qsa_debug_page_of(size, j) == j // size, (size, j)


def test_even_cut(debug):
    """Every unit is one CTA's, the ranges differ by at most one, and the owner of a
    unit is the CTA whose range holds it, for sums beyond 32 bits too."""
    r = random.Random(2)
    for _ in range(400):
        parts = r.choice([1, 2, 7, 74, 148, 160])
        total = r.choice([r.randint(0, 5), r.randint(0, 1000), r.randint(0, 1 << 45), parts, parts - 1, parts + 1])
        begin = [debug.qsa_debug_cut_begin(total, parts, c) for c in range(parts + 1)]
        sizes = [b - a for a, b in zip(begin, begin[1:])]
        assert begin[0] == 0 and begin[-1] == total and max(sizes) - min(sizes) <= 1 and min(sizes) >= 0
        for u in {0, total - 1, *(b + d for b in begin for d in (-1, 0, 1)), *(r.randint(0, max(total - 1, 0)) for _ in range(20))}:
            if 0 <= u < total:
                c = debug.qsa_debug_cut_owner(total, parts, u)
                assert begin[c] <= u < begin[c + 1]


@pytest.mark.parametrize("rows", [128, 256])
def test_first_tile_slots(debug, rows):
    """A sequence's tiles fit between its first slot and the next one's, the last
    sequence's into the grid; offsets outside the tokens count as the nearer end."""
    r = random.Random(3)
    for _ in range(300):
        B, per = r.randint(1, 40), r.choice([1, 2, 7, 12, 64, r.randint(1, 64)])
        new = [r.choice([0, 0, 1, 2, r.randint(0, 300), r.randint(0, 20000)]) for _ in range(B)]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        T = cu[-1]
        first = [debug.qsa_debug_first_tile_slot(b, cu[b], T, per, rows) for b in range(B + 1)]
        for b in range(B):
            assert first[b] + -(-new[b] * per // rows) <= first[b + 1]
        assert first[B] <= -(-T * per // rows) + B
        assert debug.qsa_debug_first_tile_slot(0, -5, T, per, rows) == 0
        assert debug.qsa_debug_first_tile_slot(B, 2 ** 31 - 1, T, per, rows) == first[B]
    T = (1 << 24) - 1
    assert debug.qsa_debug_first_tile_slot(4096, T, T, 64, rows) == T * 64 // rows + 4096
