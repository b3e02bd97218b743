"""What the paged-cache operators are measured on: cases, inputs, plain forms.

Four operators that together serve a layer from a paged key-value cache:

* ``norm_rope``: RMS norm of every query and key head, then the rotation of
  its first ``rope_dim`` dims, by one position or by three (time, height,
  width);
* ``append``: the same on the way into the cache: queries out, keys normed
  and rotated into their pages, values beside them;
* ``decode``: attention of one new token per sequence over its pages, full or
  with a sliding window and sinks (first tokens that stay visible);
* ``prefill``: attention of the new tokens of a ragged batch over the pages,
  cached tokens and the new ones before it, full or with window and sinks.

``own`` picks the framework's calls instead of the plain forms.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# query heads, key-value heads, head dim: the QSA layer's shape, then generic
# grouped, multi-head and multi-query ones
HEADS = [(24, 2, 256), (16, 2, 256), (32, 8, 128), (28, 4, 128), (7, 7, 128), (16, 16, 64), (40, 5, 64), (40, 1, 64)]
EPS = 1e-6
THETA = 1e7
YARN_ORIGINAL = 262144.0


# ------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = {"op": op, "dtype": "bf16", "hq": 24, "hk": 2, "d": 256, "rope_dim": 64, "axes": 1, "yarn": 0.0}
    if op in ("decode", "prefill"):
        c.update(page=64, window=0, sinks=0)
    if op == "append":
        c.update(page=64)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's queries and keys of 64 sequences: latency
        _case("norm_rope", "norm_rope_step_64", T=64),
        # the queries and keys of a 32K prompt
        _case("norm_rope", "norm_rope_prompt_32k", T=32768),
        # image and video tokens, three axes, an odd count
        _case("norm_rope", "norm_rope_video_10007", T=10007, dtype="fp16", hq=32, hk=8, d=128, rope_dim=128, axes=3),
        # one decode step of 64 sequences at mixed depths
        _case("append", "append_step_64", B=64, nmin=1, nmax=1, cmin=1000, cmax=262143),
        # prompts of 13 requests, small pages
        _case("append", "append_prompts_13", B=13, nmin=37, nmax=8192, cmin=0, cmax=5000, page=16),
        # one user, a short chat
        _case("decode", "decode_1x509", B=1, lmin=509, lmax=509),
        # a serving batch at mixed depths, small pages
        _case("decode", "decode_37x32k", B=37, lmin=33, lmax=32768, page=16, hq=32, hk=8, d=128),
        # a long-context batch up to the layer's 256K
        _case("decode", "decode_64x256k", B=64, lmin=16384, lmax=262144),
        # window layers of a long-context batch: most pages are given back
        _case("decode", "decode_window_128x100k", B=128, lmin=500, lmax=100003, window=4096, sinks=4),
        # the last chunk of a prompt, few rows over a long prefix
        _case("prefill", "prefill_chunk_37_over_20k", B=1, nmin=37, nmax=37, cmin=20011, cmax=20011),
        # prompts of 8 requests through a window layer
        _case("prefill", "prefill_window_8x8k", B=8, nmin=301, nmax=8192, cmin=0, cmax=3001, window=1024, sinks=4, page=16),
        # one whole 32K prompt through a dense layer
        _case("prefill", "prefill_32k", B=1, nmin=32768, nmax=32768, cmin=0, cmax=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "prefill"])
    hq, hk, d = rng.choice(HEADS)
    kw = {"dtype": rng.choice(["bf16", "bf16", "fp16"]), "hq": hq, "hk": hk, "d": d}
    page = rng.choice([16, 16, 32, 48, 64, 128])
    if op in ("norm_rope", "append"):
        kw["rope_dim"] = rng.choice([r for r in (32, 64, 128) if r <= d])
        kw["axes"] = rng.choice([1, 1, 3])
        kw["yarn"] = rng.choice([0.0, 0.0, 4.0])
        most = int(32768 * 26 * 256 / ((hq + hk) * d))
        if op == "norm_rope":
            kw["T"] = _log_int(rng, 1, most)
        else:
            B = _log_int(rng, 1, 128)
            n = _log_int(rng, 1, max(1, most // (4 * B)))
            kw.update(B=B, nmin=max(1, n // rng.choice([1, 3, 10])), nmax=n, cmin=0, cmax=rng.choice([0, 777, 262143]), page=page)
        return _case(op, **kw)
    if rng.random() < 0.5:
        kw["window"] = _log_int(rng, 16, 8192)
        kw["sinks"] = rng.choice([0, 1, 4, 64])
    kw["page"] = page
    if op == "decode":
        B = _log_int(rng, 1, 256)
        # at most about a quarter of the largest listed batch's bytes
        most = int(min(262144, 3e9 / (B * hk * d * 4)))
        L = _log_int(rng, 1, most)
        kw.update(B=B, lmin=max(1, L // rng.choice([1, 4, 50])), lmax=L)
        return _case(op, **kw)
    B = _log_int(rng, 1, 16)
    # at most about a half of the largest listed prompt's products
    side = math.sqrt(0.5 * 32768 ** 2 * 24 * 256 / (B * hq * d))
    n = _log_int(rng, 1, int(min(16384, side * 0.7)))
    c = rng.choice([0, _log_int(rng, 1, max(1, int(min(65536, side * side / (4 * n)))))])
    kw.update(B=B, nmin=max(1, n // rng.choice([1, 5, 40])), nmax=n, cmin=c // 2, cmax=c)
    return _case(op, **kw)


def _spread(lo, hi, n, phase):
    """n whole numbers from lo to hi, spread over their logarithm, hi first."""
    lo1, hi1 = lo + 1, hi + 1
    return [hi] + [int(lo1 * (hi1 / lo1) ** ((b * 0.6180339887 + phase) % 1.0)) - 1 for b in range(1, n)]


def _lens(case):
    """(cached tokens, new tokens) of each sequence."""
    B = case["B"]
    if case["op"] == "decode":
        return [L - 1 for L in _spread(case["lmin"], case["lmax"], B, 0.3)], [1] * B
    return _spread(case["cmin"], case["cmax"], B, 0.7), _spread(case["nmin"], case["nmax"], B, 0.3)


def _first_visible(case, pos):
    """The first key that the window leaves to a query at `pos`."""
    return max(0, pos - case["window"] + 1) if case["window"] else 0


# ------------------------------------------------------------------ inputs
def _randn(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _positions(case, T, gen):
    """Tokens of a video of 14 x 18 patches a frame after a text of random length."""
    if case["axes"] == 1:
        return None
    i = torch.arange(T, device="cuda")
    start = torch.randint(0, 100000, (1,), generator=gen, device="cuda")
    return torch.stack([start + i // 252, start + (i // 18) % 14, start + i % 18]).to(torch.int32)


def _sections(case):
    """Rotary pairs of the three axes: 11, 11 and 10 of 32, and in proportion."""
    half = case["rope_dim"] // 2
    w = half * 10 // 32
    h = (half - w) // 2
    return [half - w - h, h, w]


def _paged(case, s, gen):
    """A pool of pages and the table; only pages with a visible or a new
    token are there, in random order."""
    page, dt = case["page"], DTYPES[case["dtype"]]
    cached, new = _lens(case)
    used = []
    for b, (c, n) in enumerate(zip(cached, new)):
        total = c + n
        if case["op"] == "append":
            keep = range(c // page, (total - 1) // page + 1)
        else:
            lo = _first_visible(case, c)
            keep = sorted(set(range(0, min(-(-case["sinks"] // page), -(-total // page)))) | set(range(lo // page, (total - 1) // page + 1)))
        used.append(keep)
    n_pages = sum(len(k) for k in used) + 3
    where = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu().numpy()
    table = np.full((case["B"], max(-(-(c + n) // page) for c, n in zip(cached, new))), -1, np.int32)
    at = 0
    for b, keep in enumerate(used):
        keep = np.fromiter(keep, np.int64)
        table[b, keep] = where[at:at + len(keep)]
        at += len(keep)
    s["table"] = torch.from_numpy(table).cuda()
    s["k_pages"] = _randn(gen, dt, n_pages, page, case["hk"], case["d"])
    s["v_pages"] = _randn(gen, dt, n_pages, page, case["hk"], case["d"])
    s["cached"], s["new"] = cached, new
    s["cache_len"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
    s["cu_new"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    return sum(new)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt, hq, hk, d = case["op"], DTYPES[case["dtype"]], case["hq"], case["hk"], case["d"]
    s = {"case": case}
    T = case["T"] if op == "norm_rope" else _paged(case, s, gen)
    s["T"] = T
    if op in ("norm_rope", "append"):
        # queries, keys and values as one projection's output, the way a layer has them
        qkv = _randn(gen, dt, T, hq + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_weight"], s["k_weight"] = (0.2 * _randn(gen, dt, d)).to(dt), (0.2 * _randn(gen, dt, d)).to(dt)
        s["positions"] = _positions(case, T, gen)
        s["pos0"] = 12345 if op == "norm_rope" else 0
        s["q_out"] = torch.zeros(T, hq, d, dtype=dt, device="cuda")
        if op == "norm_rope":
            s["k_out"] = torch.zeros(T, hk, d, dtype=dt, device="cuda")
    else:
        s["q"] = _randn(gen, dt, T, hq, d)
        s["out"] = torch.zeros(T, hq, d, dtype=dt, device="cuda")
        s["lse"] = torch.zeros(T, hq, dtype=torch.float32, device="cuda")
    if own:
        import block_sparse_long_qsa_b200 as qsa
        kw = {"rope_dim": case["rope_dim"], "rope_theta": THETA, "norm_eps": EPS, "norm_zero_centred": 1, "rope_axes": case["axes"],
              "yarn_factor": case["yarn"], "yarn_original_max": YARN_ORIGINAL, "window": case.get("window", 0), "n_sinks": case.get("sinks", 0)}
        s["p"] = qsa.layer_params(hq, hk, d, dtype=dt, rope_section=_sections(case), **kw)
        if op != "norm_rope":
            s["kv"] = qsa.PagedKV(s["k_pages"], s["v_pages"], s["table"])
            s["ws"] = qsa.paged_workspace(s["p"], case["B"], T)
    return s


# ------------------------------------------------------------- plain forms
def _freqs(case):
    """The rotary frequencies and the factor on the rotated dims."""
    rd, s = case["rope_dim"], case["yarn"]
    f = [THETA ** (-2.0 * i / rd) for i in range(rd // 2)]
    if s <= 1.0:
        return f, 1.0
    at = lambda turns: rd * math.log(YARN_ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(THETA))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0.0), min(math.ceil(at(1.0)), rd - 1.0)
    mix = [min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(rd // 2)]
    return [x / s * m + x * (1 - m) for x, m in zip(f, mix)], 0.1 * math.log(s) + 1.0


def _axis_of_pair(case):
    """Axis i % 3 while that axis has pairs left, time after that."""
    sec, half = _sections(case), case["rope_dim"] // 2
    return [i % 3 if i % 3 and i < 3 * sec[i % 3] else 0 for i in range(half)]


def _plain_norm_rope(case, x, weight, pos):
    """pos [axes][T], whole numbers."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (1.0 + weight.float())
    f, factor = _freqs(case)
    f = torch.tensor(f, dtype=torch.float64, device=x.device)
    p = pos.double() if case["axes"] == 1 else pos.double()[_axis_of_pair(case)]     # [1 or pairs][T]
    angle = p.t() * f                                                                # 64 bits: far positions
    cos, sin = (factor * angle.cos()).float()[:, None], (factor * angle.sin()).float()[:, None]
    h = case["rope_dim"] // 2
    a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_positions(case, s):
    if s["positions"] is not None:
        return s["positions"]
    if case["op"] == "norm_rope":
        return s["pos0"] + torch.arange(s["T"], device="cuda")[None]
    return _plain_slots(s)[1][None]


def _plain_slots(s):
    """The sequence and the cache position of each new token."""
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), s["cu_new"].diff(), output_size=s["T"])
    return seq, s["cache_len"][seq] + torch.arange(s["T"], device="cuda") - s["cu_new"][seq]


def _plain_rows(case, s, b, lo, hi):
    """Keys and values of tokens [lo, hi) of sequence b, in 32 bits, head first."""
    page = case["page"]
    ids = s["table"][b, lo // page:(hi - 1) // page + 1]
    cut = slice(lo % page, lo % page + hi - lo)
    return [pool[ids].flatten(0, 1)[cut].float().transpose(0, 1) for pool in (s["k_pages"], s["v_pages"])]


def _plain_attend(case, s, b, q, pos0):
    """q [n][hq][d] at positions pos0 .. of sequence b."""
    n, hq, d = q.shape
    hk = case["hk"]
    lo, hi = _first_visible(case, pos0), pos0 + n
    sinks = min(case["sinks"], lo)
    k, v = _plain_rows(case, s, b, lo, hi)
    at = torch.arange(lo, hi, device="cuda")
    if sinks:
        k0, v0 = _plain_rows(case, s, b, 0, sinks)
        k, v = torch.cat([k0, k], 1), torch.cat([v0, v], 1)
        at = torch.cat([torch.arange(sinks, device="cuda"), at])
    score = (q.float().reshape(n, hk, hq // hk, d).permute(1, 2, 0, 3).flatten(1, 2) @ k.transpose(1, 2)) / math.sqrt(d)
    score = score.view(hk, hq // hk, n, -1)
    if n > 1 or case["window"]:
        at_q = torch.arange(pos0, pos0 + n, device="cuda")[:, None]
        seen = at <= at_q
        if case["window"]:
            seen &= (at > at_q - case["window"]) | (at < case["sinks"])
        score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = (score - top).exp()
    total = e.sum(-1, keepdim=True)
    out = (e.flatten(1, 2) @ v).view(hk, hq // hk, n, d) / total
    lse = (top + total.log())[..., 0]
    return out.permute(2, 0, 1, 3).reshape(n, hq, d).to(q.dtype), lse.permute(2, 0, 1).reshape(n, hq)


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op in ("norm_rope", "append"):
        pos = _plain_positions(case, s)
        q = _plain_norm_rope(case, s["q"], s["q_weight"], pos).to(dt)
        k = _plain_norm_rope(case, s["k"], s["k_weight"], pos).to(dt)
        if op == "norm_rope":
            return {"q": q, "k": k}
        seq, at = _plain_slots(s)
        page = s["table"][seq, at // case["page"]]
        s["k_pages"][page, at % case["page"]] = k
        s["v_pages"][page, at % case["page"]] = s["v"]
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    outs, lses, row = [], [], 0
    for b, (c, n) in enumerate(zip(s["cached"], s["new"])):
        for i in range(0, n, 512):
            m = min(512, n - i)
            o, lse = _plain_attend(case, s, b, s["q"][row + i:row + i + m], c + i)
            outs.append(o)
            lses.append(lse)
        row += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def run(state):
    s = state
    if not own:
        return _plain(s)
    import block_sparse_long_qsa_b200 as qsa
    op, B = s["case"]["op"], s["case"].get("B", 0)
    if op == "norm_rope":
        qsa.qsa_norm_rope(s["p"], s["T"], s["pos0"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["q_out"], s["k_out"], positions=s["positions"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        qsa.qsa_paged_append(s["p"], s["kv"], B, s["T"], s["cu_new"], s["cache_len"], s["k"], s["v"], s["ws"], q=s["q"], q_out=s["q_out"],
                             q_weight=s["q_weight"], k_weight=s["k_weight"], positions=s["positions"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "decode":
        qsa.qsa_paged_decode(s["p"], s["kv"], B, s["cache_len"], s["q"], s["out"], s["ws"], lse=s["lse"])
    else:
        qsa.qsa_paged_prefill(s["p"], s["kv"], B, s["T"], s["cu_new"], s["cache_len"], s["q"], s["out"], s["ws"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ----------------------------------------------------- the definition, 64 bits
def _exact_turn(case, x, weight, pos):
    """x [T][h][d], pos [T][pairs], numpy."""
    x = x / np.sqrt(np.mean(np.square(x), -1, keepdims=True) + EPS) * (1.0 + weight)
    half = case["rope_dim"] // 2
    i = np.arange(half)
    f = np.power(THETA, -i / half)
    factor = 1.0
    if case["yarn"] > 1.0:
        # pair index at which a wavelength fits `turns` times into the original context
        index = lambda turns: half * np.log(YARN_ORIGINAL / (2 * np.pi * turns)) / np.log(THETA)  # noqa: E731
        lo, hi = max(np.floor(index(32.0)), 0.0), min(np.ceil(index(1.0)), 2 * half - 1.0)
        share = np.clip((i - lo) / (hi - lo), 0.0, 1.0)
        f = f * (1.0 - share) + f / case["yarn"] * share
        factor = 0.1 * np.log(case["yarn"]) + 1.0
    turn = factor * np.exp(1j * (pos * f))[:, None]
    z = (x[..., :half] + 1j * x[..., half:2 * half]) * turn
    return np.concatenate([z.real, z.imag, x[..., 2 * half:]], -1)


def _f64(t):
    return t.double().cpu().numpy()


def exact(case, seed):
    s = prepare(case, seed)
    op, hk, d = case["op"], case["hk"], case["d"]
    if op in ("norm_rope", "append"):
        cached, new = (s["cached"], s["new"]) if op == "append" else ([s["pos0"]], [s["T"]])
        flat = np.concatenate([c + np.arange(n) for c, n in zip(cached, new)])
        half = case["rope_dim"] // 2
        if case["axes"] == 1:
            pos = np.repeat(flat[:, None], half, 1)
        else:
            _, h, w = _sections(case)
            axis = np.zeros(half, np.int64)
            axis[1:3 * h:3] = 1
            axis[2:3 * w:3] = 2
            pos = s["positions"].cpu().numpy()[axis].T
        q, k = np.empty(s["q"].shape), np.empty(s["k"].shape)
        for i in range(0, s["T"], 4096):
            c = slice(i, i + 4096)
            q[c] = _exact_turn(case, _f64(s["q"][c]), _f64(s["q_weight"]), pos[c])
            k[c] = _exact_turn(case, _f64(s["k"][c]), _f64(s["k_weight"]), pos[c])
        if op == "norm_rope":
            return {"q": q, "k": k}
        kp, vp, table, v = _f64(s["k_pages"]), _f64(s["v_pages"]), s["table"].cpu().numpy(), _f64(s["v"])
        row = 0
        for b, (c, n) in enumerate(zip(cached, new)):
            at = c + np.arange(n)
            slot = table[b, at // case["page"]], at % case["page"]
            kp[slot], vp[slot] = k[row:row + n], v[row:row + n]
            row += n
        return {"q": q, "k_pages": kp, "v_pages": vp}
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    per = case["hq"] // hk
    row = 0
    for b, (c, n) in enumerate(zip(s["cached"], s["new"])):
        for i in range(0, n, 1024):
            m = min(1024, n - i)
            first, last = c + i, c + i + m - 1
            # the keys any of these tokens sees, one by one
            keys = torch.arange(last + 1, device="cuda")
            if case["window"]:
                keys = keys[(keys < case["sinks"]) | (keys > first - case["window"])]
            page = s["table"][b].long()[keys // case["page"]]
            at = torch.arange(first, last + 1, device="cuda")
            away = keys[None] > at[:, None]
            if case["window"]:
                away |= (keys[None] <= at[:, None] - case["window"]) & (keys[None] >= case["sinks"])
            for g in range(hk):
                k = s["k_pages"][page, keys % case["page"], g].double()
                v = s["v_pages"][page, keys % case["page"], g].double()
                for h in range(g * per, (g + 1) * per):
                    x = (s["q"][row + i:row + i + m, h].double() @ k.t()) * d ** -0.5
                    x[away] = -math.inf
                    lse[row + i:row + i + m, h] = torch.logsumexp(x, -1)
                    out[row + i:row + i + m, h] = torch.softmax(x, -1) @ v
        row += n
    return {"out": out, "lse": lse}


# -------------------------------------------------------------------- floor
def _seen(case, c, n):
    """(keys that any new token sees, pairs of a new token and a key it sees)."""
    lo = _first_visible(case, c)
    keys = c + n - lo + min(case["sinks"], lo)
    pos = np.arange(c, c + n, dtype=np.int64)
    first = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros_like(pos)
    return keys, int((pos + 1 - first + np.minimum(case["sinks"], first)).sum())


def work(case):
    hq, hk, d, op = case["hq"], case["hk"], case["d"], case["op"]
    if op == "norm_rope":
        T = case["T"]
        return {"bytes": 4 * T * (hq + hk) * d + 4 * d + 4 * T * (case["axes"] if case["axes"] > 1 else 0), "flops": 10 * T * (hq + hk) * d}
    cached, new = _lens(case)
    T = sum(new)
    if op == "append":
        return {"bytes": 4 * T * (hq + 2 * hk) * d + 4 * d + 4 * T * (case["axes"] if case["axes"] > 1 else 0), "flops": 10 * T * (hq + hk) * d}
    seen = [_seen(case, c, n) for c, n in zip(cached, new)]
    return {"bytes": 4 * T * hq * d + 4 * T * hq + 4 * sum(k for k, _ in seen) * hk * d, "flops": 4 * hq * d * sum(p for _, p in seen)}
