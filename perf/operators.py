"""Timed cases of the 4-bit KV cache: writing K/V rows quantised, reading rows
back, and attention over the cache.

A case is a dict of plain values.  ``lens`` gives each sequence's length in the
cache after the call and ``new`` how many of its last positions the call is about
(rows written, rows read back, or query tokens), both as comma-separated numbers.

Kinds:
  write   append the ``new`` rows of every sequence, then read the same rows back
          (what the cache holds is returned as the values it stands for)
  read    read the ``new`` last rows of every sequence from a filled cache
  attend  causal attention of the ``new`` last positions over the whole cache

``own`` selects the framework's kernels; where it is false ``run`` computes the
same thing with elementary torch operations in 32 bits.
"""

import math

import numpy as np
import torch

own = False

PAGE = 64   # positions of one page
TILE = 16   # positions of one tile: the unit the page is made of
GROUP = 32  # neighbouring values of one row that share a scale and a minimum

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _text(values):
    return ",".join(str(int(v)) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _case(name, kind, dtype, heads, kv_heads, d, lens, new):
    return {"name": name, "kind": kind, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "d": d,
            "lens": _text(lens), "new": _text(new)}


def listed():
    b8 = [512 + 128 * i for i in range(8)]            # the 8-lane workload's prompts
    odd = [517 + 129 * i for i in range(8)]
    serve = [16384 - 247 * i for i in range(64)]      # many long sequences of a server
    return [
        # one decode step of eight lanes: one row each, where the launch is what it costs
        _case("write_step_8", "write", "fp32", 32, 8, 64, [n + 1 for n in b8], [1] * 8),
        # the prompts of eight lanes, odd lengths, in one call
        _case("write_prompts_odd", "write", "fp16", 32, 8, 64, odd, odd),
        # a long prompt of the 128-dim shape
        _case("write_prompt_8192", "write", "bf16", 32, 8, 128, [8192], [8192]),
        # a parked conversation of 8192 positions comes back
        _case("read_8192", "read", "bf16", 32, 8, 64, [8192], [8192]),
        # eight conversations of odd lengths come back in 32 bits
        _case("read_odd_fp32", "read", "fp32", 32, 8, 128, odd, odd),
        # one decode step, one lane, short context: the smallest call
        _case("decode_1x160", "attend", "bf16", 32, 8, 64, [160], [1]),
        # one decode step of the eight-lane workload with 32-bit activations
        _case("decode_8_fp32", "attend", "fp32", 32, 8, 64, [n + 65 for n in b8], [1] * 8),
        # one decode step at the long context
        _case("decode_1x8192", "attend", "bf16", 32, 8, 64, [8200], [1]),
        # one decode step of many long sequences: the memory-bound end
        _case("decode_64x16384", "attend", "bf16", 32, 8, 128, serve, [1] * 64),
        # the 2048-token prompt of the 128-dim shape
        _case("prompt_2048", "attend", "bf16", 32, 8, 128, [2048], [2048]),
        # the last pass of a long prompt: 2048 tokens that see 8192 positions
        _case("prompt_2048_of_8192", "attend", "fp16", 32, 8, 64, [8192], [2048]),
        # eight prompts of odd lengths with 32-bit activations
        _case("prompts_odd_fp32", "attend", "fp32", 32, 8, 64, odd, odd),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 8])
    if kind in ("write", "read"):
        n = _log(rng, 1, 32)
        top = max(1, 8192 // n)
        lens = [_log(rng, 1, top) for _ in range(n)]
        new = lens if kind == "read" or rng.random() < 0.5 else [_log(rng, 1, v) for v in lens]
    else:
        form = rng.choice(["token", "token", "few", "prompt"])
        if form == "prompt":
            n = _log(rng, 1, 8)
            top = 2048 // n
            new = [_log(rng, max(1, top // 8), top) for _ in range(n)]
            lens = [v + rng.choice([0, _log(rng, 1, 4 * top)]) for v in new]
        else:
            n = _log(rng, 1, 48)
            lens = [_log(rng, 17, 16384) for _ in range(n)]
            new = [1] * n if form == "token" else [rng.randint(1, 8) for _ in range(n)]
    return {"kind": kind, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "d": d,
            "lens": _text(lens), "new": _text(new)}


# ---- the cache's layout ------------------------------------------------------
#
# pool [layers][pages][kv heads][4 tiles][20 d] bytes; a tile of 16 positions is
#   [8 d] K codes: 32-bit words of 8 codes, word w of row r holds values 8 w .. 8 w + 7
#   [8 d] V codes: 16-bit units of 4 codes, unit q of row r holds values 4 q .. 4 q + 3
#   [d] K scales, [d] K minima, [d] V scales, [d] V minima (fp16)
# in the orders below; a value is minimum + scale * code.


def _tile_places(d):
    """Word index of every K word, 16-bit index of every V unit and parameter."""
    g_n = d // GROUP
    r, w = torch.meshgrid(torch.arange(TILE), torch.arange(d // 8), indexing="ij")
    i, lane = (r // 8) * g_n + w // 4, (r % 8) * 4 + w % 4
    k_word = (i // 4) * 128 + lane * 4 + i % 4
    r, q = torch.meshgrid(torch.arange(TILE), torch.arange(d // 4), indexing="ij")
    i, lane = (q // 8) * 2 + r // 8, (q % 8) * 4 + (r % 8) // 2
    v_unit = 4 * d + ((i // 4) * 128 + lane * 4 + i % 4) * 2 + r % 2
    r, g = torch.meshgrid(torch.arange(TILE), torch.arange(g_n), indexing="ij")
    i = (r // 8) * g_n + g
    scale = ((i // 4) * 16 + ((r % 8) // 2) * 4 + i % 4) * 2 + r % 2
    k_scale, v_scale = 8 * d + scale, 9 * d + scale
    k_min, v_min = 8 * d + d // 2 + r * g_n + g, 9 * d + d // 2 + g * TILE + r
    return k_word, v_unit, k_scale, k_min, v_scale, v_min


def _halves(x, down):
    """fp16 neighbour of x (float64): the largest not above it, or the smallest not below."""
    h = x.to(torch.float16)
    away = h.double() > x if down else h.double() < x
    step = torch.nextafter(h, torch.full_like(h, -math.inf if down else math.inf))
    return torch.where(away, step, h)


def _quantise(x):
    """Codes [..., d], scales and minima [..., d/32] of rows [..., d]: per group of 32
    values the minimum rounded down to fp16, the scale (max - min) / 15 rounded up to
    fp16, codes rounded to nearest even.  In 64 bits: values sit next to a border."""
    v = x.double().reshape(*x.shape[:-1], -1, GROUP)
    low = _halves(v.amin(-1), True)
    scale = _halves((v.amax(-1) - low.double()) / 15, False)
    s = torch.where(scale > 0, scale, torch.ones_like(scale)).double().unsqueeze(-1)
    code = torch.round((v - low.double().unsqueeze(-1)) / s).to(torch.uint8)
    return code.reshape(x.shape), scale, low


def _places(pool, block_table, seq, positions, d):
    """First 32-bit word of the tile of every (position, kv head)."""
    page = block_table[seq, positions // PAGE].long()
    heads = pool.shape[2]
    tile = (page[:, None] * heads + torch.arange(heads, device=pool.device)) * (PAGE // TILE)
    return (tile + (positions % PAGE // TILE)[:, None]) * (5 * d)


def _write(pool, block_table, seq, start, k, v, d):
    positions = torch.arange(start, start + k.shape[0], device=pool.device)
    base = _places(pool, block_table, seq, positions, d)
    row = positions % TILE
    k_word, v_unit, k_scale, k_min, v_scale, v_min = (p.to(pool.device) for p in _tile_places(d))
    words, halves = pool.view(torch.int32).view(-1), pool.view(torch.int16).view(-1)

    def packed(code, as_type):
        return (code[..., ::2] | (code[..., 1::2] << 4)).contiguous().view(as_type)

    for x, place_code, place_s, place_m in ((k, k_word, k_scale, k_min), (v, v_unit, v_scale, v_min)):
        code, scale, low = _quantise(x)
        if x is k:
            words[(base[:, :, None] + place_code[row][:, None, :])] = packed(code, torch.int32)
        else:
            halves[(2 * base[:, :, None] + place_code[row][:, None, :])] = packed(code, torch.int16)
        halves[(2 * base[:, :, None] + place_s[row][:, None, :])] = scale.view(torch.int16)
        halves[(2 * base[:, :, None] + place_m[row][:, None, :])] = low.view(torch.int16)


def _read(pool, block_table, seq, start, stop, d):
    """K and V values (float32) of a sequence's positions start .. stop - 1, [n, kv heads, d]."""
    positions = torch.arange(start, stop, device=pool.device)
    base = _places(pool, block_table, seq, positions, d)
    row = positions % TILE
    k_word, v_unit, k_scale, k_min, v_scale, v_min = (p.to(pool.device) for p in _tile_places(d))
    words, halves = pool.view(torch.int32).view(-1), pool.view(torch.int16).view(-1)
    out = []
    for kind, place_code, place_s, place_m in (("k", k_word, k_scale, k_min), ("v", v_unit, v_scale, v_min)):
        if kind == "k":
            unit, n = words[base[:, :, None] + place_code[row][:, None, :]], 8
        else:
            unit, n = halves[2 * base[:, :, None] + place_code[row][:, None, :]].int(), 4
        shift = torch.arange(0, 4 * n, 4, device=pool.device, dtype=torch.int32)
        code = (unit[..., None] >> shift) & 15
        scale = halves[2 * base[:, :, None] + place_s[row][:, None, :]].view(torch.float16).float()
        low = halves[2 * base[:, :, None] + place_m[row][:, None, :]].view(torch.float16).float()
        code = code.reshape(*code.shape[:2], d // GROUP, GROUP).float()
        out.append((low[..., None] + scale[..., None] * code).reshape(*code.shape[:2], d))
    return out


# ---- inputs ---------------------------------------------------------------------


def _rows(n, heads, d, gen, device, keys):
    """K or V rows as a decoder makes them: keys have a few large channels."""
    x = torch.randn((n, heads, d), generator=gen, device=device)
    if keys:
        gain = torch.ones(d, device=device)
        gain[3], gain[d // 2 + 5] = 6.0, 4.0
        x = x * gain + 0.5 * torch.randn((1, heads, d), generator=gen, device=device) * gain
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    d, heads, kv_heads, dtype = case["d"], case["heads"], case["kv_heads"], DTYPES[case["dtype"]]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    n_pages = [-(-v // PAGE) for v in lens]
    order = torch.randperm(sum(n_pages), generator=gen, device=dev).int()
    table = torch.zeros((len(lens), max(n_pages)), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(n_pages):
        table[s, :n] = order[at:at + n]
        at += n
    pool = torch.zeros((1, at, kv_heads, PAGE // TILE * 20 * d), dtype=torch.uint8, device=dev)
    total = sum(new)
    state = {"case": case, "lens": lens, "new": new, "pool": pool, "table": table,
             "cu": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev),
             "kv_lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    if case["kind"] != "write":
        for s, n in enumerate(lens):
            for a in range(0, n, 4096):
                m = min(4096, n - a)
                _write(pool, table, s, a, _rows(m, kv_heads, d, gen, dev, True),
                       _rows(m, kv_heads, d, gen, dev, False), d)
    if case["kind"] == "write":
        state["k"] = _rows(total, kv_heads, d, gen, dev, True).to(dtype)
        state["v"] = _rows(total, kv_heads, d, gen, dev, False).to(dtype)
    if case["kind"] == "attend":
        state["q"] = torch.randn((total, heads, d), generator=gen, device=dev).to(dtype)
    if own:
        from persistent_megakernel_02_b200 import Kv4Cache

        state["cache"] = Kv4Cache(pool, table, head_dim=d)
        state["batch"] = state["cache"].batch(state["cu"], state["kv_lens"], n_rows=total, max_new=max(new),
                                              max_len=max(lens))
        shape = (total, heads if case["kind"] == "attend" else kv_heads, d)
        state["out"] = torch.empty(shape, dtype=dtype, device=dev)
        if case["kind"] != "attend":
            state["out2"] = torch.empty(shape, dtype=dtype, device=dev)
    return state


# ---- one pass -------------------------------------------------------------------


def _plain_attend(q, k, v, n_len):
    """Causal attention of the last q.shape[0] positions of n_len (float32)."""
    n, heads, d = q.shape
    rep = heads // k.shape[1]
    k, v = k.transpose(0, 1), v.transpose(0, 1)
    qh = q.float().reshape(n, k.shape[0], rep, d).permute(1, 2, 0, 3).reshape(k.shape[0], rep * n, d)
    s = (qh @ k.transpose(1, 2)) * (1.0 / math.sqrt(d))
    see = torch.arange(n_len, device=q.device)[None, :] <= torch.arange(n_len - n, n_len, device=q.device)[:, None]
    s = s.view(k.shape[0], rep, n, n_len).masked_fill(~see, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p.view(k.shape[0], rep * n, n_len) @ v).view(k.shape[0], rep, n, d) / p.sum(-1, keepdim=True)
    return o.permute(2, 0, 1, 3).reshape(n, heads, d).to(q.dtype)


def run(state):
    case = state["case"]
    kind, d = case["kind"], case["d"]
    if own:
        cache, batch = state["cache"], state["batch"]
        if kind == "write":
            cache.append(0, state["k"], state["v"], batch)
        if kind in ("write", "read"):
            cache.read(0, state["out"], state["out2"], batch)
            return {"k": state["out"], "v": state["out2"]}
        cache.attend(0, state["q"], state["out"], batch)
        return {"out": state["out"]}
    dtype = DTYPES[case["dtype"]]
    pool, table = state["pool"], state["table"]
    spans, at = [], 0
    for n_len, n in zip(state["lens"], state["new"]):
        spans.append((n_len, n, at))
        at += n
    if kind == "write":
        for s, (n_len, n, at) in enumerate(spans):
            _write(pool, table, s, n_len - n, state["k"][at:at + n], state["v"][at:at + n], d)
    if kind in ("write", "read"):
        got = [_read(pool, table, s, n_len - n, n_len, d) for s, (n_len, n, at) in enumerate(spans)]
        return {"k": torch.cat([g[0] for g in got]).to(dtype), "v": torch.cat([g[1] for g in got]).to(dtype)}
    out = torch.empty_like(state["q"])
    for s, (n_len, n, at) in enumerate(spans):
        k, v = _read(pool, table, s, 0, n_len, d)
        out[at:at + n] = _plain_attend(state["q"][at:at + n], k, v, n_len)
    return {"out": out}


def work(case):
    d, heads, kv_heads = case["d"], case["heads"], case["kv_heads"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    size = 4 if case["dtype"] == "fp32" else 2
    row4 = kv_heads * 2 * (d // 2 + d // GROUP * 4)  # bytes of one position's K and V in the cache
    row = kv_heads * 2 * d * size
    rows = sum(new)
    if case["kind"] == "write":  # rows in, codes out; codes in, rows out
        return {"bytes": 2 * rows * (row + row4), "flops": 8 * rows * kv_heads * 2 * d}
    if case["kind"] == "read":
        return {"bytes": rows * (row + row4), "flops": 2 * rows * kv_heads * 2 * d}
    pairs = sum(n * (n_len - n) + n * (n + 1) // 2 for n_len, n in zip(lens, new))
    return {"bytes": sum(lens) * row4 + 2 * rows * heads * d * size, "flops": 4 * d * heads * pairs}


# ---- the definition in 64 bits -----------------------------------------------------


def _np_toward(x, down):
    h = x.astype(np.float16)
    wrong = h.astype(np.float64) > x if down else h.astype(np.float64) < x
    return np.where(wrong, np.nextafter(h, np.float16(-np.inf if down else np.inf)), h).astype(np.float64)


def _exact_quantised(x):
    """The values the cache holds for rows x [n, heads, d] (numpy float64)."""
    out = np.empty_like(x)
    for a in range(0, x.shape[2], GROUP):
        part = x[:, :, a:a + GROUP]
        low = _np_toward(part.min(-1, keepdims=True), True)
        step = _np_toward((part.max(-1, keepdims=True) - low) / 15.0, False)
        code = np.rint((part - low) / np.where(step == 0, 1.0, step))
        out[:, :, a:a + GROUP] = low + step * code
    return out


def _exact_rows(pool, pages, n_len, head, d):
    """K and V (float64) of one kv head's positions 0 .. n_len - 1, straight from the bytes."""
    raw = pool[0, pages.long(), head].reshape(-1, 20 * d)  # one row per tile
    g_n = d // GROUP
    k_byte = np.empty((TILE, d), np.int64)
    v_byte = np.empty((TILE, d), np.int64)
    par = np.empty((4, TILE, d), np.int64)  # byte of the K scale, K minimum, V scale, V minimum
    for r in range(TILE):
        for c in range(d):
            g, w, u = c // 32, c // 8, c // 4
            slot = (r // 8) * g_n + g
            lane = (r % 8) * 4 + w % 4
            k_byte[r, c] = 4 * ((slot // 4) * 128 + lane * 4 + slot % 4) + (c % 8) // 2
            v_slot = g * 2 + r // 8
            v_lane = (u % 8) * 4 + (r % 8) // 2
            v_byte[r, c] = 8 * d + 4 * ((v_slot // 4) * 128 + v_lane * 4 + v_slot % 4) + 2 * (r % 2) + (c % 4) // 2
            pair = 4 * ((slot // 4) * 16 + ((r % 8) // 2) * 4 + slot % 4) + 2 * (r % 2)
            par[0, r, c], par[2, r, c] = 16 * d + pair, 18 * d + pair
            par[1, r, c], par[3, r, c] = 17 * d + 2 * (r * g_n + g), 19 * d + 2 * (g * TILE + r)
    odd = (torch.arange(d, device=pool.device) % 2).bool()
    half = raw.view(torch.float16)

    def value(byte, s, m):
        byte, s, m = (torch.from_numpy(x).to(pool.device) for x in (byte, s, m))
        b = raw[:, byte]
        code = torch.where(odd, torch.div(b, 16, rounding_mode="floor"), b % 16).double()
        return (half[:, m // 2].double() + half[:, s // 2].double() * code).reshape(-1, d)[:n_len]

    return value(k_byte, par[0], par[1]), value(v_byte, par[2], par[3])


def exact(case, seed):
    state = prepare(case, seed)
    kind, d, heads, kv_heads = case["kind"], case["d"], case["heads"], case["kv_heads"]
    lens, new = state["lens"], state["new"]
    if kind == "write":
        return {x: _exact_quantised(state[x].double().cpu().numpy()) for x in ("k", "v")}
    pool, table = state["pool"], state["table"]
    total = sum(new)
    if kind == "read":
        got = [torch.empty((total, kv_heads, d), dtype=torch.float64, device=pool.device) for _ in range(2)]
    else:
        got = [torch.empty((total, heads, d), dtype=torch.float64, device=pool.device)]
    at = 0
    for s, (n_len, n) in enumerate(zip(lens, new)):
        pages = table[s, : -(-n_len // PAGE)]
        for h in range(kv_heads):
            k, v = _exact_rows(pool, pages, n_len, h, d)
            if kind == "read":
                got[0][at:at + n, h], got[1][at:at + n, h] = k[n_len - n:], v[n_len - n:]
                continue
            rep = heads // kv_heads
            for hq in range(h * rep, (h + 1) * rep):
                for a in range(0, n, 1024):
                    q = state["q"][at + a:at + min(n, a + 1024), hq].double()
                    last = n_len - n + a + torch.arange(q.shape[0], device=q.device)
                    s_ = torch.einsum("qd,kd->qk", q, k) / math.sqrt(d)
                    s_[torch.arange(n_len, device=q.device)[None, :] > last[:, None]] = -math.inf
                    got[0][at + a:at + a + q.shape[0], hq] = torch.einsum("qk,kd->qd", torch.softmax(s_, -1), v)
        at += n
    if kind == "read":
        return {"k": got[0], "v": got[1]}
    return {"out": got[0]}
