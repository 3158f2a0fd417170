"""Cases that measure the 4-bit KV cache and the quantised caches around it.

Four operators on a layer's key/value cache:

  write    quantise T new rows into an INT4 cache as they are appended, and
           read them back
  read     read a run of positions of an INT4 or FP8 cache back as bf16 rows
  decode   one token per sequence: rotate q and k, store the new row in the
           INT4 cache, attend the cache with a sink logit per query head
  prefill  T rows on an INT4 or FP8 cache that already holds some

An INT4 row is d / 32 blocks of 32 elements. A block with m its element of
largest magnitude (the positive one of a tie) has the scale s = -m / 8 rounded
to 5 significant bits and the codes u = min(15, floor(x / s + 8.5)); it stands
for s (u - 8), which bf16 holds exactly. Codes lie two to a byte, the even
element in the low half; caches are [B][n_kv][rows][...]. An FP8 row has one
fp32 scale amax / 448 and e4m3 codes.

``own`` false: elementary torch operations. ``own`` true: the library's calls.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 32
THETA, SCALING, ORIG_CTX, ALPHA, BETA = 150000.0, 32.0, 4096, 1.0, 32.0
SEQUENCE_ROWS = 1 << 23   # rows made and quantised at a time


def _case(name, op, B, n_q, n_kv, d, off, T, window=0, ring=0, fmt="int4", fused=False, sink=True):
    return dict(name=name, op=op, B=B, n_q=n_q, n_kv=n_kv, d=d, off=off, T=T, window=window, ring=ring, fmt=fmt,
                fused=fused, sink=sink)


def listed():
    return [
        # one token of every sequence of a serving batch enters the cache
        _case("write_step", "write", 16, 64, 8, 64, off=1000, T=1, fused=True),
        # a training-length prompt batch, heads of 96
        _case("write_prompts_d96", "write", 8, 8, 4, 96, off=0, T=4096),
        # a long prompt out of a fused qkv projection
        _case("write_prompt_fused", "write", 1, 64, 8, 64, off=129, T=8192, fused=True),
        # a whole long context read back, to go on with it in bf16
        _case("read_long", "read", 1, 64, 8, 64, off=131071, T=131071),
        # an odd stretch of an FP8 cache with wide heads
        _case("read_fp8_d128", "read", 3, 16, 4, 128, off=5003, T=4099, fmt="fp8"),
        # the smallest call: a short chat, where latency counts
        _case("decode_short", "decode", 1, 8, 2, 64, off=80, T=1),
        # a band layer, whose ring keeps the last rows only
        _case("decode_band_ring", "decode", 16, 64, 8, 64, off=1501, T=1, window=128, ring=384),
        # an ordinary batch with heads of 96 and an odd length
        _case("decode_batch_d96", "decode", 8, 8, 4, 96, off=4097, T=1),
        # one sequence at the longest context
        _case("decode_long", "decode", 1, 64, 8, 64, off=131071, T=1),
        # a serving batch of long contexts: the largest
        _case("decode_handoff", "decode", 16, 64, 8, 64, off=65536, T=1),
        # the next turn of a long conversation
        _case("prefill_turn", "prefill", 2, 64, 8, 64, off=16384, T=512, fused=True),
        # a band layer's odd chunk on an FP8 cache, heads of 96
        _case("prefill_band_fp8_d96", "prefill", 3, 8, 4, 96, off=1000, T=777, window=128, fmt="fp8"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "read", "decode", "decode", "prefill"])
    d = rng.choice([64, 64, 96, 128])
    n_kv, mult, B = log(1, 8), rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), log(1, 16)
    window = rng.choice([0, 0, 0, 16, 128, 200])
    fmt = rng.choice(["int4", "fp8"]) if op in ("read", "prefill") else "int4"
    ring, off, T = 0, 0, 1
    if op == "write":
        off, T = rng.choice([0, log(1, 2000)]), log(1, 8192)
    elif op == "read":
        off = log(1, 131071)
        T = rng.choice([off, log(1, off)])
    elif op == "decode":
        off = rng.choice([0, log(1, 131071), log(1, 131071), log(1, 131071)])
        if window and rng.random() < 0.5:
            off, ring = min(off, 4000), 384
    else:
        off, T = rng.choice([0, log(1, 16384)]), log(1, 1024)
        while n_kv * mult * T * (off + T) * B > 2 * 64 * 512 * 16896:
            B, T, off = max(1, B // 2), max(1, T // 2), off * 3 // 4
    most = 16 * 65536 * 8 * 64
    while B * n_kv * d * (off + T) > most // 4:
        B, off = max(1, B // 2), off if B > 1 else off // 2
        T = min(T, off) if op == "read" else T
    return {k: v for k, v in _case("", op, B, n_kv * mult, n_kv, d, off, T, window if op in ("decode", "prefill") else 0,
                                   ring, fmt, rng.random() < 0.5, rng.random() < 0.8).items() if k != "name"}


def _row_bytes(case):
    """Bytes of one stored position of one KV head, keys and values."""
    d = case["d"]
    return 2 * (d // 2 + 2 * d // BLOCK) if case["fmt"] == "int4" else 2 * (d + 4)


def _pairs(off, T, window):
    """(query, key) pairs that T rows at positions off.. admit."""
    p = np.arange(off, off + T, dtype=np.int64) + 1
    return int((np.minimum(p, window) if window else p).sum())


def work(case):
    B, n_q, n_kv, d, off, T = (case[k] for k in ("B", "n_q", "n_kv", "d", "off", "T"))
    row, bf16 = _row_bytes(case) * n_kv * B, 2 * 2 * d * n_kv * B   # a position's bytes: stored, and as bf16
    if case["op"] == "write":
        return {"bytes": T * (2 * bf16 + row), "flops": 0}
    if case["op"] == "read":
        return {"bytes": T * (bf16 + row), "flops": 0}
    prefix = min(off, case["window"] - 1) if case["window"] else off
    io = T * B * n_q * (2 * 2 * d + 4)
    return {"bytes": prefix * row + T * (2 * bf16 + row) + io, "flops": 4 * d * n_q * B * _pairs(off, T, case["window"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(seed, stream, shape):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000 + stream) % (1 << 62))
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rope_tables(n, d):
    """YaRN rotary tables (NTK by parts), fp32 [n, d/2]."""
    h = d // 2
    i = torch.arange(h, dtype=torch.float64, device="cuda")
    freq = THETA ** (i / h)
    at = [h * math.log(ORIG_CTX / (x * 2 * math.pi)) / math.log(THETA) for x in (BETA, ALPHA)]
    mask = 1 - ((i - at[0]) / (at[1] - at[0])).clamp(0, 1)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * ((1 - mask) / (SCALING * freq) + mask / freq)
    conc = 0.1 * math.log(SCALING) + 1
    return (conc * angle.cos()).float(), (conc * angle.sin()).float()


def _rows(case, seed, stream, n, first=0):
    """n cache rows [B, n, n_kv, d] bf16 of every sequence: some channels are
    several times as large as others, as keys' are."""
    gain = torch.exp(0.5 * _normal(seed, 7, (case["n_kv"], case["d"])))
    return (_normal(seed, stream + 10 * first, (case["B"], n, case["n_kv"], case["d"])) * gain).to(torch.bfloat16)


def prepare(case, seed):
    B, n_q, n_kv, d, off, T = (case[k] for k in ("B", "n_q", "n_kv", "d", "off", "T"))
    s = dict(case)
    cap = off + T
    s["cap"] = cap = case["ring"] or (cap + 15) // 16 * 16
    if case["fused"]:
        x = _normal(seed, 1, (B, T, d * (n_q + 2 * n_kv))).to(torch.bfloat16)
        q, k, v = (t.unflatten(2, (-1, d)) for t in x.split([n_q * d, n_kv * d, n_kv * d], 2))
    else:
        q = _normal(seed, 1, (B, T, n_q, d)).to(torch.bfloat16)
        k, v = (_normal(seed, i, (B, T, n_kv, d)).to(torch.bfloat16) for i in (2, 3))
    s.update(q=q, k=k, v=v, sinks=_normal(seed, 4, (n_q,)) if case["sink"] else None, scale=1 / math.sqrt(d))
    if case["op"] in ("decode", "prefill"):
        s["cos"], s["sin"] = _rope_tables(off + T, d)
    # the rows that the cache holds already, filled in a run of appends; the
    # cache is the handle that a program keeps (with `own` the library's)
    n = case["ring"] or max(1, SEQUENCE_ROWS // (B * n_kv))
    if own:
        import sink_augmented_gqa_b200 as sa
        s["cache"] = sa.KVCache(B, cap, n_kv, d, ring=case["window"] if case["ring"] else 0,
                                fp8=case["fmt"] == "fp8", int4=case["fmt"] == "int4")
    else:
        bytes_, scales = (d // 2, (d // BLOCK,)) if case["fmt"] == "int4" else (d, ())
        kind = torch.bfloat16 if case["fmt"] == "int4" else torch.float32
        rows = off + T
        for x in ("k", "v"):
            s[x + "_codes"] = torch.zeros((B, n_kv, rows, bytes_), dtype=torch.uint8, device="cuda")
            s[x + "_scales"] = torch.zeros((B, n_kv, rows) + scales, dtype=kind, device="cuda")
    for i, at in enumerate(range(0, off, n)):
        kr, vr = (_rows(case, seed, x, min(n, off - at), i) for x in (5, 6))
        if own:
            s["cache"].append(kr, vr)
        else:
            _store(s, kr, vr, at)
        del kr, vr
    if own:
        s["snapshot"] = s["cache"].snapshot()
        if case["op"] == "decode":
            s["workspace"] = sa.decode_workspace(B, n_q, n_kv, d)
        elif case["op"] == "prefill":
            s["workspace"] = sa.prefill_quant_workspace(s["cache"], T, case["window"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _significant(x, bits):
    """fp64 or fp32 x rounded to so many significant bits, ties to even."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2 ** bits), e - bits)


def _rotate(x, cos, sin, at):
    """RoPE of x [B, T, H, d] at positions at + t: the exact rotation rounded
    once to bf16 (in 64 bits: a result next to a rounding border decides a
    code)."""
    h = x.shape[-1] // 2
    a, b = x[..., :h].double(), x[..., h:].double()
    c, s = (t[at:at + x.shape[1], None].double() for t in (cos, sin))
    return _significant(torch.cat((a * c - b * s, b * c + a * s), -1), 8).to(torch.bfloat16)


def _quantise4(x):
    b = x.float().unflatten(-1, (-1, BLOCK))
    hi, lo = b.amax(-1), b.amin(-1)
    m = torch.where(hi >= -lo, hi, lo)
    s = torch.where(m.abs() < 2.0 ** -120, 0.0, _significant(-m / 8, 5))
    u = torch.where(s[..., None] == 0, 8.0, torch.floor(b / s[..., None] + 8.5)).clamp(0, 15).to(torch.uint8).flatten(-2)
    return u[..., ::2] | u[..., 1::2] << 4, s.to(torch.bfloat16)


def _quantise8(x):
    x = x.float()
    s = x.abs().amax(-1) / torch.full((), 448.0, device=x.device)
    y = x / torch.where(s == 0, 1.0, s)[..., None]
    return y.to(torch.float8_e4m3fn).view(torch.uint8), s


def _store(s, k, v, at):
    """Quantises rows k, v [B, n, n_kv, d] into positions at.. of the state's cache."""
    for x, rows in (("k", k), ("v", v)):
        codes, scales = (_quantise4 if s["fmt"] == "int4" else _quantise8)(rows.transpose(1, 2))
        s[x + "_codes"][:, :, at:at + rows.shape[1]] = codes
        s[x + "_scales"][:, :, at:at + rows.shape[1]] = scales


def _load(s, x, start, stop):
    """Positions [start, stop) as fp32 [B, n_kv, n, d]."""
    codes, scales = s[x + "_codes"][:, :, start:stop], s[x + "_scales"][:, :, start:stop].float()
    if s["fmt"] == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scales[..., None]
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (u.unflatten(-1, (-1, BLOCK)) * scales[..., None]).flatten(-2)


def _read(s, start, stop):
    return tuple(_load(s, x, start, stop).transpose(1, 2).to(torch.bfloat16) for x in ("k", "v"))


def _attend(s):
    """The call's rows stored, then attended together with what the cache
    held: out [B, T, n_q, d], lse [B, n_q, T]."""
    B, T, n_q, d = s["q"].shape
    off, n_kv, window = s["off"], s["n_kv"], s["window"]
    q = _rotate(s["q"], s["cos"], s["sin"], off).float()
    _store(s, _rotate(s["k"], s["cos"], s["sin"], off), s["v"], off)
    lo = max(0, off + 1 - window) if window else 0
    K, V = _load(s, "k", lo, off + T), _load(s, "v", lo, off + T)
    if s["op"] == "prefill":   # which attends the rows as they read back
        K, V = K.to(torch.bfloat16).float(), V.to(torch.bfloat16).float()
    q = q.unflatten(2, (n_kv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [B, n_kv, m T, d]
    scores = (q @ K.transpose(2, 3) * s["scale"]).unflatten(2, (-1, T))
    p, j = torch.arange(off, off + T, device="cuda")[:, None], torch.arange(lo, off + T, device="cuda")
    if T > 1:
        scores.masked_fill_((j > p) | (j <= p - window if window else j < 0), -math.inf)
    sink = s["sinks"].view(n_kv, -1, 1, 1) if s["sinks"] is not None else torch.full((1, 1, 1, 1), -math.inf, device="cuda")
    top = torch.maximum(scores.amax(-1, keepdim=True), sink)
    w = scores.sub_(top).exp_()
    total = w.sum(-1, keepdim=True) + torch.exp(sink - top)
    out = (w.flatten(2, 3) @ V).unflatten(2, (-1, T)) / total
    lse = (top + total.log()).squeeze(-1).flatten(1, 2)
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16), lse


def _run_own(s):
    import sink_augmented_gqa_b200 as sa
    cache, off, T = s["cache"], s["off"], s["T"]
    if s["op"] == "read":
        return cache.read(off - T, off)
    cache.restore(s["snapshot"])
    if s["op"] == "write":
        cache.append(s["k"], s["v"])
        return cache.read(off, off + T)
    call = sa.attn_decode if s["op"] == "decode" else sa.attn_prefill_quant
    out, lse = call(cache, s["q"], s["k"], s["v"], s["sinks"], s["window"], s["scale"], s["cos"], s["sin"],
                    workspace=s["workspace"], return_lse=True)
    return (out, lse) + cache.read(off, off + T)


def run(s):
    if own:
        return _run_own(s)
    off, T = s["off"], s["T"]
    if s["op"] == "read":
        return _read(s, off - T, off)
    if s["op"] == "write":
        _store(s, s["k"], s["v"], off)
        return _read(s, off, off + T)
    return _attend(s) + _read(s, off, off + T)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _to_bf16(x):
    """numpy fp64 rounded once to 8 significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def _stands_for(fmt, x):
    """What the rows x (fp64, bf16 values) stand for once stored."""
    if fmt == "fp8":
        s = (x.abs().amax(-1, keepdim=True).float() / torch.tensor([448.0], device=x.device))
        y = (x.float() / torch.where(s == 0, torch.ones_like(s), s)).to(torch.float8_e4m3fn)
        return y.double() * s.double()
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK))
    top, bottom = b.max(-1, keepdim=True).values, b.min(-1, keepdim=True).values
    m = torch.where(top + bottom >= 0, top, bottom)
    s = torch.from_numpy(np.ldexp(np.rint(np.frexp(-m.cpu().numpy() / 8)[0] * 32),
                                  np.frexp(-m.cpu().numpy() / 8)[1] - 5)).to(x.device)
    y = b / torch.where(s == 0, torch.ones_like(s), s)
    u = torch.zeros_like(y)
    for step in range(1, 16):   # the codes' borders, a value on one going up
        u += y >= step - 8.5
    return (s * (u - 8)).reshape(x.shape)


def exact(case, seed):
    B, n_q, n_kv, d, off, T, window = (case[k] for k in ("B", "n_q", "n_kv", "d", "off", "T", "window"))
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    held = lambda x, b, g, lo: _held(case, s, x, b, g, lo, off)   # noqa: E731
    if case["op"] == "read":
        return tuple(torch.stack([torch.stack([held(x, b, g, off - T) for g in range(n_kv)], 1) for b in range(B)])
                     .to(torch.bfloat16).double() for x in ("k", "v"))
    cos = s["cos"][off:].double().cpu().numpy()[:, None] if case["op"] != "write" else None
    sin = s["sin"][off:].double().cpu().numpy()[:, None] if case["op"] != "write" else None

    def rotated(x):
        x = x.double().cpu().numpy()
        if cos is not None:
            re, im = x[..., :d // 2], x[..., d // 2:]
            x = _to_bf16(np.concatenate([re * cos - im * sin, im * cos + re * sin], -1))
        return torch.from_numpy(x).cuda()

    k_new, v_new = _stands_for(case["fmt"], rotated(s["k"])), _stands_for(case["fmt"], s["v"].double())
    back = tuple(t.to(torch.bfloat16).double() for t in (k_new, v_new))
    if case["op"] == "write":
        return back
    if case["op"] == "prefill":
        k_new, v_new = back
    q = rotated(s["q"])
    out = torch.empty((B, T, n_q, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, n_q, T), dtype=torch.float64, device="cuda")
    lo = max(0, off - window + 1) if window else 0
    age = torch.arange(off, off + T, device="cuda")[:, None] - torch.arange(lo, off + T, device="cuda")[None]
    seen = (age >= 0) & (age < window) if window else age >= 0
    for b in range(B):
        for h in range(n_q):
            g = h * n_kv // n_q
            if h % (n_q // n_kv) == 0:
                K, V = (torch.cat([held(x, b, g, lo), new[b, :, g]]) for x, new in (("k", k_new), ("v", v_new)))
                if case["op"] == "prefill":
                    K, V = K.to(torch.bfloat16).double(), V.to(torch.bfloat16).double()
            z = torch.where(seen, q[b, :, h] @ K.T / math.sqrt(d), -math.inf)
            if s["sinks"] is not None:
                z = torch.cat([z, s["sinks"][h].double().expand(T, 1)], 1)
            lse[b, h] = torch.logsumexp(z, 1)
            out[b, :, h] = torch.exp(z[:, :K.shape[0]] - lse[b, h][:, None]) @ V
    return (out, lse) + back


def _held(case, s, x, b, g, lo, hi):
    """Stored positions [lo, hi) of one head in fp64."""
    codes, scales = s[x + "_codes"][b, g, lo:hi], s[x + "_scales"][b, g, lo:hi].double()
    if case["fmt"] == "fp8":
        return codes.view(torch.float8_e4m3fn).double() * scales[:, None]
    low, high = codes.remainder(16), codes.div(16, rounding_mode="floor")
    u = torch.empty((hi - lo, case["d"]), dtype=torch.float64, device="cuda")
    u[:, 0::2], u[:, 1::2] = low.double(), high.double()
    return (u - 8) * scales.repeat_interleave(BLOCK, -1)
