"""Cases, inputs and plain forms of attention over shared and windowed parts of the latent cache.

Four operators.  ``SharedPrefix`` decompresses a prefix of the paged cache into keys and values for
every head, once for all sequences that share it; ``mla_prefix_attend`` lets the query rows of a whole
batch attend to that prefix in one scan and merges each row's attention over its sequence's own tokens.
``DecodeStep(window=, sinks=)`` is the decode step in which a token sees the last ``window`` tokens and
the first ``sinks`` ones, and ``mla_prefill_window`` the same for a chunk of new tokens.  ``run``
computes an operator in elementary torch operations, or, where ``own`` is true, makes the framework's
call.
"""
import math

import torch

own = False

DEV = "cuda"
HEADS, D_C, D_HC, D_R, ROW, PAGE = 128, 512, 128, 64, 576, 64
SCALE = 1.0 / math.sqrt(D_HC + D_R)


def listed():
    op, pre = {"op": "open"}, {"op": "prefix"}
    win, chunk = {"op": "window"}, {"op": "chunk"}
    return [
        # a system prompt of 4,100 tokens made ready for the batches that will share it
        {"name": "open_4100_bf16", **op, "tokens": 4100, "cache": "bf16"},
        # a shorter one out of an FP8 cache
        {"name": "open_1001_fp8", **op, "tokens": 1001, "cache": "fp8"},
        # the smallest: two sequences behind a prompt of 513 tokens
        {"name": "prefix_2x513", **pre, "rows": 2, "tokens": 513},
        # an odd batch behind a prompt of a few pages
        {"name": "prefix_37x2001", **pre, "rows": 37, "tokens": 2001},
        # a decode batch behind a long instruction
        {"name": "prefix_64x8192", **pre, "rows": 64, "tokens": 8192},
        # many samples of one long prompt
        {"name": "prefix_256x16384", **pre, "rows": 256, "tokens": 16384},
        # one long conversation with a window of 4,096 and four sink tokens
        {"name": "window_1x4096", **win, "batch": 1, "queries": 1, "lo": 65536, "hi": 65536, "window": 4096,
         "sinks": 4, "cache": "bf16"},
        # a ragged batch, lengths from 128 to 32,768, a window of 1,024 and a page of sinks
        {"name": "window_64x1024", **win, "batch": 64, "queries": 1, "lo": 128, "hi": 32768, "window": 1024,
         "sinks": 64, "cache": "bf16"},
        # four drafts for each of 16 sequences, odd window and sinks
        {"name": "window_16q4x2047", **win, "batch": 16, "queries": 4, "lo": 8000, "hi": 8192, "window": 2047,
         "sinks": 5, "cache": "bf16"},
        # the FP8 cache at its benchmark batch
        {"name": "window_128x4096_fp8", **win, "batch": 128, "queries": 1, "lo": 8192, "hi": 8192, "window": 4096,
         "sinks": 4, "cache": "fp8"},
        # a prompt's chunk of 4,096 behind 12,288 tokens, a window of 1,024
        {"name": "chunk_4096x1024", **chunk, "tokens": 4096, "length": 16384, "window": 1024, "sinks": 4,
         "cache": "bf16"},
        # a short odd chunk out of an FP8 cache, no sinks
        {"name": "chunk_257x511_fp8", **chunk, "tokens": 257, "length": 5001, "window": 511, "sinks": 0,
         "cache": "fp8"},
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["open", "prefix", "prefix", "window", "window", "chunk"])
    if op == "open":
        return {"op": op, "tokens": _log(rng, 64, 4100), "cache": rng.choice(["bf16", "fp8", "nvfp4"])}
    if op == "prefix":
        return {"op": op, "rows": _log(rng, 1, 256), "tokens": _log(rng, 64, 16384)}
    sinks = rng.choice([0, 1, 4, rng.randrange(2, 129)])
    cache = rng.choice(["bf16", "bf16", "fp8"])
    if op == "window":
        q = rng.choice([1, 1, 1, 2, 4])
        lo = _log(rng, 64, 32768)
        return {"op": op, "batch": _log(rng, 1, 128 // q), "queries": q, "lo": lo,
                "hi": min(65536, lo + rng.choice([0, rng.randrange(1, 4096)])), "window": _log(rng, 16, 4096),
                "sinks": sinks, "cache": cache}
    tokens = _log(rng, 256, 4096)
    return {"op": op, "tokens": tokens, "length": min(16384, tokens + rng.randrange(0, 12289)),
            "window": _log(rng, 16, 1024), "sinks": sinks, "cache": rng.choice([cache, "nvfp4"])}


# ---------------------------------------------------------------------------------- inputs

def _lengths(case, seed):
    """The sequences' lengths, from the seed alone."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    lo = max(case["lo"], case["queries"])
    return torch.randint(lo, max(case["hi"], lo) + 1, (case["batch"],), generator=gen).tolist()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).bfloat16()

    def cache(pages):
        """A pool of latent rows N(0, 1): bf16 rows, or codes, scales and rotary keys."""
        if case["cache"] == "bf16":
            return {"kv_pool": normal(pages, PAGE, ROW)}
        spread = torch.exp2(torch.randn(pages, PAGE, generator=gen, device=DEV) * 0.25)
        kr = normal(pages, PAGE, D_R)
        if case["cache"] == "fp8":
            c = torch.randn(pages, PAGE, D_C, generator=gen, device=DEV) * spread[..., None]
            sigma = c.abs().amax(dim=-1) / 448.0
            return {"kv_pool": (c / sigma[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), "kv_scale": sigma,
                    "kr_pool": kr}
        codes = torch.randint(0, 256, (pages, PAGE, D_C // 2), generator=gen, device=DEV, dtype=torch.uint8)
        blocks = torch.randint(0x58, 0x7F, (pages, PAGE, D_C // 16), generator=gen, device=DEV, dtype=torch.uint8)
        return {"kv_pool": torch.cat([codes, blocks], dim=-1), "kv_scale": spread / 480.0, "kr_pool": kr}

    s = {"case": dict(case)}
    if op in ("open", "window", "chunk"):
        s["w_uk"] = normal(HEADS, D_HC, D_C, std=D_C ** -0.5)
        s["w_uv"] = normal(HEADS, D_HC, D_C, std=D_C ** -0.5)
        s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op == "open":
        pages = (case["tokens"] + PAGE - 1) // PAGE
        s["kv"] = cache(pages)
        s["table"] = torch.randperm(pages, generator=gen, device=DEV).int()
    elif op == "prefix":
        R, P = case["rows"], case["tokens"]
        # the prefix as its cache rows and its decompressed keys and values, kept in bf16; the latents'
        # products with weights N(0, 1/512) are N(0, 1)
        s["k"], s["v"] = normal(HEADS, P, D_HC), normal(HEADS, P, D_HC)
        s["k_r"] = normal(P, ROW)[:, D_C:]
        s["q_c"], s["q_r"] = normal(R, HEADS, D_HC), normal(R, HEADS, D_R)
        # every row's attention over its own tokens: some 1 to 4,096 of them
        s["own_out"] = normal(R, HEADS, D_HC, std=0.1)
        s["own_lse"] = torch.rand(R, HEADS, generator=gen, device=DEV) * math.log(4096.0) + 0.5
        s["out"] = torch.empty(R, HEADS, D_HC, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(R, HEADS, dtype=torch.float32, device=DEV)
    else:
        # the pool holds the pages that some query still sees; the table's other entries are -1
        lens = _lengths(case, seed) if op == "window" else [case["length"]]
        q = case["queries"] if op == "window" else case["tokens"]
        W, n = case["window"], case["sinks"]
        width = (max(lens) + PAGE - 1) // PAGE
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        held = []
        for b, S in enumerate(lens):
            first = max(0, S - q + 1 - W) // PAGE
            held += [(b, p) for p in range((S + PAGE - 1) // PAGE) if p >= first or p * PAGE < n]
        s["kv"] = cache(len(held))
        place = torch.randperm(len(held), generator=gen, device=DEV).int().cpu()
        at = torch.tensor(held)
        table[at[:, 0], at[:, 1]] = place
        s["lens"], s["table"] = lens, table.to(DEV)
        rows = len(lens) * q
        s["q_c"], s["q_r"] = normal(rows, HEADS, D_HC), normal(rows, HEADS, D_R)
        s["out"] = torch.empty(rows, HEADS, D_HC, dtype=torch.bfloat16, device=DEV)
    if own:
        _handle(s)
    return s


def _values(kv, slots):
    """Cache rows `slots` as the values they stand for: latents [..., 512] and rotary keys [..., 64], 32 bits."""
    pool = kv["kv_pool"].flatten(0, 1)[slots]
    if "kv_scale" not in kv:
        return pool[..., :D_C].float(), pool[..., D_C:].float()
    sigma = kv["kv_scale"].flatten()[slots][..., None]
    if pool.shape[-1] == D_C:
        c = pool.view(torch.float8_e4m3fn).float() * sigma
    else:
        both = torch.stack([pool[..., :256] & 15, pool[..., :256] >> 4], dim=-1).flatten(-2)
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
        c = torch.where(both >= 8, -1.0, 1.0) * grid[(both & 7).long()]
        c = c * pool[..., 256:].contiguous().view(torch.float8_e4m3fn).float().repeat_interleave(16, dim=-1) * sigma
    return c, kv["kr_pool"].flatten(0, 1)[slots].float()


# ---------------------------------------------------------------------------------- one pass

def _plain_open(s):
    at = torch.arange(s["case"]["tokens"], device=DEV)
    c, kr = _values(s["kv"], s["table"].long()[at // PAGE] * PAGE + at % PAGE)
    return {"k": torch.matmul(c, s["w_uk"].float().transpose(1, 2)).bfloat16(),
            "v": torch.matmul(c, s["w_uv"].float().transpose(1, 2)).bfloat16(), "k_r": kr.bfloat16()}


def _plain_prefix(s):
    kr, out, lse = s["k_r"].float(), [], []
    for h in range(0, HEADS, 16):  # sixteen heads' scores at a time
        q_c, q_r = s["q_c"][:, h:h + 16].float().transpose(0, 1), s["q_r"][:, h:h + 16].float().transpose(0, 1)
        x = (torch.matmul(q_c, s["k"][h:h + 16].float().transpose(1, 2)) + torch.matmul(q_r, kr.T)) * SCALE
        own_lse = s["own_lse"][:, h:h + 16].T[..., None]
        top = torch.maximum(x.amax(dim=-1, keepdim=True), own_lse)
        p, w = torch.exp(x - top), torch.exp(own_lse - top)
        total = p.sum(dim=-1, keepdim=True) + w
        o = torch.matmul(p, s["v"][h:h + 16].float()) + w * s["own_out"][:, h:h + 16].float().transpose(0, 1)
        out.append((o / total).transpose(0, 1))
        lse.append((top + torch.log(total))[..., 0].T)
    return {"out": torch.cat(out, dim=1).bfloat16(), "lse": torch.cat(lse, dim=1)}


def _visible(s):
    """For every query row the positions it sees, padded to the longest: [rows, most] and whether each counts."""
    case = s["case"]
    W, n, q = case["window"], case["sinks"], case["queries"]
    lens = torch.tensor(s["lens"], device=DEV)
    last = (lens[:, None] - q + torch.arange(q, device=DEV)).flatten()[:, None]
    first = (last - W + 1).clamp(min=0)
    sink = torch.arange(n, device=DEV)[None, :].expand(last.shape[0], n)
    near = first + torch.arange(min(W, max(s["lens"])), device=DEV)[None, :]
    return torch.cat([sink, near], dim=1), torch.cat([sink < first, near <= last], dim=1)


def _plain_window(s):
    case = s["case"]
    pos, live = _visible(s)
    pos = torch.where(live, pos, 0)
    seq = torch.arange(case["batch"], device=DEV).repeat_interleave(case["queries"])[:, None]
    page = s["table"].long()[seq, pos // PAGE]
    c, kr = _values(s["kv"], torch.where(live, page * PAGE + pos % PAGE, 0))
    q_abs = torch.matmul(s["q_c"].float().transpose(0, 1), s["w_uk"].float()).transpose(0, 1)
    x = (torch.matmul(q_abs, c.transpose(1, 2)) + torch.matmul(s["q_r"].float(), kr.transpose(1, 2))) * SCALE
    x = x.masked_fill(~live[:, None, :], float("-inf"))
    p = torch.exp(x - x.amax(dim=-1, keepdim=True))
    o = torch.matmul(p, c) / p.sum(dim=-1, keepdim=True)
    return {"out": torch.matmul(o.transpose(0, 1), s["w_uv"].float().transpose(1, 2)).transpose(0, 1).bfloat16()}


def _span(s):
    """A chunk's visible positions: the sinks and everything from the first query's window on."""
    case = s["case"]
    first = max(0, case["length"] - case["tokens"] + 1 - case["window"])
    at = torch.arange(case["length"], device=DEV)
    return at[(at >= first) | (at < case["sinks"])]


def _plain_chunk(s):
    case = s["case"]
    at = _span(s)
    c, kr = _values(s["kv"], s["table"].long()[0, at // PAGE] * PAGE + at % PAGE)
    pos = torch.arange(case["length"] - case["tokens"], case["length"], device=DEV)[:, None]
    seen = (at <= pos) & ((at > pos - case["window"]) | (at < case["sinks"]))
    out = []
    for h in range(0, HEADS, 8):  # eight heads' scores at a time
        k = torch.matmul(c, s["w_uk"][h:h + 8].float().transpose(1, 2))
        v = torch.matmul(c, s["w_uv"][h:h + 8].float().transpose(1, 2))
        q_c, q_r = s["q_c"][:, h:h + 8].float().transpose(0, 1), s["q_r"][:, h:h + 8].float().transpose(0, 1)
        x = (torch.matmul(q_c, k.transpose(1, 2)) + torch.matmul(q_r, kr.T)) * SCALE
        x = x.masked_fill(~seen, float("-inf"))
        p = torch.exp(x - x.amax(dim=-1, keepdim=True))
        out.append((torch.matmul(p, v) / p.sum(dim=-1, keepdim=True)).transpose(0, 1))
    return {"out": torch.cat(out, dim=1).bfloat16()}


def _handle(s):
    """What a program makes once and keeps: the prefix, the step's captured graph, workspaces."""
    if "handle" in s:
        return s["handle"]
    from mla_latent_kv_absorb_gb300 import binding

    case = s["case"]
    if case["op"] == "prefix":
        s["handle"] = binding.SharedPrefix.of(s["k"], s["v"], s["k_r"])
        s["workspace"] = s["handle"].workspace(case["rows"])
    elif case["op"] == "window":
        step = binding.DecodeStep(s["lens"], w_uk=s["w_uk"], w_uv=s["w_uv"], block_table=s["table"],
                                  queries_per_seq=case["queries"], window=case["window"], sinks=case["sinks"], **s["kv"])
        s["handle"], s["graph"] = step, step.capture(s["q_c"], s["q_r"])
    elif case["op"] == "chunk":
        size = binding.mla_prefill_window_workspace_bytes(case["length"], case["tokens"], case["window"], case["sinks"])
        s["handle"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    else:
        s["handle"] = None
    return s["handle"]


def _own(s):
    from mla_latent_kv_absorb_gb300 import binding

    case, handle = s["case"], _handle(s)
    if case["op"] == "open":
        p = binding.SharedPrefix(case["tokens"], w_uk=s["w_uk"], w_uv=s["w_uv"], block_table_row=s["table"],
                                 dev_error=s["err"], **s["kv"])
        return {"k": p.k, "v": p.v, "k_r": p.k_r}
    if case["op"] == "prefix":
        binding.mla_prefix_attend(handle, s["q_c"], s["q_r"], s["out"], lse=s["lse"], own_out=s["own_out"],
                                  own_lse=s["own_lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "window":
        s["graph"].replay()
        return {"out": handle.out}
    binding.mla_prefill_window(block_table_row=s["table"][0], seq_len=case["length"], window=case["window"],
                               sinks=case["sinks"], q_c=s["q_c"], q_r=s["q_r"], w_uk=s["w_uk"], w_uv=s["w_uv"],
                               out=s["out"], dev_error=s["err"], workspace=handle, **s["kv"])
    return {"out": s["out"]}


def run(s):
    if own:
        return _own(s)
    return {"open": _plain_open, "prefix": _plain_prefix, "window": _plain_window,
            "chunk": _plain_chunk}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------------- the work

ROW_BYTES = {"bf16": 1152, "fp8": 512 + 4 + 128, "nvfp4": 288 + 4 + 128}


def work(case):
    op = case["op"]
    weights = 2 * HEADS * D_HC * D_C * 2
    pair = 2 * HEADS * (D_HC + D_R + D_HC)  # one query row and one key, decompressed
    if op == "open":
        P = case["tokens"]
        return {"bytes": P * (ROW_BYTES[case["cache"]] + 2 * HEADS * D_HC * 2 + 128) + weights,
                "flops": 2 * 2 * P * D_C * HEADS * D_HC}
    if op == "prefix":
        R, P = case["rows"], case["tokens"]
        return {"bytes": P * (2 * HEADS * D_HC * 2 + 128) + R * HEADS * (D_HC + D_R + 2 * D_HC) * 2 + 2 * R * HEADS * 4,
                "flops": R * P * pair}
    W, n = case["window"], case["sinks"]
    if op == "window":
        q, rows = case["queries"], case["batch"] * case["queries"]
        mean = (case["lo"] + case["hi"]) // 2
        seen = min(mean, W + n)
        return {"bytes": case["batch"] * min(mean, W + n + q - 1) * ROW_BYTES[case["cache"]] + weights +
                rows * HEADS * (D_HC + D_R + D_HC) * 2,
                # absorbed: a row's 128 heads against each token's 576 and 512 values, and the two products
                "flops": rows * (seen * 2 * HEADS * (ROW + D_C) + 4 * HEADS * D_HC * D_C)}
    T, S = case["tokens"], case["length"]
    held = min(S, T + W - 1 + n)
    pairs = sum(min(p + 1, W + min(n, max(0, p + 1 - W))) for p in range(S - T, S))
    return {"bytes": held * ROW_BYTES[case["cache"]] + weights + T * HEADS * (D_HC + D_R + D_HC) * 2,
            "flops": pairs * pair + 2 * 2 * held * D_C * HEADS * D_HC}


# ---------------------------------------------------------------------------------- 64 bits

def _rows64(kv, slots):
    """Cache rows in 64 bits (the quantised ones decoded by their fields)."""
    pool = kv["kv_pool"].reshape(-1, kv["kv_pool"].shape[-1]).index_select(0, slots)
    if "kv_scale" not in kv:
        pool = pool.double()
        return pool[:, :D_C], pool[:, D_C:]

    def e4m3(code):  # sign, four exponent bits (bias 7), three mantissa bits
        code = code.double()
        mag = torch.remainder(code, 128)
        e, m = torch.div(mag, 8, rounding_mode="floor"), torch.remainder(mag, 8)
        return torch.where(code >= 128, -1.0, 1.0) * torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m * 2.0 ** -9)

    sigma = kv["kv_scale"].reshape(-1).index_select(0, slots).double().unsqueeze(1)
    kr = kv["kr_pool"].reshape(-1, D_R).index_select(0, slots).double()
    if pool.shape[1] == D_C:
        return e4m3(pool) * sigma, kr
    code = torch.empty(pool.shape[0], D_C, dtype=torch.float64, device=DEV)
    code[:, 0::2] = torch.remainder(pool[:, :256], 16).double()
    code[:, 1::2] = torch.div(pool[:, :256], 16, rounding_mode="floor").double()
    mag = torch.remainder(code, 8)
    e, m = torch.div(mag, 2, rounding_mode="floor"), torch.remainder(mag, 2)
    value = torch.where(code >= 8, -1.0, 1.0) * torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2)
    return value * e4m3(pool[:, 256:]).repeat_interleave(16, dim=1) * sigma, kr


def _attend64(q_c, q_r, k, v, kr, seen=None):
    """One head: queries [T, 128] and [T, 64], keys and values [n, 128], rotary keys [n, 64]."""
    x = (q_c.double() @ k.double().T + q_r.double() @ kr.double().T) / math.sqrt(192.0)
    if seen is not None:
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, dim=1)
    return torch.softmax(x, dim=1) @ v.double(), lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "open":
        at = torch.arange(case["tokens"], device=DEV)
        c, kr = _rows64(s["kv"], s["table"][torch.div(at, PAGE, rounding_mode="floor")].long() * PAGE + at.remainder(PAGE))
        k, v = (torch.einsum("pc,hdc->hpd", c, w.double()) for w in (s["w_uk"], s["w_uv"]))
        return {"k": k, "v": v, "k_r": kr}
    if op == "prefix":
        R = case["rows"]
        out = torch.empty(R, HEADS, D_HC, dtype=torch.float64, device=DEV)
        lse = torch.empty(R, HEADS, dtype=torch.float64, device=DEV)
        for h in range(HEADS):
            o, part = _attend64(s["q_c"][:, h], s["q_r"][:, h], s["k"][h], s["v"][h], s["k_r"])
            mine = s["own_lse"][:, h].double()
            lse[:, h] = torch.logaddexp(part, mine)
            out[:, h] = o * (part - lse[:, h]).exp()[:, None] + \
                s["own_out"][:, h].double() * (mine - lse[:, h]).exp()[:, None]
        return {"out": out, "lse": lse}
    W, n = case["window"], case["sinks"]
    if op == "window":
        q, rows = case["queries"], []
        for b, S in enumerate(s["lens"]):
            for t in range(q):
                last = S - q + t
                at = torch.tensor([j for j in range(last + 1) if j < n or j > last - W], device=DEV)
                c, kr = _rows64(s["kv"], s["table"][b].long()[at // PAGE] * PAGE + at % PAGE)
                r = b * q + t
                # (q W_UK) c = q (W_UK c): the keys are never formed
                folded = torch.einsum("hd,hdc->hc", s["q_c"][r].double(), s["w_uk"].double())
                x = (folded @ c.T + s["q_r"][r].double() @ kr.T) / math.sqrt(192.0)
                rows.append(torch.einsum("hc,hdc->hd", torch.softmax(x, dim=1) @ c, s["w_uv"].double()))
        return {"out": torch.stack(rows)}
    T, S = case["tokens"], case["length"]
    at = _span(s)
    c, kr = _rows64(s["kv"], s["table"][0].long()[at // PAGE] * PAGE + at % PAGE)
    behind = torch.arange(S - T, S, device=DEV)[:, None] - at[None, :]  # how far each key lies behind each query
    seen = (behind >= 0) & ((behind < W) | (at[None, :] < n))
    out = torch.empty(T, HEADS, D_HC, dtype=torch.float64, device=DEV)
    for h in range(HEADS):
        out[:, h] = _attend64(s["q_c"][:, h], s["q_r"][:, h], c @ s["w_uk"][h].double().T, c @ s["w_uv"][h].double().T,
                              kr, seen)[0]
    return {"out": out}
