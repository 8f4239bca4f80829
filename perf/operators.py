"""Cases, inputs and plain forms of the operators around the decode step.

Three operators: ``mla_rope`` (rotary positions on part of a head), ``mla_rope_append_kv`` (new
tokens into the paged latent cache, the position rotation applied on the way, the tokens' queries
rotated and split in the same call) and ``mla_linear_w4`` (few-row products with 4-bit weights and
group scales).  ``run`` computes an operator in elementary torch operations, or, where ``own`` is
true, makes the framework's call.
"""
import math

import torch

own = False

DEV = "cuda"
HEADS, D_C, D_HC, D_R, ROW, PAGE = 128, 512, 128, 64, 576, 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# The long-context scaling of the rotary cases: 4,096 trained positions stretched 40 times.
YARN = {"scaling": "yarn", "factor": 40.0, "original_len": 4096}
NONE = {"scaling": "none", "factor": 1.0, "original_len": 0}
LINEAR = {"scaling": "linear", "factor": 4.0, "original_len": 0}


def listed():
    rope = {"op": "rope", "base": 10000.0}
    app = {"op": "append", "base": 10000.0, "layout": "interleaved"}
    w4 = {"op": "w4"}
    return [
        # the query of one new token: q [1, 128, 192] into q_c and the rotated q_R
        {"name": "rope_q_1", **rope, **YARN, "layout": "interleaved", "tokens": 1, "heads": 128, "head_dim": 192,
         "dim": 64, "offset": 128, "dtype": "bf16", "split": True, "pos_lo": 0, "pos_hi": 163840, "pitch": 0},
        # a decode batch of 64 sequences at contexts up to 32,768, halves layout
        {"name": "rope_q_64", **rope, **NONE, "layout": "half", "tokens": 64, "heads": 128, "head_dim": 192,
         "dim": 64, "offset": 128, "dtype": "bf16", "split": True, "pos_lo": 0, "pos_hi": 32768, "pitch": 0},
        # the queries of a prefill chunk: 4,096 new tokens behind a long prefix
        {"name": "rope_q_4096", **rope, **YARN, "layout": "interleaved", "tokens": 4096, "heads": 128,
         "head_dim": 192, "dim": 64, "offset": 128, "dtype": "bf16", "split": True, "pos_lo": 12288,
         "pos_hi": 16384, "pitch": 0},
        # cached keys moved to other positions: k_R out of gathered rows of 576, rotated back by a shift
        {"name": "rope_keys_65537", **rope, **LINEAR, "layout": "half", "tokens": 65537, "heads": 1, "head_dim": 64,
         "dim": 64, "offset": 0, "dtype": "bf16", "split": False, "pos_lo": -4096, "pos_hi": 0, "pitch": 576},
        # one new token of one sequence into a bf16 cache, with its query
        {"name": "append_1_bf16_q", **app, **YARN, "tokens": 1, "cache": "bf16", "pages": 33, "query": True,
         "pitch": 576},
        # one new token of each of 128 sequences into an FP8 cache, with their queries
        {"name": "append_128_fp8_q", **app, **NONE, "tokens": 128, "cache": "fp8", "pages": 2048, "query": True,
         "pitch": 576},
        # a prefill chunk of odd length into a bf16 cache, rows out of a wider projection
        {"name": "append_4097_bf16", **app, **YARN, "tokens": 4097, "cache": "bf16", "pages": 256, "query": False,
         "pitch": 2112},
        # a prompt into an NVFP4 cache and out again as the rows that the decompressed prefill reads
        {"name": "append_4096_nvfp4", **app, **YARN, "tokens": 4096, "cache": "nvfp4", "pages": 64, "query": False,
         "pitch": 576},
        # the absorb of one sequence's query: W_UK in int4, groups of 32
        {"name": "w4_absorb_1", **w4, "rows": 1, "heads": 128, "n": 512, "k": 128, "format": "int4", "group": 32,
         "zero": False},
        # the value projection of a decode batch of 16: W_UV in NVFP4
        {"name": "w4_out_16", **w4, "rows": 16, "heads": 128, "n": 128, "k": 512, "format": "nvfp4", "group": 16,
         "zero": False},
        # the output projection (128 heads x 128 into 8,192) of one token, int4 with zero points
        {"name": "w4_dense_1", **w4, "rows": 1, "heads": 1, "n": 8192, "k": 16384, "format": "int4", "group": 128,
         "zero": True},
        # the same projection for 33 tokens (drafts of a small batch), groups of 64
        {"name": "w4_dense_33", **w4, "rows": 33, "heads": 1, "n": 8192, "k": 16384, "format": "int4", "group": 64,
         "zero": False},
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "w4"])
    scale = dict(rng.choice([YARN, NONE, LINEAR]))
    if scale["scaling"] != "none":
        scale["factor"] = rng.choice([2.0, 4.0, 8.0, 40.0])
    if op == "rope":
        heads = rng.choice([1, 5, 16, 64, 128])
        dim, rest = rng.choice([(64, 128), (64, 0), (64, 64), (32, 96), (128, 0)])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 4096 * 128 * 192 // (heads * (dim + rest) * (2 if dtype == "fp32" else 1))
        lo = rng.choice([0, 0, 4096, 100000, -8192])
        return {"op": "rope", "base": rng.choice([10000.0, 500000.0]), **scale,
                "layout": rng.choice(["interleaved", "half"]), "tokens": _log(rng, 1, min(65537, most)),
                "heads": heads, "head_dim": dim + rest, "dim": dim, "offset": rng.choice([0, rest]),
                "dtype": dtype, "split": bool(rest and rng.random() < 0.6), "pos_lo": lo,
                "pos_hi": lo + _log(rng, 64, 163840), "pitch": 0}
    if op == "append":
        n = _log(rng, 1, 4097)
        cache = rng.choice(["bf16", "fp8", "nvfp4"])
        pages = (n + PAGE - 1) // PAGE + (0 if cache == "nvfp4" else _log(rng, 1, 512))
        return {"op": "append", "base": 10000.0, **scale, "layout": rng.choice(["interleaved", "half"]),
                "tokens": n, "cache": cache, "pages": pages, "query": n <= 512 and rng.random() < 0.6,
                "pitch": rng.choice([576, 576, 640, 2112])}
    fmt = rng.choice(["int4", "int4", "nvfp4"])
    group = 16 if fmt == "nvfp4" else rng.choice([32, 64, 128])
    if rng.random() < 0.4:
        heads, (n, k) = 128, rng.choice([(512, 128), (128, 512)])
    else:
        heads, n = 1, _log(rng, 200, 8192)
        k = max(group, 32) * max(1, _log(rng, 512, 16384) // max(group, 32))
    return {"op": "w4", "rows": _log(rng, 1, 33), "heads": heads, "n": n, "k": k, "format": fmt, "group": group,
            "zero": fmt == "int4" and rng.random() < 0.5}


# ---------------------------------------------------------------------------------- inputs

def _frequencies(case):
    """(inverse frequencies in 64 bits, multiplier of cos and sin) of the case's scaling."""
    dim = case.get("dim", D_R)
    i = torch.arange(dim // 2, dtype=torch.float64)
    freq = case["base"] ** (-2.0 * i / dim)
    if case["scaling"] == "linear":
        return freq / case["factor"], 1.0
    if case["scaling"] == "yarn":
        # pairs that turn more than 32 times over the trained length keep their frequency, those that
        # turn less than once are slowed by the factor, a linear ramp over the pair index between
        def pair(turns):
            return dim * math.log(case["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(case["base"]))

        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), dim - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return freq * (1 - ramp) + freq / case["factor"] * ramp, 0.1 * math.log(case["factor"]) + 1.0
    return freq, 1.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=DEV).to(dtype)

    def integers(lo, hi, *shape, dtype=torch.int32):
        return torch.randint(lo, hi, shape, generator=gen, device=DEV, dtype=dtype)

    s = {"case": dict(case)}
    if case["op"] in ("rope", "append"):
        freq, s["mult"] = _frequencies(case)
        s["freq"] = freq.to(DEV)
    if case["op"] == "rope":
        T, H, D, dt = case["tokens"], case["heads"], case["head_dim"], DTYPES[case["dtype"]]
        if case["pitch"]:  # the last head_dim of rows of `pitch`
            s["x"] = normal(T, case["pitch"], dtype=dt)[:, case["pitch"] - H * D:].unflatten(1, (H, D))
        else:
            s["x"] = normal(T, H, D, dtype=dt)
        s["positions"] = integers(case["pos_lo"], case["pos_hi"], T)
        rot = case["dim"]
        s["out"] = torch.empty(T, H, rot if case["split"] else D, dtype=dt, device=DEV)
        s["rest"] = torch.empty(T, H, D - rot, dtype=dt, device=DEV) if case["split"] else None
    elif case["op"] == "append":
        n, pages = case["tokens"], case["pages"]
        # the row that the layer's down projection gives: c_KV then k_R, the last 576 of `pitch`
        rows = normal(n, case["pitch"])[:, case["pitch"] - ROW:]
        spread = torch.exp2(torch.randn(n, 1, generator=gen, device=DEV)).to(torch.bfloat16)
        rows[:, :D_C] *= spread
        s["c_kv"], s["k_r"] = rows[:, :D_C], rows[:, D_C:]
        s["positions"] = integers(0, 163840, n)
        s["dev_error"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        order = torch.randperm(pages, generator=gen, device=DEV)
        if case["cache"] == "nvfp4":  # one prompt: its pages in shuffled order, its rows read back
            used = (n + PAGE - 1) // PAGE
            s["table"] = order[:used].to(torch.int32).reshape(1, -1)
            s["slots"] = ((order[:used] * PAGE)[:, None] + torch.arange(PAGE, device=DEV)).reshape(-1)[:n].int()
            s["positions"] = torch.arange(n, device=DEV, dtype=torch.int32)
            s["lens"] = torch.tensor([n], dtype=torch.int32, device=DEV)
            s["cu"] = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            s["rows"] = torch.empty(n, ROW, dtype=torch.bfloat16, device=DEV)
            s["pool"] = integers(0, 256, pages, PAGE, D_C // 2 + D_C // 16, dtype=torch.uint8)
        else:  # tokens of many sequences: slots anywhere in the pool, one in sixteen a padding row
            s["slots"] = torch.randperm(pages * PAGE, generator=gen, device=DEV)[:n].int()
            if n >= 16:
                s["slots"][::16] = -1
            if case["cache"] == "bf16":
                s["pool"] = normal(pages, PAGE, ROW)
            else:
                s["pool"] = integers(0, 0x7F, pages, PAGE, D_C, dtype=torch.uint8)  # finite e4m3 codes
        if case["cache"] != "bf16":
            s["scale"] = torch.rand(pages, PAGE, generator=gen, device=DEV)
            s["kr"] = normal(pages, PAGE, D_R)
        if case["query"]:
            s["q"] = normal(n, HEADS, D_HC + D_R)
            s["q_c"] = torch.empty(n, HEADS, D_HC, dtype=torch.bfloat16, device=DEV)
            s["q_r"] = torch.empty(n, HEADS, D_R, dtype=torch.bfloat16, device=DEV)
    else:
        R, H, N, K, G = case["rows"], case["heads"], case["n"], case["k"], case["group"]
        s["x"] = normal(R, H, K)
        s["codes"] = integers(0, 256, H, N, K // 2, dtype=torch.uint8)
        s["zero"], s["tensor_scale"] = None, 1.0
        if case["format"] == "int4":
            s["scale"] = ((torch.rand(H, N, K // G, generator=gen, device=DEV) + 0.5) / (4 * math.sqrt(K))).bfloat16()
            if case["zero"]:
                s["zero"] = integers(5, 12, H, N, K // G, dtype=torch.uint8)
        else:  # e4m3 scales in [1, 448], the tensor's own scale bringing the weights to about 1/sqrt(K)
            s["scale"] = integers(0x38, 0x7F, H, N, K // G, dtype=torch.uint8)
            s["tensor_scale"] = 1.0 / (256.0 * math.sqrt(K))
        s["out"] = torch.empty(R, H, N, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------------- one pass

def _rotate(x, positions, freq, mult, layout):
    """x [tokens, heads, dim] in 32 bits, every pair turned by position * frequency."""
    angle = positions.double()[:, None, None] * freq
    c, s = (angle.cos() * mult).float(), (angle.sin() * mult).float()
    if layout == "half":
        a, b = x.float().chunk(2, dim=-1)
        return torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)


def _plain_rope(s):
    case, x = s["case"], s["x"]
    o, d = case["offset"], case["dim"]
    y = _rotate(x[..., o:o + d], s["positions"], s["freq"], s["mult"], case["layout"]).to(x.dtype)
    if case["split"]:
        return {"out": y, "rest": torch.cat([x[..., :o], x[..., o + d:]], dim=-1)}
    return {"out": torch.cat([x[..., :o], y, x[..., o + d:]], dim=-1)}


def _e2m1(v):
    """The e2m1 code nearest to v, ties to the even code, magnitudes past 6 to 6."""
    a = v.abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return (code + 8 * torch.signbit(v)).to(torch.uint8)


def _e2m1_values(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=device)


def _plain_append(s):
    case = s["case"]
    keep = torch.nonzero(s["slots"] >= 0).flatten()
    slot = s["slots"][keep].long()
    c = s["c_kv"][keep].float()
    k = _rotate(s["k_r"][:, None, :], s["positions"], s["freq"], s["mult"], case["layout"])[keep, 0].bfloat16()
    out = {}
    if case["cache"] == "bf16":
        s["pool"].view(-1, ROW)[slot] = torch.cat([c.bfloat16(), k], dim=1)
        out["pool"] = s["pool"]
    else:
        top = c.abs().amax(dim=1)
        limit = 448.0 if case["cache"] == "fp8" else 2688.0
        sigma = torch.where(top > 0, top / limit, torch.ones_like(top))
        s["scale"].view(-1)[slot] = sigma
        s["kr"].view(-1, D_R)[slot] = k
        out["scale"], out["kr"] = s["scale"], s["kr"]
        if case["cache"] == "fp8":
            codes = (c / sigma[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s["pool"].view(-1, D_C)[slot] = codes
            out["pool"] = s["pool"].view(torch.float8_e4m3fn)
        else:
            blocks = c.view(-1, 32, 16)
            sb = (blocks.abs().amax(dim=2) / sigma[:, None] / 6.0).to(torch.float8_e4m3fn)
            den = sigma[:, None, None] * sb.float()[:, :, None]
            q = _e2m1(torch.where(den == 0, blocks * 0.0, blocks / den)).view(-1, D_C)
            s["pool"].view(-1, 288)[slot] = torch.cat([q[:, 0::2] | q[:, 1::2] << 4, sb.view(torch.uint8)], dim=1)
            # the prompt's rows, read back through the table in logical order
            at = (s["table"][0].long() * PAGE)[:, None] + torch.arange(PAGE, device=c.device)
            at = at.view(-1)[:case["tokens"]]
            stored = s["pool"].view(-1, 288)[at]
            both = torch.stack([stored[:, :256] & 15, stored[:, :256] >> 4], dim=-1).view(-1, 32, 16)
            value = _e2m1_values(c.device)[both.long()] * stored[:, 256:].view(torch.float8_e4m3fn).float()[:, :, None]
            latent = (value * s["scale"].view(-1)[at][:, None, None]).view(-1, D_C).bfloat16()
            out["rows"] = torch.cat([latent, s["kr"].view(-1, D_R)[at]], dim=1)
    if case["query"]:
        out["q_c"] = s["q"][..., :D_HC].clone()
        out["q_r"] = _rotate(s["q"][..., D_HC:], s["positions"], s["freq"], s["mult"], case["layout"]).bfloat16()
    return out


def _plain_w4(s):
    case = s["case"]
    H, N, K, G = case["heads"], case["n"], case["k"], case["group"]
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=-1).view(H, N, K // G, G)
    if case["format"] == "int4":
        zero = 8.0 if s["zero"] is None else s["zero"].float()[..., None]
        w = (codes.float() - zero) * s["scale"].float()[..., None]
    else:
        w = _e2m1_values(codes.device)[codes.long()] * s["scale"].view(torch.float8_e4m3fn).float()[..., None]
    y = torch.matmul(s["x"].float().transpose(0, 1), w.view(H, N, K).transpose(1, 2)) * s["tensor_scale"]
    return {"out": y.transpose(0, 1).bfloat16()}


def _rope_of(s, binding):
    """The rotation's constants, made once and kept by the program."""
    if "rope" not in s:
        case = s["case"]
        s["rope"] = binding.Rope(case.get("dim", D_R), base=case["base"], layout=case["layout"],
                                 scaling=case["scaling"], factor=case["factor"], original_len=case["original_len"])
    return s["rope"]


def _own(s):
    from mla_latent_kv_absorb_gb300 import binding

    case = s["case"]
    if case["op"] == "rope":
        binding.mla_rope(_rope_of(s, binding), s["x"], s["positions"], s["out"], rest=s["rest"],
                         rot_offset=case["offset"])
        return {"out": s["out"], "rest": s["rest"]} if case["split"] else {"out": s["out"]}
    if case["op"] == "append":
        quant = {} if case["cache"] == "bf16" else {"kv_scale": s["scale"], "kr_pool": s["kr"]}
        query = {"q": s["q"], "q_c": s["q_c"], "q_r": s["q_r"]} if case["query"] else {}
        binding.mla_rope_append_kv(_rope_of(s, binding), s["c_kv"], s["k_r"], s["positions"], s["slots"],
                                   kv_pool=s["pool"], dev_error=s["dev_error"], **quant, **query)
        out = {}
        if case["cache"] == "bf16":
            out["pool"] = s["pool"]
        else:
            out["scale"], out["kr"] = s["scale"], s["kr"]
            if case["cache"] == "fp8":
                out["pool"] = s["pool"].view(torch.float8_e4m3fn)
            else:
                binding.mla_gather_kv(kv_pool=s["pool"], block_table=s["table"], seq_lens=s["lens"],
                                      cu_seqlens=s["cu"], out=s["rows"], dev_error=s["dev_error"], **quant)
                out["rows"] = s["rows"]
        if case["query"]:
            out["q_c"], out["q_r"] = s["q_c"], s["q_r"]
        return out
    if "weight" not in s:
        s["weight"] = binding.W4Weight(s["codes"], s["scale"], zero=s["zero"], group=case["group"],
                                       tensor_scale=s["tensor_scale"])
    binding.mla_linear_w4(s["x"], s["weight"], s["out"])
    return {"out": s["out"]}


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "w4": _plain_w4}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------------- the work

def work(case):
    if case["op"] == "rope":
        T, H, D = case["tokens"], case["heads"], case["head_dim"]
        return {"bytes": 2 * T * H * D * (4 if case["dtype"] == "fp32" else 2) + 4 * T, "flops": 6 * T * H * case["dim"] // 2}
    if case["op"] == "append":
        n = case["tokens"]
        written = n - (n + 15) // 16 if case["cache"] != "nvfp4" and n >= 16 else n
        row = {"bf16": 1152, "fp8": 512 + 4 + 128, "nvfp4": 288 + 4 + 128}[case["cache"]]
        moved = written * (1152 + row) + 8 * n
        if case["cache"] == "nvfp4":
            moved += n * (row + 1152)  # read back as bf16 rows
        if case["query"]:
            moved += 2 * n * HEADS * (D_HC + D_R) * 2
        return {"bytes": moved, "flops": 3 * n * D_R * (1 + HEADS * case["query"])}
    R, H, N, K, G = case["rows"], case["heads"], case["n"], case["k"], case["group"]
    per_group = 1 if case["format"] == "nvfp4" else 3 if case["zero"] else 2
    return {"bytes": H * N * (K // 2 + K // G * per_group) + 2 * R * H * (K + N), "flops": 2 * R * H * N * K}


# ---------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)

    def turned(x, layout):
        """exp(i angle) times the pairs as complex numbers."""
        x = x.double()
        d = x.shape[-1]
        z = torch.complex(x[..., :d // 2], x[..., d // 2:]) if layout == "half" else \
            torch.view_as_complex(x.unflatten(-1, (d // 2, 2)).contiguous())
        angle = torch.outer(s["positions"].double(), s["freq"]).unsqueeze(1)
        z = z * torch.polar(torch.full_like(angle, s["mult"]), angle)
        return torch.cat([z.real, z.imag], dim=-1) if layout == "half" else torch.view_as_real(z).flatten(-2)

    if case["op"] == "rope":
        o, d = case["offset"], case["dim"]
        x = s["x"].double()
        y = turned(x[..., o:o + d], case["layout"])
        left, right = x[..., :o], x[..., o + d:]
        if case["split"]:
            return {"out": y, "rest": torch.cat([left, right], dim=-1)}
        return {"out": torch.cat([left, y, right], dim=-1)}
    if case["op"] == "append":
        live = s["slots"] >= 0
        slot = s["slots"][live].long()
        c = s["c_kv"][live].double()
        k = turned(s["k_r"].unsqueeze(1), case["layout"]).squeeze(1)[live]
        out = {}
        if case["cache"] == "bf16":
            pool = s["pool"].double().flatten(0, 1)
            pool[slot] = torch.cat([c, k], dim=1)
            out["pool"] = pool.unflatten(0, (-1, PAGE))
        else:
            sigma = (c.abs().amax(dim=1) / (448.0 if case["cache"] == "fp8" else 2688.0)).float().double()
            sigma = torch.where(sigma > 0, sigma, torch.ones_like(sigma))  # the cache holds it in 32 bits
            scale, kr = s["scale"].double().flatten(), s["kr"].double().flatten(0, 1)
            scale[slot], kr[slot] = sigma, k
            out["scale"], out["kr"] = scale.unflatten(0, (-1, PAGE)), kr.unflatten(0, (-1, PAGE))
            if case["cache"] == "fp8":
                pool = s["pool"].view(torch.float8_e4m3fn).double().flatten(0, 1)
                pool[slot] = (c / sigma[:, None]).to(torch.float8_e4m3fn).double()
                out["pool"] = pool.unflatten(0, (-1, PAGE))
            else:  # the format fixes each rounding to 4 bits in 32-bit steps: at its borders 64 bits decide otherwise
                out["rows"] = None
        if case["query"]:
            out["q_c"] = s["q"][..., :D_HC].double()
            out["q_r"] = turned(s["q"][..., D_HC:], case["layout"])
        return out
    H, N, K, G = case["heads"], case["n"], case["k"], case["group"]
    low, high = torch.remainder(s["codes"], 16), torch.div(s["codes"], 16, rounding_mode="floor")
    code = torch.empty(H, N, K, dtype=torch.uint8, device=DEV)
    code[..., 0::2], code[..., 1::2] = low, high
    scale = s["scale"].double() if case["format"] == "int4" else s["scale"].view(torch.float8_e4m3fn).double()
    out = torch.empty(case["rows"], H, N, dtype=torch.float64, device=DEV)
    for n0 in range(0, N, 2048):  # a slab of the outputs at a time
        part = code[:, n0:n0 + 2048].double()
        if case["format"] == "int4":
            zero = 8.0 if s["zero"] is None else s["zero"][:, n0:n0 + 2048].double().repeat_interleave(G, dim=2)
            value = part - zero
        else:  # sign, two exponent bits, one mantissa bit
            mag = torch.remainder(part, 8)
            e, m = torch.div(mag, 2, rounding_mode="floor"), torch.remainder(mag, 2)
            value = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2) * torch.where(part >= 8, -1.0, 1.0)
        value = value * scale[:, n0:n0 + 2048].repeat_interleave(G, dim=2)
        out[:, :, n0:n0 + 2048] = torch.einsum("rhk,hnk->rhn", s["x"].double(), value) * s["tensor_scale"]
    return {"out": out}
