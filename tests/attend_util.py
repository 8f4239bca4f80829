"""Attention in 64 bits for the tests of shared prefixes and windows, with the error that a kernel may make.

Bounds, derived from the kernels' roundings (u = 2^-8 is half a step of bf16 relative to the value):
scores are fp32 sums of exact products of bf16 values, n of them: off by at most e = n 2^-23 sum |q_d k_d|
* scale (truncating sums), so each weight by a factor within exp(+-e), and the weights' sum too; P is
rounded to bf16 (u) before it multiplies v, the sum over keys in fp32 adds n_keys 2^-23; 2^x is within
2^-21.  With a = sum_j w_j |v_j| that is at most (u + 2 e + 2^-20 + n_keys 2^-23) a, and the output's own
rounding adds u |out|.  Log-sum-exps are not rounded to bf16: e + 2^-20 (1 + |lse|) + n_keys 2^-23."""
import math

import torch

SCALE = 1.0 / math.sqrt(192.0)
U = 2.0 ** -8


def attend64(q_c, q_r, k, v, k_r, *, scale=SCALE, seen=None):
    """q_c [T, H, 128], q_r [T, H, 64], k and v [H, n, 128], k_r [n, 64], seen [T, n] (None: all): out [T, H, 128],
    lse [T, H], sum_j w_j |v_j| and the scores' bound e [T, H]; rows that see nothing get 0 and -inf."""
    q_c, q_r, k, v, k_r = (x.double() for x in (q_c, q_r, k, v, k_r))
    T, H = q_c.shape[:2]
    out, size = (torch.zeros(T, H, 128, dtype=torch.float64, device=k.device) for _ in range(2))
    lse, e = (torch.zeros(T, H, dtype=torch.float64, device=k.device) for _ in range(2))
    for h in range(H):
        x = (q_c[:, h] @ k[h].T + q_r[:, h] @ k_r.T) * scale
        mag = (q_c[:, h].abs() @ k[h].abs().T + q_r[:, h].abs() @ k_r.abs().T) * scale
        if seen is not None:
            x = x.masked_fill(~seen, -math.inf)
            mag = mag.masked_fill(~seen, 0.0)
        lse[:, h] = torch.logsumexp(x, dim=1)
        w = torch.exp(x - torch.where(lse[:, h].isinf(), 0.0, lse[:, h])[:, None])
        vh = v[h]
        if seen is not None:  # keys that no row sees may hold anything
            vh = torch.where(seen.any(dim=0)[:, None], vh, 0.0)
            w = torch.where(seen, w, 0.0)
        out[:, h], size[:, h] = w @ vh, w @ vh.abs()
        e[:, h] = 192 * 2.0 ** -23 * mag.amax(dim=1)
    return out, lse, size, e


def merge64(parts):
    """Parts (out, lse, size, e) of one softmax joined."""
    lse = torch.logsumexp(torch.stack([p[1] for p in parts]), dim=0)
    w = [torch.exp(p[1] - lse)[..., None] for p in parts]
    zero = lambda p, x: torch.where(p[1].isinf()[..., None], 0.0, x)  # noqa: E731  a part without keys may hold anything
    out = sum(wi * zero(p, p[0]) for wi, p in zip(w, parts))
    size = sum(wi * zero(p, p[2]) for wi, p in zip(w, parts))
    return out, lse, size, torch.stack([p[3] for p in parts]).amax(dim=0)


def check(got, ref, *, keys, extra=0.0, absolute=0.0, what=""):
    """Every output within the bound; extra: further relative error of the weights and values, absolute: of the values."""
    out, lse, size, e = ref
    tol = (U + 2 * e[..., None] + 2.0 ** -20 + keys * 2.0 ** -23 + extra) * size + U * out.abs() + absolute + 1e-30
    err = (got.double() - out).abs()
    worst = float((err / tol).max())
    assert torch.isfinite(got.float()).all(), f"{what}: non-finite values"
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound at {int((err / tol).argmax())}"
    return worst


def check_lse(got, ref, *, keys, extra=0.0, what=""):
    _, lse, _, e = ref
    tol = e + 2.0 ** -20 * (1 + lse.abs()) + keys * 2.0 ** -23 + extra
    worst = float(((got.double() - lse).abs() / tol).max())
    assert worst <= 1.0, f"{what}: log-sum-exp {worst:.2f} times the bound"
    return worst


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def cache_values(kv, slots):
    """The latents [n, 512] and rotary keys [n, 64] that the cache rows `slots` stand for, in 64 bits."""
    pool = kv["kv_pool"].flatten(0, 1)[slots]
    if "kv_scale" not in kv:
        return pool[:, :512].double(), pool[:, 512:].double()
    sigma = kv["kv_scale"].flatten()[slots].double()[:, None]
    if pool.shape[1] == 512:
        c = pool.view(torch.float8_e4m3fn).double() * sigma
    else:
        codes = torch.stack([pool[:, :256] & 15, pool[:, :256] >> 4], dim=-1).flatten(-2)
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=pool.device)
        c = torch.where(codes >= 8, -1.0, 1.0) * grid[(codes & 7).long()] * sigma
        c = c * pool[:, 256:].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1)
    return c, kv["kr_pool"].flatten(0, 1)[slots].double()


def make_cache(gen, pages, kind):
    """A cache of `pages` pages of latents of about unit size: kv_pool, and kv_scale and kr_pool where quantised."""
    if kind == "bf16":
        return {"kv_pool": normal(gen, pages, 64, 576)}
    kr = normal(gen, pages, 64, 64)
    if kind == "fp8":
        c = torch.randn(pages, 64, 512, generator=gen, device="cuda")
        sigma = c.abs().amax(dim=-1) / 448.0
        return {"kv_pool": (c / sigma[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), "kv_scale": sigma, "kr_pool": kr}
    codes = torch.randint(0, 256, (pages, 64, 256), generator=gen, device="cuda", dtype=torch.uint8)
    blocks = torch.randint(0x58, 0x7F, (pages, 64, 32), generator=gen, device="cuda", dtype=torch.uint8)
    sigma = (torch.rand(pages, 64, generator=gen, device="cuda") + 0.5) / 480.0
    return {"kv_pool": torch.cat([codes, blocks], dim=-1), "kv_scale": sigma, "kr_pool": kr}


def bf16_step(x):
    """The distance between bf16 values around x (64 bits)."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -126))) - 7)
