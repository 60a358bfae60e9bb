"""Timing cases of the 4-bit key/value cache: append, read, decode attention, block-sparse decode, eviction.

The cache holds K and V as E2M1 codes (two to a byte, the even element in the low nibble) with one E4M3
scale per 16 elements and one fp32 scale per tensor, head-major: codes [B, H_kv, L_max, d_h / 2], scales
[B, H_kv, L_max, d_h / 16]. ``run`` computes the operators with elementary torch operations in fp32 where
``own`` is false, and with the framework's calls where it is true; ``exact`` gives fp64 values.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one short chat turn: a launch-latency step, odd length inside the first pages of a cache
        dict(name="decode_one_short", op="decode", B=1, H_q=64, H_kv=4, d=128, L_max=512, lo=301, hi=301, weights=False),
        # a mid-size batch of small heads; one slot of the batch is padding (no tokens)
        dict(name="decode_batch_d64", op="decode", B=24, H_q=32, H_kv=8, d=64, L_max=9088, lo=0, hi=9001, weights=False),
        # one long document: few (sequence, head) pairs, so the keys have to be split over the GPU
        dict(name="decode_one_128k", op="decode", B=1, H_q=64, H_kv=4, d=128, L_max=131072, lo=131071, hi=131071,
             weights=False),
        # a loaded server: sequences uniform in [16K, 128K]
        dict(name="decode_batch_long", op="decode", B=32, H_q=64, H_kv=4, d=128, L_max=131072, lo=16384, hi=131072,
             weights=False),
        # the same step with the weights kept for a later eviction
        dict(name="decode_weights", op="decode", B=16, H_q=64, H_kv=4, d=128, L_max=16384, lo=1000, hi=16300, weights=True),
        # block-sparse decode of one sequence, weights kept
        dict(name="sparse_one", op="sparse", B=1, H_q=64, H_kv=4, d=128, d_idx=64, k=16, L_max=8192, lo=5003, hi=5003,
             weights=True),
        # block-sparse decode of the benchmark's batch: 64 sequences in [16K, 128K]
        dict(name="sparse_batch", op="sparse", B=64, H_q=64, H_kv=4, d=128, d_idx=64, k=16, L_max=131072, lo=16384,
             hi=131072, weights=False),
        # every sequence of a decode batch writes its new token (and it is read back)
        dict(name="append_step", op="append", B=64, H_q=64, H_kv=4, d=128, L_max=4096, lo=1, hi=1, at=3000),
        # chunks of four prompts, continuing cached prefixes, read back for the next chunk's attention
        dict(name="append_prompts", op="append", B=4, H_q=64, H_kv=4, d=128, L_max=32768, lo=4099, hi=11001, at=20000),
        # a short budget kept by two sequences
        dict(name="evict_small", op="evict", B=2, H_q=64, H_kv=4, d=128, d_idx=64, L_max=2048, lo=1400, hi=1601, keep=1000,
             recent=129, first=4),
        # a batch of prompts compressed after prefill
        dict(name="evict_prompts", op="evict", B=16, H_q=64, H_kv=4, d=128, d_idx=64, L_max=32768, lo=20001, hi=32768,
             keep=4096, recent=256, first=4),
        # one long document cut to an eighth
        dict(name="evict_one_long", op="evict", B=1, H_q=64, H_kv=4, d=128, d_idx=64, L_max=131072, lo=131000, hi=131000,
             keep=16384, recent=1000, first=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "sparse", "append", "evict"])
    d = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 4]) if op == "sparse" else rng.choice([1, 2, 4, 4, 8])
    H_q = H_kv * rng.choice([1, 4, 8, 16, 16])
    B = _log(rng, 1, 64)
    hi = _log(rng, 40, min(131072, 8_000_000 // (B * H_kv)))
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    case = dict(op=op, B=B, H_q=H_q, H_kv=H_kv, d=d, L_max=-(-hi // 128) * 128, lo=lo, hi=hi)
    if op == "decode":
        case["weights"] = rng.random() < 0.4
        if rng.random() < 0.2:
            case["lo"] = 0
    elif op == "sparse":
        case.update(d_idx=rng.choice([32, 64]), k=rng.choice([2, 4, 8, 16, 16]), weights=rng.random() < 0.5)
    elif op == "append":
        hi = max(1, hi // 8) if rng.random() < 0.6 else 1
        lo = max(1, hi // 3)
        at = rng.randrange(0, 5000)
        case.update(lo=lo, hi=hi, at=at, L_max=-(-(hi + at) // 128) * 128)
    else:
        recent = rng.randrange(0, max(1, lo // 4))
        first = rng.choice([0, 1, 4])
        keep = min(hi, max(recent + first + 1, _log(rng, 1, hi)))
        case.update(d_idx=rng.choice([32, 64, 128]), recent=recent, first=first, keep=keep)
    return case


# ------------------------------------------------------------------------------------------ inputs
def _lengths(case):
    """B lengths spread evenly over [lo, hi] (the same ones whatever the seed, so that the work is)."""
    B = case["B"]
    if B == 1:
        return [case["hi"]]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // (B - 1) for i in range(B)]


def _quantise(x, t):
    """Codes [..., d / 2] and scales [..., d / 16] (both uint8) of x [..., d]."""
    y = x.float() / torch.full((), t, dtype=torch.float32, device=x.device)
    g = y.unflatten(-1, (-1, 16))
    amax = g.abs().amax(-1, keepdim=True)
    six = torch.full((), 6.0, device=x.device)
    s8 = (amax / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    a = (g / torch.where(s > 0, s, torch.ones_like(s))).abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = torch.where(s > 0, c + 8 * (g < 0).to(torch.uint8), torch.zeros_like(c)).flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], s8.squeeze(-1).view(torch.uint8)


def _values(codes, scales, t):
    """fp32 values [..., d] of codes and scales."""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    lut = torch.cat([mag, -mag])
    both = torch.arange(256, device=codes.device)
    pairs = torch.stack([lut[both & 15], lut[both >> 4]], -1)
    x = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    x *= scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    x *= t
    return x.flatten(-2)


def _cache(case, gen, L_max, t_k, t_v, fill):
    """A cache whose first `fill` rows of every sequence hold quantised N(0, 1) rows (K with a few strong channels)."""
    B, H, d = case["B"], case["H_kv"], case["d"]
    c = {"k_scale": t_k, "v_scale": t_v, "B": B, "H_kv": H, "d": d, "L_max": L_max}
    for n, t in (("k", t_k), ("v", t_v)):
        codes = torch.zeros((B, H, L_max, d // 2), dtype=torch.uint8, device=DEVICE)
        scales = torch.zeros((B, H, L_max, d // 16), dtype=torch.uint8, device=DEVICE)
        for b in range(B if fill else 0):
            x = torch.randn((H, fill, d), device=DEVICE, generator=gen)
            if n == "k":
                x[..., ::23] *= 2.5
            codes[b, :, :fill], scales[b, :, :fill] = _quantise(x.bfloat16(), t)
        c[n + "_codes"], c[n + "_scales"] = codes, scales
    return c


def _handle(c):
    """The framework's cache handle over the tensors of `c`."""
    import block_sparse_long_idx_b200 as msa

    return msa.KV4Cache(c["k_codes"], c["k_scales"], c["v_codes"], c["v_scales"], k_scale=c["k_scale"], v_scale=c["v_scale"])


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed * 7919 + 17)
    B, H_q, H_kv, d, L_max = (case[n] for n in ("B", "H_q", "H_kv", "d", "L_max"))
    lens = _lengths(case)
    s = {"case": case}
    perm = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
    lens = [lens[p] for p in perm]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEVICE)

    if case["op"] in ("decode", "sparse"):
        s["cache"] = _cache(case, gen, L_max, 1.0, 0.75, max(lens))
        s["lens"] = i32(lens)
        s["q"] = torch.randn((B, H_q, d), device=DEVICE, generator=gen).bfloat16()
        if case["weights"]:
            s["w"] = torch.rand((B, H_kv, L_max), device=DEVICE, generator=gen)
            s["w_out"] = torch.zeros_like(s["w"])
            s["decay"] = 0.96875
    if case["op"] == "sparse":
        s["q_idx"] = torch.randint(-3, 4, (B, H_kv, case["d_idx"]), device=DEVICE, generator=gen).bfloat16()
        s["k_idx"] = torch.empty((B, L_max, H_kv, case["d_idx"]), device=DEVICE, dtype=torch.bfloat16)
        for b in range(B):
            s["k_idx"][b] = torch.randint(-3, 4, (L_max, H_kv, case["d_idx"]), device=DEVICE, generator=gen).bfloat16()
    if case["op"] == "append":
        T = sum(lens)
        s["cache"] = _cache(case, gen, L_max, 1.0, 0.75, 0)
        s["starts"] = i32([max(0, case["at"] - 37 * b) for b in range(B)])
        s["cu"] = i32(np.cumsum([0] + lens).tolist())
        s["T"] = T
        qkv = torch.randn((T, H_q + 2 * H_kv, d), device=DEVICE, generator=gen).bfloat16()  # the fused projection's output
        s["k"], s["v"] = qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
    if case["op"] == "evict":
        keep = case["keep"]
        s["cache"] = _cache(case, gen, L_max, 1.0, 0.75, max(lens))
        s["to"] = _cache(case, gen, -(-keep // 128) * 128, 1.0, 0.75, 0)
        s["lens"] = i32(lens)
        # accumulated weights: a heavy tail, with equal values among them
        w = torch.randn((B, H_kv, L_max), device=DEVICE, generator=gen).mul_(2).exp_()
        s["w"] = (w * 64).round() / 64
        s["k_idx"] = torch.randint(-3, 4, (B, L_max, H_kv, case["d_idx"]), device=DEVICE, generator=gen).bfloat16()
        left = [min(n, keep) for n in lens]
        s["left_cu"] = i32(np.cumsum([0] + left).tolist())
        s["T"] = sum(left)
        s["zero"] = i32([0] * B)
    if case["op"] in ("append", "evict"):
        # which cache row each packed row is: (sequence, position)
        n = lens if case["op"] == "append" else [min(x, case["keep"]) for x in lens]
        st = s["starts"] if case["op"] == "append" else s["zero"]
        s["row_b"] = torch.repeat_interleave(torch.arange(B, device=DEVICE), torch.tensor(n, device=DEVICE))
        first = torch.tensor(np.cumsum([0] + n)[:-1], device=DEVICE)
        s["row_j"] = torch.arange(sum(n), device=DEVICE) - first[s["row_b"]] + st.long()[s["row_b"]]
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _attend(q, K, V, seen):
    """out, lse, p of q [B, H_q, d] over K, V [B, H_kv, n, d] where seen [B, H_kv, n]; rows that see nothing are 0, -inf."""
    B, H_q, d = q.shape
    H_kv = K.shape[1]
    x = torch.matmul(q.float().view(B, H_kv, H_q // H_kv, d), K.transpose(-1, -2)) / math.sqrt(d)
    x = x.masked_fill(~seen.unsqueeze(2), -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - torch.where(m.isinf(), torch.zeros_like(m), m)).exp()
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.matmul(p, V)
    lse = (total.log() + m).squeeze(-1)
    return out.reshape(B, H_q, d).bfloat16(), lse.reshape(B, H_q), p


def _plain_decode(s):
    c = s["cache"]
    seen = torch.arange(c["L_max"], device=DEVICE) < s["lens"].view(-1, 1, 1)
    seen = seen.expand(-1, c["H_kv"], -1)
    K = _values(c["k_codes"], c["k_scales"], c["k_scale"])
    V = _values(c["v_codes"], c["v_scales"], c["v_scale"])
    out, lse, p = _attend(s["q"], K, V, seen)
    r = {"out": out, "lse": lse}
    if "w" in s:
        r["w_out"] = torch.where(seen, s["decay"] * s["w"] + p.sum(2), s["w_out"])
    return r


def _plain_sparse(s):
    c, case = s["cache"], s["case"]
    B, H, L, k = c["B"], c["H_kv"], c["L_max"], case["k"]
    nb = L // 128
    last = (s["lens"].long() - 1) // 128
    x = torch.einsum("bld,bd->bl", s["k_idx"].transpose(1, 2).reshape(B * H, L, -1).float(),
                     s["q_idx"].reshape(B * H, -1).float()).view(B, H, nb, 128).amax(-1)
    at = torch.arange(nb, device=DEVICE)
    local = last.view(B, 1, 1)
    x = x.masked_fill(at == local, math.inf).masked_fill(at > local, -math.inf)
    order = x.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    sel = torch.where(order <= local, order, nb).sort(-1).values
    if k > nb:
        sel = torch.cat([sel, sel.new_full((B, H, k - nb), nb)], -1)
    chosen = torch.where(sel < nb, sel, -1)
    pos = (chosen.clamp(min=0).unsqueeze(-1) * 128 + torch.arange(128, device=DEVICE)).flatten(-2)
    seen = (pos < s["lens"].view(-1, 1, 1)) & (chosen >= 0).repeat_interleave(128, -1)

    def rows(n):
        t = c[n]
        return t.gather(2, pos.unsqueeze(-1).expand(-1, -1, -1, t.shape[-1]))

    K = _values(rows("k_codes"), rows("k_scales"), c["k_scale"])
    V = _values(rows("v_codes"), rows("v_scales"), c["v_scale"])
    out, lse, p = _attend(s["q"], K, V, seen)
    r = {"out": out, "lse": lse, "block_idx": chosen.int()}
    if "w" in s:
        visible = torch.arange(L, device=DEVICE) < s["lens"].view(-1, 1, 1)
        add = torch.zeros_like(s["w"]).scatter_add_(2, pos, torch.where(seen, p.sum(2), torch.zeros_like(p[:, :, 0])))
        r["w_out"] = torch.where(visible, s["decay"] * s["w"] + add, s["w_out"])
    return r


def _plain_read(c, b, j):
    k = _values(c["k_codes"][b, :, j], c["k_scales"][b, :, j], c["k_scale"])
    v = _values(c["v_codes"][b, :, j], c["v_scales"][b, :, j], c["v_scale"])
    return k.bfloat16(), v.bfloat16()


def _plain_append(s):
    c, b, j = s["cache"], s["row_b"], s["row_j"]
    c["k_codes"][b, :, j], c["k_scales"][b, :, j] = _quantise(s["k"], c["k_scale"])
    c["v_codes"][b, :, j], c["v_scales"][b, :, j] = _quantise(s["v"], c["v_scale"])
    k, v = _plain_read(c, b, j)
    return {"k": k, "v": v}


def _plain_evict(s):
    c, to, case = s["cache"], s["to"], s["case"]
    keep, recent, first = case["keep"], case["recent"], case["first"]
    n = s["lens"].long().view(-1, 1, 1)
    at = torch.arange(c["L_max"], device=DEVICE)
    always = (at < first) | (at >= n - recent)
    w = torch.where(always, torch.full_like(s["w"], math.inf), s["w"]).masked_fill(at >= n, -math.inf)
    left = n.clamp(max=keep)
    order = w.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    taken = torch.arange(keep, device=DEVICE) < left
    kept = torch.where(taken, order, c["L_max"]).sort(-1).values
    src = torch.where(taken, kept, 0)

    def moved(x, old):
        row = x.gather(2, src.unsqueeze(-1).expand(-1, -1, -1, x.shape[-1]))
        old[:, :, :keep] = torch.where(taken.unsqueeze(-1), row, old[:, :, :keep])

    moved(c["k_codes"], to["k_codes"])
    moved(c["k_scales"], to["k_scales"])
    moved(c["v_codes"], to["v_codes"])
    moved(c["v_scales"], to["v_scales"])
    k_idx = torch.zeros((c["B"], to["L_max"], c["H_kv"], case["d_idx"]), dtype=torch.bfloat16, device=DEVICE)
    moved(s["k_idx"].transpose(1, 2), k_idx.transpose(1, 2))
    w_to = torch.zeros((c["B"], c["H_kv"], to["L_max"]), device=DEVICE)
    moved(s["w"].unsqueeze(-1), w_to.unsqueeze(-1))
    k, v = _plain_read(to, s["row_b"], s["row_j"])
    return {"lens": left.view(-1).int(), "kept": torch.where(taken, kept, -1).int(), "k_idx": k_idx, "w": w_to, "k": k, "v": v}


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"decode": _plain_decode, "sparse": _plain_sparse, "append": _plain_append, "evict": _plain_evict}[op](s)
    import block_sparse_long_idx_b200 as msa

    if "handle" not in s:
        s["handle"] = _handle(s["cache"])
        if "to" in s:
            s["to_handle"] = _handle(s["to"])
    kv = s["handle"]
    more = dict(weights=s["w"], weights_out=s["w_out"], decay=s["decay"]) if "w_out" in s else {}
    if op == "decode":
        out, lse = msa.msa_kv4_decode(s["q"], kv, s["lens"], **more)
        r = {"out": out, "lse": lse}
    elif op == "sparse":
        out, lse, sel = msa.msa_sparse_decode_kv4(s["q"], s["q_idx"], kv, s["k_idx"], s["lens"], k=s["case"]["k"], **more)
        r = {"out": out, "lse": lse, "block_idx": sel}
    elif op == "append":
        msa.msa_kv4_append(kv, s["k"], s["v"], s["starts"], s["cu"])
        k, v = msa.msa_kv4_read(kv, s["starts"], s["cu"], s["T"])
        return {"k": k, "v": v}
    else:
        case, to = s["case"], s["to_handle"]
        w_to = torch.zeros((case["B"], case["H_kv"], s["to"]["L_max"]), device=DEVICE)
        k_idx = torch.zeros((case["B"], s["to"]["L_max"], case["H_kv"], case["d_idx"]), dtype=torch.bfloat16, device=DEVICE)
        left, kept = msa.msa_kv4_evict(kv, to, s["w"], s["lens"], case["keep"], recent=case["recent"], first=case["first"],
                                       weights_dst=w_to, k_idx_cache=s["k_idx"], k_idx_dst=k_idx)
        k, v = msa.msa_kv4_read(to, s["zero"], s["left_cu"], s["T"])
        return {"lens": left, "kept": kept, "k_idx": k_idx, "w": w_to, "k": k, "v": v}
    if "w_out" in s:
        r["w_out"] = s["w_out"]
    return r


def work(case):
    B, H_q, H_kv, d = (case[n] for n in ("B", "H_q", "H_kv", "d"))
    lens = _lengths(case)
    row = 2 * (d // 2 + d // 16)  # bytes of one cached (token, head): K and V
    if case["op"] == "decode":
        n = sum(lens)
        return {"bytes": n * H_kv * (row + (8 if case["weights"] else 0)) + 4 * B * H_q * d + 4 * B * H_q,
                "flops": 4.0 * n * H_q * d}
    if case["op"] == "sparse":
        d_idx, k = case["d_idx"], case["k"]
        sel = sum(min(n, (k - 1) * 128 + (n - 1) % 128 + 1) for n in lens)
        idx = sum((n - 1) // 128 * 128 for n in lens)
        w = 8 * sum(lens) * H_kv if case["weights"] else 0
        return {"bytes": idx * H_kv * d_idx * 2 + sel * H_kv * row + 4 * B * H_q * d + 4 * B * H_q + 4 * B * H_kv * k + w,
                "flops": 2.0 * idx * H_kv * d_idx + 4.0 * sel * H_q * d}
    if case["op"] == "append":
        T = sum(lens)  # bf16 rows in, packed rows out; packed rows in, bf16 rows out
        return {"bytes": 2 * T * H_kv * (4 * d + row), "flops": 6.0 * T * H_kv * 2 * d}
    left = sum(min(n, case["keep"]) for n in lens)
    kept = left * H_kv * (2 * (row + 4 + 2 * case["d_idx"]) + 4)
    return {"bytes": 4 * sum(lens) * H_kv + kept + left * H_kv * (row + 4 * d), "flops": float(sum(lens) * H_kv)}


# ------------------------------------------------------------------------------------------ 64 bits
_MAGS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_table():
    """Value of every E4M3 byte from its fields (bias 7, subnormals, no infinities)."""
    v = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append((-x if c & 128 else x) if c & 127 != 127 else math.nan)
    return v


def _nearest(x, table):
    """Index of the entry of the ascending `table` nearest to each x >= 0; ties to the even index."""
    t = torch.tensor(table, dtype=torch.float64, device=x.device)
    up = torch.searchsorted(t, x.contiguous()).clamp(1, len(table) - 1)
    lo, hi = x - t[up - 1], t[up] - x
    return torch.where((lo < hi) | ((lo == hi) & (up % 2 == 1)), up - 1, up)


def _values64(codes, scales, t):
    lut = torch.tensor(_MAGS + [-m for m in _MAGS], dtype=torch.float64, device=codes.device)
    e4 = torch.tensor(_e4m3_table(), dtype=torch.float64, device=codes.device)
    c = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.float64, device=codes.device)
    c[..., 0::2] = lut[(codes % 16).long()]
    c[..., 1::2] = lut[(codes // 16).long()]
    return c * e4[scales.long()].repeat_interleave(16, -1) * float(np.float32(t))


def _stored64(x, t):
    """The values that x is held as, from the format's definition."""
    y = (x.double() / float(np.float32(t))).float().double().unflatten(-1, (-1, 16))
    steps = _e4m3_table()[:127]
    s = torch.tensor(steps, dtype=torch.float64, device=x.device)[_nearest((y.abs().amax(-1) / 6).float().double(), steps)].unsqueeze(-1)
    q = (y.abs() / torch.where(s > 0, s, 1.0)).float().double()
    m = torch.tensor(_MAGS, dtype=torch.float64, device=x.device)[_nearest(q, _MAGS)]
    return (torch.where(s > 0, m * s, 0.0) * y.sign() * float(np.float32(t))).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c, B, H = s["cache"], case["B"], case["H_kv"]
    if case["op"] == "append":
        return {"k": _stored64(s["k"], c["k_scale"]), "v": _stored64(s["v"], c["v_scale"])}
    lens = s["lens"].tolist()
    if case["op"] == "evict":
        keep, recent, first = case["keep"], case["recent"], case["first"]
        kept = np.full((B, H, keep), -1, dtype=np.int32)
        k_idx = torch.zeros((B, s["to"]["L_max"], H, case["d_idx"]), dtype=torch.float64, device=DEVICE)
        w_to = torch.zeros((B, H, s["to"]["L_max"]), dtype=torch.float64, device=DEVICE)
        ks, vs = [], []
        for b, n in enumerate(lens):
            m = min(n, keep)
            for h in range(H):
                j = np.arange(n)
                if n > keep:
                    mid = j[first:n - recent]
                    w = s["w"][b, h, first:n - recent].double().cpu().numpy()
                    mid = mid[np.lexsort((mid, -w))[:keep - first - recent]]
                    j = np.sort(np.concatenate([j[:first], mid, j[n - recent:]]))
                kept[b, h, :m] = j
                jt = torch.from_numpy(j).to(DEVICE)
                k_idx[b, :m, h] = s["k_idx"][b, jt, h].double()
                w_to[b, h, :m] = s["w"][b, h, jt].double()
                for n_, to in (("k", ks), ("v", vs)):
                    to.append(_values64(c[n_ + "_codes"][b, h, jt], c[n_ + "_scales"][b, h, jt], c[n_ + "_scale"]))
        out = {}
        for n_, to in (("k", ks), ("v", vs)):
            out[n_] = torch.cat([torch.stack(to[b * H:(b + 1) * H], 1) for b in range(B)])
        return {"lens": torch.tensor([min(n, keep) for n in lens], dtype=torch.int32), "kept": torch.from_numpy(kept), "k_idx": k_idx,
                "w": w_to, **out}
    H_q, d, G = case["H_q"], case["d"], case["H_q"] // H
    r = {"out": torch.zeros((B, H_q, d), dtype=torch.float64, device=DEVICE),
         "lse": torch.full((B, H_q), -math.inf, dtype=torch.float64, device=DEVICE)}
    if "w" in s:
        r["w_out"] = s["w_out"].double()
    if case["op"] == "sparse":
        k = case["k"]
        r["block_idx"] = torch.full((B, H, k), -1, dtype=torch.int32, device=DEVICE)
    for b, n in enumerate(lens):
        for h in range(H if n else 0):
            pos = torch.arange(n, device=DEVICE)
            if case["op"] == "sparse":
                local = (n - 1) // 128
                x = (s["k_idx"][b, :local * 128, h].double() @ s["q_idx"][b, h].double()).view(local, 128)
                x = x.amax(-1).cpu().numpy() if local else np.zeros(0)
                best = np.lexsort((np.arange(local), -x))[:k - 1]
                sel = np.sort(np.append(best, local))
                r["block_idx"][b, h, :len(sel)] = torch.from_numpy(sel.astype(np.int32)).to(DEVICE)
                pos = (torch.from_numpy(sel).to(DEVICE)[:, None] * 128 + torch.arange(128, device=DEVICE)).flatten()
                pos = pos[pos < n]
            K = _values64(c["k_codes"][b, h, pos], c["k_scales"][b, h, pos], c["k_scale"])
            V = _values64(c["v_codes"][b, h, pos], c["v_scales"][b, h, pos], c["v_scale"])
            x = s["q"][b, h * G:(h + 1) * G].double() @ K.T / math.sqrt(d)
            p = torch.softmax(x, -1)
            r["out"][b, h * G:(h + 1) * G] = p @ V
            r["lse"][b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            if "w" in s:
                r["w_out"][b, h, :n] = s["decay"] * s["w"][b, h, :n].double()
                r["w_out"][b, h, pos] += p.sum(0)
    return r
