"""The 4-bit key/value cache on the GPU against its float64 definition (tests/ref_kv4.py).

Codes, scales, read values, selections and moved rows are compared exactly. Tolerances of the attention,
from what is rounded (half steps: bf16 2^-8, fp16 2^-11, fp32 2^-24 of the value):
  logits  q is fp16 after an exact power of two (an error of 2^-25 of the row's largest |q| at most, for
          elements below 2^-14 of it, else none), products are exact, the sum of d <= 128 products and
          its scaling are fp32: |dx| <= (d + 2) 2^-24 S + 2^-25 S' with S the largest sum_d |q K| / sqrt(d)
          and S' = max|q| sum|K| / sqrt(d) <= d S''; taken together as e = 2^-16 S + 2^-25 S'.
  lse     e + 2^-22 |lse| (stored in fp32, from a base-2 logarithm) + 2^-20 (ex2 and the sums).
  weights p (2 e + 2^-19): exp of two logit errors, ex2's 2^-22, sums of up to 16 heads.
  out     p is rounded to fp16 (2^-11 of it at most, while it is a normal number) and sums are fp32, so before
          rounding the error is (2^-11 + 2 e + 2^-19) sum_j p_j |V_j|; then bf16: 2^-8 |out|. P is held against a
          reference set 7 powers of two below the row's maximum and raised, never lowered: the largest weight
          has P >= 2^7. A P below fp16's normal range is off by half a subnormal step, 2^-25, which is at most
          2^-25 / 2^7 = 2^-32 of the largest weight, itself at most 1: + 2^-32 sum_j |V_j|. It shows where the
          heavy keys' V is 0, so that keys of p = 1e-9 are all that an element holds."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import block_sparse_long_idx_b200 as msa  # noqa: E402
from tests import ref_kv4 as ref  # noqa: E402

DEVICE_CHECK = 6


def i32(x):
    return torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")


def make_cache(B, L_max, H, d, ts=(1.0, 0.75), fill=0xFF):
    """A cache whose rows hold `fill` (0xFF: NaN scales) until they are appended."""
    c = msa.KV4Cache.empty(B, L_max, H, d, ts[0], ts[1])
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(fill)
    return c


def fill_cache(B, L_max, H, d, lens, seed, ts=(1.0, 0.75), v_bump=None):
    """A cache with random rows for the first lens[b] positions, and their float64 values (K, V lists)."""
    g = torch.Generator("cuda").manual_seed(seed)
    c = make_cache(B, L_max, H, d, ts)
    T = int(sum(lens))
    k = torch.randn((T, H, d), device="cuda", generator=g)
    k[..., ::23] *= 3
    v = torch.randn((T, H, d), device="cuda", generator=g)
    if v_bump is not None:
        v_bump(v)
    cu = np.concatenate([[0], np.cumsum(lens)])
    msa.msa_kv4_append(c, k.bfloat16(), v.bfloat16(), i32(np.zeros(B)), i32(cu))
    return c


def host_values(c, b, r, n):
    K = ref.values(c.k_codes[b, r, :n].cpu().numpy(), c.k_scales[b, r, :n].cpu().numpy(), c.k_scale)
    V = ref.values(c.v_codes[b, r, :n].cpu().numpy(), c.v_scales[b, r, :n].cpu().numpy(), c.v_scale)
    return K, V


def check_decode(c, q, lens, out, lse, block_idx=None, w=None, w_out=None, w_before=None, decay=1.0, seqs=None):
    H, d = c.H_kv, c.d_h
    G = q.shape[1] // H
    qh, oh, lh = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in (range(c.B) if seqs is None else seqs):
        n = int(lens[b])
        for r in range(H):
            pos = np.arange(n)
            if block_idx is not None:
                bl = block_idx[b, r]
                pos = np.concatenate([np.arange(x * 128, min(n, x * 128 + 128)) for x in bl if x >= 0] + [np.arange(0)]).astype(int)
            K, V = host_values(c, b, r, n)
            K, V = K[pos], V[pos]
            hs = slice(r * G, (r + 1) * G)
            want, wl, p, pv, S = ref.attend(qh[b, hs], K, V)
            big = float((np.abs(qh[b, hs]).max(-1)[:, None] * np.abs(K).sum(-1)[None]).max() / np.sqrt(d)) if len(pos) else 0.0
            e = 2.0 ** -16 * S + 2.0 ** -25 * big
            tol = (2.0 ** -11 + 2 * e + 2.0 ** -19) * pv + 2.0 ** -8 * np.abs(want) + 2.0 ** -32 * np.abs(V).sum(0)
            assert np.isfinite(oh[b, hs]).all()
            bad = np.abs(oh[b, hs] - want) > tol + 1e-30
            assert not bad.any(), (b, r, n, np.argwhere(bad)[:3], np.abs(oh[b, hs] - want).max())
            if len(pos):
                assert (np.abs(lh[b, hs] - wl) <= e + 2.0 ** -22 * np.abs(wl) + 2.0 ** -20).all(), (b, r, lh[b, hs], wl)
            else:
                assert (lh[b, hs] == -np.inf).all() and (oh[b, hs] == 0).all()
            if w_out is not None:
                got = w_out[b, r].double().cpu().numpy()
                ww = decay * w[b, r, :n].double().cpu().numpy() if w is not None else np.zeros(n)
                add = np.zeros(n)
                add[pos] = p.sum(0)
                assert (np.abs(got[:n] - ww - add) <= 2.0 ** -22 * (ww + add) + (2 * e + 2.0 ** -19) * add).all(), (b, r)
                assert np.array_equal(got[n:], w_before[b, r, n:].double().cpu().numpy()), "behind the length"


# ------------------------------------------------------------------------------------------ append and read
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [1.0, 0.75, 0.037, 2.0 ** -40])
def test_append_codes_and_read_values(d, t):
    """Codes and scales are the definition's, rows that are not written keep their bytes; the rows read back
    are the values' bf16 roundings. Chunks of several lengths (none, one row, many) from a strided source."""
    B, H, L_max = 5, 3, 384
    lens, starts = [0, 1, 200, 0, 130], [7, 383, 11, 0, 250]
    T = sum(lens)
    rng = np.random.default_rng(d)
    x = rng.standard_normal((T, 2 * H + 2, d)) * t
    x[5] = 0
    x[6] *= 1e-4                                   # groups that round to a zero scale
    x[7] *= 5e4                                    # saturating groups
    x[8, :, ::16] = 0
    x[9] = np.sign(x[9]) * t * rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], size=x[9].shape)  # ties
    x[10, :, 1:] = -0.0
    big = torch.from_numpy(x).cuda().bfloat16()
    k, v = big[:, 1:1 + H], big[:, H + 1:2 * H + 1]
    c = make_cache(B, L_max, H, d, (t, 2 * t), fill=0xA5)
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    msa.msa_kv4_append(c, k, v, i32(starts), cu)
    for x_, codes, scales, tt in ((k, c.k_codes, c.k_scales, c.k_scale), (v, c.v_codes, c.v_scales, c.v_scale)):
        wc, ws = ref.quantise(x_.float().cpu().numpy(), tt)
        want_c, want_s = np.full(codes.shape, 0xA5, np.uint8), np.full(scales.shape, 0xA5, np.uint8)
        i = 0
        for b in range(B):
            for j in range(lens[b]):
                want_c[b, :, starts[b] + j], want_s[b, :, starts[b] + j] = wc[i], ws[i]
                i += 1
        assert np.array_equal(scales.cpu().numpy(), want_s)
        assert np.array_equal(codes.cpu().numpy(), want_c)
    kr, vr = msa.msa_kv4_read(c, i32(starts), cu, T)
    for got, x_, tt in ((kr, k, c.k_scale), (vr, v, c.v_scale)):
        val = ref.values(*ref.quantise(x_.float().cpu().numpy(), tt), tt)
        assert torch.equal(got, torch.from_numpy(val).float().cuda().bfloat16())


def test_append_one_row_each_and_bad_rows():
    """One row per sequence without tables; rows that the tables put outside are left out and reported."""
    B, H, d, L_max = 4, 2, 128, 256
    c = make_cache(B, L_max, H, d, fill=0)
    k = torch.randn((B, H, d), device="cuda").bfloat16()
    v = torch.randn((B, H, d), device="cuda").bfloat16()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    msa.msa_kv4_append(c, k, v, i32([0, 5, 255, 17]), workspace=ws)
    assert msa.msa_get_device_error(ws) == 0
    kr, _ = msa.msa_kv4_read(c, i32([0, 5, 255, 17]))
    assert torch.equal(kr.cpu(), torch.from_numpy(ref.values(*ref.quantise(k.float().cpu().numpy(), 1.0), 1.0)).bfloat16())
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    for starts, cu, T in (([256, -1, 300, 2 ** 31 - 1], None, B), ([255, 0, 0, 0], [0, 0, 0, 0, 0], 3), ([0] * 4, [2, 2, 2, 2, 2], 2)):
        msa.msa_kv4_append(c, k[:T], v[:T], i32(starts), None if cu is None else i32(cu), workspace=ws)
        assert msa.msa_get_device_error(ws) == DEVICE_CHECK
        for t, o in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before):
            assert torch.equal(t, o)
    # two rows from position 255 on: the first is written, the second is outside
    msa.msa_kv4_append(c, k[:2], v[:2], i32([255, 0, 0, 0]), i32([0, 2, 2, 2, 2]), workspace=ws)
    assert msa.msa_get_device_error(ws) == DEVICE_CHECK
    assert torch.equal(msa.msa_kv4_read(c, i32([255] * 4))[0][0].cpu(),
                       torch.from_numpy(ref.values(*ref.quantise(k[:1].float().cpu().numpy(), 1.0), 1.0))[0].bfloat16())
    msa.msa_kv4_append(c, k[:0], v[:0], i32([0] * 4), i32([0] * 5))  # nothing to write


# ------------------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
def test_decode_lengths(d, G):
    """Lengths of no key, one, around tiles and blocks, and long ones, in one ragged batch."""
    H = 2
    lens = [0, 1, 2, 31, 32, 33, 127, 128, 129, 500, 4095, 0, 2047]
    B, L_max = len(lens), 4096
    c = fill_cache(B, L_max, H, d, lens, seed=G)
    q = torch.randn((B, H * G, d), device="cuda").bfloat16()
    out, lse = msa.msa_kv4_decode(q, c, i32(lens))
    check_decode(c, q, lens, out, lse)


@pytest.mark.parametrize("shape", [(1, 4, 40001, 16), (700, 1, 90, 4), (3, 8, 6000, 5)], ids=["one_long", "many_short", "few"])
def test_decode_splits(shape):
    """One sequence split over every SM, more sequences than a CTA has threads, segments across CTAs."""
    B, H, n, G = shape
    rng = np.random.default_rng(B)
    lens = [n] if B == 1 else rng.integers(0, n + 1, size=B)
    c = fill_cache(B, (n + 127) // 128 * 128, H, 128, lens, seed=B)
    q = torch.randn((B, H * G, 128), device="cuda").bfloat16()
    out, lse = msa.msa_kv4_decode(q, c, i32(lens))
    check_decode(c, q, lens, out, lse)
    again, lse2 = msa.msa_kv4_decode(q, c, i32(lens))
    assert torch.equal(out, again) and torch.equal(lse, lse2), "not deterministic"


def test_decode_hard_values():
    """Logits far apart and far from 0, zero and tiny and huge q rows, a few enormous V rows among small ones."""
    B, H, G, d, n = 2, 1, 8, 128, 3000

    def bump(v):
        v[100] *= 2000.0
        v[2500:2600] *= 1e-2

    c = fill_cache(B, 3200, H, d, [n, n], seed=3, ts=(0.5, 1.0), v_bump=bump)
    q = torch.randn((B, H * G, d), device="cuda")
    for h, f in enumerate([0.0, 1e-30, 1e-4, 1.0, 20.0, 60.0, 3.0, 1.0]):
        q[:, h] *= f
    q[1, 7] = 0
    q[1, 7, 5] = 300.0   # one channel decides, the other elements are nothing
    q[0, 7, 3] = 1e4     # and elements 2^-14 and less below the largest
    q = q.bfloat16()
    out, lse = msa.msa_kv4_decode(q, c, i32([n, n]))
    check_decode(c, q, [n, n], out, lse)


@pytest.mark.parametrize("G", [3, 16])
@pytest.mark.parametrize("scale, zero", [(2.0 ** -40, "q"), (2.0 ** -100, "q"), (2.0 ** 10, "K")])
def test_decode_factor_range(scale, zero, G):
    """Zero q rows (a padded batch) on a cache of tiny values, and enormous q on zero keys: all logits are 0, the
    factor on them leaves fp32's range, and the last tile is masked. Every visible key weighs the same."""
    B, H, d, n = 1, 2, 128, 45
    c = make_cache(B, 128, H, d, (scale, 1.0))
    g = torch.Generator("cuda").manual_seed(23)
    k = torch.randn((n, H, d), device="cuda", generator=g) * (scale if zero == "q" else 0.0)
    v = torch.randn((n, H, d), device="cuda", generator=g)
    msa.msa_kv4_append(c, k.bfloat16(), v.bfloat16(), i32([0]), i32([0, n]))
    q = torch.full((B, H * G, d), 0.0 if zero == "q" else 2.0 ** 125, device="cuda").bfloat16()
    w_out = torch.zeros((B, H, 128), device="cuda")
    out, lse = msa.msa_kv4_decode(q, c, i32([n]), weights_out=w_out)
    check_decode(c, q, [n], out, lse, w_out=w_out, w_before=torch.zeros_like(w_out))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_light_keys(d):
    """One key outweighs the rest by 2^29 and its V is 0 in half of the elements: those hold what the others give."""
    B, H, G, n = 1, 1, 16, 700
    c = make_cache(B, 768, H, d)
    g = torch.Generator("cuda").manual_seed(17)
    k = torch.zeros((n, H, d), device="cuda")
    k[5, 0, 0] = 4.0
    v = torch.randn((n, H, d), device="cuda", generator=g)
    v[5, :, : d // 2] = 0.0
    msa.msa_kv4_append(c, k.bfloat16(), v.bfloat16(), i32([0]), i32([0, n]))
    q = torch.zeros((B, H * G, d), device="cuda")
    q[:, :, 0] = 20.1 / 4.0 * d ** 0.5 * torch.linspace(0.2, 1.1, G, device="cuda")
    q = q.bfloat16()
    out, lse = msa.msa_kv4_decode(q, c, i32([n]))
    check_decode(c, q, [n], out, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_blocks(d):
    """Given blocks: padding, none at all, the last part of a block; weights on them with an in-place decay."""
    B, H, G, k, L_max = 4, 2, 4, 5, 1024
    lens = [1000, 129, 640, 0]
    sel = np.full((B, H, k), -1, np.int32)
    sel[0, 0], sel[0, 1] = [0, 2, 3, 6, 7], [1, 7, -1, -1, -1]
    sel[1, 0, :2], sel[1, 1, :1] = [0, 1], [1]
    sel[2, 0, :1] = [4]                                  # sel[2, 1]: nothing
    c = fill_cache(B, L_max, H, d, lens, seed=5)
    q = torch.randn((B, H * G, d), device="cuda").bfloat16()
    w = torch.rand((B, H, L_max), device="cuda")
    ws = torch.empty(msa.lib.msa_kv4_decode_workspace_size(B, H * G), dtype=torch.uint8, device="cuda")
    for decay, same in ((1.0, True), (0.5, True), (1.0, False), (0.25, False)):
        w_in = w.clone()
        w_out = w_in if same else torch.full_like(w, 7.0)
        before = w_out.clone()
        out, lse = msa.msa_kv4_decode(q, c, i32(lens), torch.from_numpy(sel).cuda(), w_in, w_out, decay, workspace=ws)
        assert msa.msa_get_device_error(ws) == 0
        check_decode(c, q, lens, out, lse, sel, w, w_out, before, decay)


def test_decode_rejects_on_device():
    """Bad lengths and bad blocks are reported; other sequences are right and bad ones' outputs stay."""
    B, H, G, d, L_max = 4, 1, 4, 128, 512
    lens = [300, 513, -1, 512]
    c = fill_cache(B, L_max, H, d, [300, 512, 512, 512], seed=6)
    q = torch.randn((B, H * G, d), device="cuda").bfloat16()
    ws = torch.empty(msa.lib.msa_kv4_decode_workspace_size(B, H * G), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 3.0)
    lse = torch.full((B, H * G), 5.0, device="cuda")
    w = torch.full((B, H, L_max), 2.0, device="cuda")
    msa.msa_kv4_decode(q, c, i32(lens), weights=w, weights_out=w, out=out, lse=lse, workspace=ws)
    assert msa.msa_get_device_error(ws) == DEVICE_CHECK
    assert (out[1:3] == 3).all() and (lse[1:3] == 5).all() and (w[1:3] == 2).all()
    check_decode(c, q, lens, out, lse, seqs=[0, 3])
    for bad in ([0, 4], [-2, 1], [1, 1], [2, 0], [0, 2 ** 31 - 1]):  # outside, invalid, twice, descending
        sel = torch.tensor([[[0, 1]], [[0, 1]], [[0, 1]], [[0, 1]]], dtype=torch.int32, device="cuda")
        sel[3, 0] = torch.tensor(bad, dtype=torch.int32)
        o, ls = msa.msa_kv4_decode(q, c, i32([300, 512, 512, 512]), sel, workspace=ws)
        assert msa.msa_get_device_error(ws) == DEVICE_CHECK, bad
        check_decode(c, q, [300, 512, 512, 512], o, ls, sel.cpu().numpy(), seqs=[0, 1, 2])


@pytest.mark.parametrize("shape", [(128, 16, 4), (64, 4, 2), (128, 6, 8)], ids=["d128_G16", "d64_G4", "d128_G6"])
def test_decode_weights(shape):
    """Accumulated weights over a ragged batch: separate and same arrays, no earlier weights, no lse asked for."""
    d, G, H = shape
    lens = [0, 1, 33, 700, 2049, 128]
    B, L_max = len(lens), 2176
    c = fill_cache(B, L_max, H, d, lens, seed=G)
    q = torch.randn((B, H * G, d), device="cuda").bfloat16()
    w = torch.rand((B, H, L_max), device="cuda")
    for w_in, decay in ((w, 0.875), (None, 1.0)):
        w_out = torch.full_like(w, -3.0)
        before = w_out.clone()
        out, lse = msa.msa_kv4_decode(q, c, i32(lens), weights=w_in, weights_out=w_out, decay=decay)
        check_decode(c, q, lens, out, lse, None, w_in, w_out, before, decay)
    w2 = w.clone()
    out2, none = msa.msa_kv4_decode(q, c, i32(lens), weights=w2, weights_out=w2, decay=1.0, want_lse=False)
    assert none is None and torch.equal(out, out2)
    check_decode(c, q, lens, out, lse, None, w, w2, w, 1.0)


def test_decode_offsets_past_32_bits():
    """A cache of more than 2^32 bytes of codes: the last sequence's rows lie behind that offset."""
    B, H, d, L_max = 9, 8, 128, 2 ** 20
    c = msa.KV4Cache.empty(B, L_max, H, d)
    assert c.k_codes.numel() > 2 ** 32
    n, at = 3000, L_max - 3000
    lens = [0] * (B - 1) + [L_max]
    c.k_scales[-1].zero_()
    c.v_scales[-1].zero_()                          # zero rows (weight of x = 0) up to the appended ones
    k = torch.randn((n, H, d), device="cuda").bfloat16() * 4
    v = torch.randn((n, H, d), device="cuda").bfloat16()
    cu = i32([0] * B + [n])
    starts = i32([0] * (B - 1) + [at])
    msa.msa_kv4_append(c, k, v, starts, cu)
    kr, vr = msa.msa_kv4_read(c, starts, cu, n)
    assert torch.equal(kr.cpu(), torch.from_numpy(ref.values(*ref.quantise(k.float().cpu().numpy(), 1.0), 1.0)).bfloat16())
    q = (torch.randn((B, H, d), device="cuda") * 2).bfloat16()
    out, lse = msa.msa_kv4_decode(q, c, i32(lens))
    for r in range(H):
        K, V = kr[:, r].double().cpu().numpy(), vr[:, r].double().cpu().numpy()
        qh = q[-1, r:r + 1].double().cpu().numpy()
        x = np.concatenate([qh @ K.T / np.sqrt(d), np.zeros((1, at))], 1)
        p = np.exp(x - x.max())
        p /= p.sum()
        want = p[:, :n] @ V
        got = out[-1, r].double().cpu().numpy()
        e = 2.0 ** -16 * (np.abs(qh) @ np.abs(K).T).max() / np.sqrt(d) + 2.0 ** -25 * np.abs(qh).max() * np.abs(K).sum(-1).max() / np.sqrt(d)
        tol = (2.0 ** -11 + 2 * e + 2.0 ** -19) * (p[:, :n] @ np.abs(V))[0] + 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -32 * np.abs(V).sum(0)
        assert (np.abs(got - want[0]) <= tol).all()
    to = msa.KV4Cache.empty(B, 2048, H, d)
    w = torch.zeros((B, H, L_max), device="cuda")
    w[-1, :, at:] = torch.rand((H, n), device="cuda") + 1
    left, kept = msa.msa_kv4_evict(c, to, w, i32(lens), 2000)
    for r in range(H):
        want = ref.keep_positions(w[-1, r].cpu().numpy(), L_max, 2000, 0, 0)
        assert np.array_equal(kept[-1, r].cpu().numpy(), want)
        assert torch.equal(to.v_codes[-1, r, :2000], c.v_codes[-1, r, torch.from_numpy(want).cuda()])


# ------------------------------------------------------------------------------------------ block-sparse decode
@pytest.mark.parametrize("shape", [(4, 128, 16, 64, 16), (2, 64, 4, 32, 3)], ids=["G16", "G4_small"])
def test_sparse_decode(shape):
    """Selections equal msa_sparse_decode's on the same index keys; the attention is that of the 4-bit values."""
    H, d, G, d_idx, k = shape
    lens = [1, 128, 129, 3000, 2500, 777]
    B, L_max = len(lens), 3200
    c = fill_cache(B, L_max, H, d, lens, seed=11)
    g = torch.Generator("cuda").manual_seed(12)
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    q_idx = torch.randint(-3, 4, (B, H, d_idx), device="cuda", generator=g).bfloat16()
    k_idx = torch.randint(-3, 4, (B, L_max, H, d_idx), device="cuda", generator=g).bfloat16()
    zeros = torch.zeros((B, L_max, H, d), device="cuda", dtype=torch.bfloat16)
    _, _, want = msa.msa_sparse_decode(q, q_idx, zeros, zeros, k_idx, i32(lens), 128, k)
    w = torch.rand((B, H, L_max), device="cuda")
    w_out = torch.full_like(w, 9.0)
    out, lse, sel = msa.msa_sparse_decode_kv4(q, q_idx, c, k_idx, i32(lens), 128, k, w, w_out, 0.75)
    assert torch.equal(sel, want)
    check_decode(c, q, lens, out, lse, sel.cpu().numpy(), w, w_out, torch.full_like(w, 9.0), 0.75)
    ws = torch.empty(msa.lib.msa_sparse_decode_kv4_workspace_size(B, L_max, H * G, H, 128, k), dtype=torch.uint8, device="cuda")
    bad = [0, 128, L_max + 1, 3000, 2500, 777]       # no token, more than the cache has
    o2, l2, s2 = msa.msa_sparse_decode_kv4(q, q_idx, c, k_idx, i32(bad), 128, k, workspace=ws)
    assert msa.msa_get_device_error(ws) == DEVICE_CHECK
    assert torch.equal(s2[[1, 3, 4, 5]], sel[[1, 3, 4, 5]]) and (s2[[0, 2]] == -1).all()
    check_decode(c, q, bad, o2, l2, s2.cpu().numpy(), seqs=[1, 3, 4, 5])  # split otherwise than above: the same to rounding


@pytest.mark.parametrize("k", [1, 2, 16])
def test_sparse_selection_long(k):
    """Top-k over rows of more blocks than a round of the selection holds, of many equal scores, and of one block;
    with one block to choose it is the local one. Outputs and weights (none before) are those of the blocks."""
    H, d, d_idx, G = 1, 64, 32, 2
    lens = [140001, 140000 - 128, 1, 40000]
    B, L_max = len(lens), 140032
    c = fill_cache(B, L_max, H, d, lens, seed=40 + k)
    g = torch.Generator("cuda").manual_seed(41)
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    q_idx = torch.randint(-3, 4, (B, H, d_idx), device="cuda", generator=g).bfloat16()
    k_idx = torch.randint(-1, 2, (B, L_max, H, d_idx), device="cuda", generator=g).bfloat16()
    q_idx[1] = 0                                     # all scores equal, zeros
    w_out = torch.full((B, H, L_max), 4.0, device="cuda")
    out, lse, sel = msa.msa_sparse_decode_kv4(q, q_idx, c, k_idx, i32(lens), 128, k, weights_out=w_out)
    for b, n in enumerate(lens):
        local = (n - 1) // 128
        s = (k_idx[b, :local * 128, 0].double() @ q_idx[b, 0].double()).view(local, 128).amax(-1).cpu().numpy() if local else np.zeros(0)
        best = np.lexsort((np.arange(local), -s))[:k - 1]
        want = np.full(k, -1)
        want[:len(best) + 1] = np.sort(np.append(best, local))
        assert sel[b, 0].tolist() == want.tolist(), b
    check_decode(c, q, lens, out, lse, sel.cpu().numpy(), None, w_out, torch.full_like(w_out, 4.0))


def test_sparse_many_sequences():
    """More sequences than a CTA has threads, of which many own no whole block, a run of them in a row: every
    sequence's blocks are scored, and its outputs are those of the blocks."""
    B, H, G, d, d_idx, k, L_max = 700, 1, 2, 64, 32, 3, 896
    rng = np.random.default_rng(60)
    lens = rng.integers(1, L_max + 1, size=B)
    lens[rng.random(B) < 0.3] = 77
    lens[100:420] = rng.integers(1, 129, size=320)
    c = fill_cache(B, L_max, H, d, lens, seed=61)
    g = torch.Generator("cuda").manual_seed(62)
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    q_idx = torch.randint(-3, 4, (B, H, d_idx), device="cuda", generator=g).bfloat16()
    k_idx = torch.randint(-3, 4, (B, L_max, H, d_idx), device="cuda", generator=g).bfloat16()
    out, lse, sel = msa.msa_sparse_decode_kv4(q, q_idx, c, k_idx, i32(lens), 128, k)
    s = torch.einsum("blhe,bhe->bl", k_idx.double(), q_idx.double()).view(B, L_max // 128, 128).amax(-1).cpu().numpy()
    for b, n in enumerate(lens):
        local = (n - 1) // 128
        best = np.lexsort((np.arange(local), -s[b, :local]))[:k - 1]
        want = np.full(k, -1)
        want[:len(best) + 1] = np.sort(np.append(best, local))
        assert sel[b, 0].tolist() == want.tolist(), b
    check_decode(c, q, lens, out, lse, sel.cpu().numpy())


@pytest.mark.parametrize("k", [3, 4, 16])
def test_sparse_selection_infinite_scores(k):
    """Blocks whose scores are all -inf come last, the lower first, and still fill a selection that has room; the
    cache in bf16 selects the same."""
    B, H, G, d, d_idx, n = 1, 1, 4, 64, 32, 700
    c = fill_cache(B, 768, H, d, [n], seed=51)
    g = torch.Generator("cuda").manual_seed(52)
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    q_idx = torch.full((B, H, d_idx), 2.0 ** 100, device="cuda").bfloat16()
    k_idx = torch.full((B, 768, H, d_idx), -1.0, device="cuda").bfloat16()
    k_idx[:, :128] = k_idx[:, 384:512] = -2.0 ** 100     # products of -2^200: blocks 0 and 3
    k_idx[:, 256:384] = 1.0                              # block 2 is the best
    want = {3: [1, 2, 5], 4: [1, 2, 4, 5], 16: [0, 1, 2, 3, 4, 5] + [-1] * 10}[k]
    out, lse, sel = msa.msa_sparse_decode_kv4(q, q_idx, c, k_idx, i32([n]), 128, k)
    assert sel.flatten().tolist() == want
    check_decode(c, q, [n], out, lse, sel.cpu().numpy())
    cu = i32([0, 768])
    c.k_scales[:, :, n:], c.v_scales[:, :, n:] = 0, 0
    kb, vb = msa.msa_kv4_read(c, i32([0]), cu, 768)
    o2, _, s2 = msa.msa_sparse_decode(q, q_idx, kb[None], vb[None], k_idx, i32([n]), 128, k)
    assert torch.equal(s2, sel)
    # bf16 P (twice 2^-8: above and below the line), partial and outputs: below 6 half steps of the largest |V|
    assert (o2.float() - out.float()).abs().max() <= 6 * 2.0 ** -8 * vb.float().abs().max()


# ------------------------------------------------------------------------------------------ eviction
def check_evict(c, to, w, lens, keep, recent, first, k_idx, fill):
    H, d_idx = c.H_kv, k_idx.shape[-1]
    w_to = torch.full((to.B, H, to.L_max), -1.0, device="cuda")
    k_to = torch.full((to.B, to.L_max, H, d_idx), 5.0, device="cuda", dtype=torch.bfloat16)
    left, kept = msa.msa_kv4_evict(c, to, w, i32(lens), keep, recent, first, w_to, k_idx, k_to)
    assert left.tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        m = min(n, keep)
        for r in range(H):
            want = ref.keep_positions(w[b, r].cpu().numpy(), n, keep, recent, first)
            got = kept[b, r].cpu().numpy()
            assert np.array_equal(got[:m], want), (b, r, n)
            assert (got[m:] == -1).all()
            j = torch.from_numpy(want).cuda()
            for x, y in ((c.k_codes, to.k_codes), (c.k_scales, to.k_scales), (c.v_codes, to.v_codes), (c.v_scales, to.v_scales)):
                assert torch.equal(y[b, r, :m], x[b, r, j])
                assert (y[b, r, m:] == fill).all(), "behind the last kept row"
            assert torch.equal(w_to[b, r, :m], w[b, r, j]) and (w_to[b, r, m:] == -1).all()
            assert torch.equal(k_to[b, :m, r], k_idx[b, j, r]) and (k_to[b, m:, r] == 5).all()


@pytest.mark.parametrize("case", [(64, 32, 100, 10, 3), (128, 64, 1, 0, 0), (128, 128, 257, 257, 0), (64, 64, 256, 0, 256),
                                  (128, 32, 1500, 200, 4)], ids=["small", "one", "recent_only", "first_only", "most"])
def test_evict(case):
    """Budgets from one token up, with nothing to choose, with all that choice; lengths below, at and above."""
    d, d_idx, keep, recent, first = case
    H, L_max = 3, 2048
    lens = [0, 1, keep - 1, keep, keep + 1, 1999, 2048]
    B = len(lens)
    c = fill_cache(B, L_max, H, d, lens, seed=keep)
    to = make_cache(B, (keep + 127) // 128 * 128 + 128, H, d, (c.k_scale, c.v_scale), fill=0x3C)
    g = torch.Generator("cuda").manual_seed(keep)
    w = torch.rand((B, H, L_max), device="cuda", generator=g)
    w[:, 1] = (w[:, 1] * 8).floor()                              # many equal weights, zeros among them
    w[4:, 2] = torch.where(w[4:, 2] < 0.5, 0.0, -0.0)            # all equal: the two zeros are one value
    w[6, 0] = torch.randn((L_max,), device="cuda", generator=g) * 1e-38  # signs, subnormal numbers
    k_idx = torch.randn((B, L_max, H, d_idx), device="cuda", generator=g).bfloat16()
    check_evict(c, to, w, lens, keep, recent, first, k_idx, 0x3C)


@pytest.mark.parametrize("n", [16385, 100003, 150001])
def test_evict_long(n):
    """Long sequences, weights as attention leaves them (a few heavy ones, most of one magnitude)."""
    H, d, keep = 2, 64, n // 5
    lens = [n, n - 7]
    L_max = (n + 127) // 128 * 128
    c = fill_cache(2, L_max, H, d, lens, seed=n)
    to = make_cache(2, (keep + 127) // 128 * 128, H, d, (c.k_scale, c.v_scale), fill=0x11)
    g = torch.Generator("cuda").manual_seed(n)
    w = torch.randn((2, H, L_max), device="cuda", generator=g).mul_(2).exp_() / n
    w[0, 1] = (w[0, 1] * n * 16).round()
    k_idx = torch.randn((2, L_max, H, 32), device="cuda", generator=g).bfloat16()
    check_evict(c, to, w, lens, keep, 100, 2, k_idx, 0x11)


def test_evict_without_companions_and_bad_length():
    B, H, d, L_max, keep = 3, 2, 128, 512, 128
    c = fill_cache(B, L_max, H, d, [512] * 3, seed=1)
    to = make_cache(B, 128, H, d, (c.k_scale, c.v_scale), fill=0x22)
    w = torch.rand((B, H, L_max), device="cuda")
    ws = torch.empty(msa.lib.msa_kv4_evict_workspace_size(B, H, keep), dtype=torch.uint8, device="cuda")
    left, kept = msa.msa_kv4_evict(c, to, w, i32([400, 513, 512]), keep, workspace=ws)
    assert msa.msa_get_device_error(ws) == DEVICE_CHECK
    assert left.tolist() == [128, 0, 128] and (kept[1] == -1).all() and (to.k_codes[1] == 0x22).all()
    for b, n in ((0, 400), (2, 512)):
        for r in range(H):
            want = ref.keep_positions(w[b, r].cpu().numpy(), n, keep, 0, 0)
            assert np.array_equal(kept[b, r].cpu().numpy(), want)
            assert torch.equal(to.k_codes[b, r], c.k_codes[b, r, torch.from_numpy(want).cuda()])


# ------------------------------------------------------------------------------------------ together
def test_serving_run():
    """Prompt rows in, decode steps that add a row and accumulate weights, an eviction, more steps."""
    B, H, G, d, L_max, keep = 3, 2, 8, 128, 640, 256
    g = torch.Generator("cuda").manual_seed(21)
    c = make_cache(B, L_max, H, d)
    lens = np.array([400, 37, 300])
    T = int(lens.sum())
    x = torch.randn((2, T, H, d), device="cuda", generator=g).bfloat16()
    msa.msa_kv4_append(c, x[0], x[1], i32([0] * B), i32(np.concatenate([[0], np.cumsum(lens)])))
    w = torch.zeros((B, H, L_max), device="cuda")

    def steps(c, lens, w, count):
        for _ in range(count):
            kv = torch.randn((2, B, H, d), device="cuda", generator=g).bfloat16()
            q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
            msa.msa_kv4_append(c, kv[0], kv[1], i32(lens))
            lens = lens + 1
            before = w.clone()
            out, lse = msa.msa_kv4_decode(q, c, i32(lens), weights=w, weights_out=w)
            check_decode(c, q, lens, out, lse, None, before, w, before, 1.0)
        return lens

    lens = steps(c, lens, w, 3)
    to = make_cache(B, 384, H, d, (c.k_scale, c.v_scale), fill=0x7F)
    w_to = torch.zeros((B, H, 384), device="cuda")
    left, kept = msa.msa_kv4_evict(c, to, w, i32(lens), keep, recent=16, first=4, weights_dst=w_to)
    assert left.tolist() == [256, 40, 256]
    for b in range(B):
        for r in range(H):
            want = ref.keep_positions(w[b, r].cpu().numpy(), int(lens[b]), keep, 16, 4)
            assert np.array_equal(kept[b, r, :len(want)].cpu().numpy(), want)
    steps(to, np.array(left.tolist()), w_to, 2)


def test_graph_replay_and_streams():
    """Captured calls give the eager results bit for bit and follow new inputs in the same buffers; two
    streams with workspaces of their own do not disturb one another."""
    B, H, G, d, L_max, d_idx, k = 4, 2, 16, 128, 1536, 64, 4
    lens = i32([1000, 1, 1536, 700])
    c = fill_cache(B, L_max, H, d, [1536] * 4, seed=31)
    to = make_cache(B, 512, H, d, (c.k_scale, c.v_scale), fill=0)
    g = torch.Generator("cuda").manual_seed(32)
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    q_idx = torch.randint(-3, 4, (B, H, d_idx), device="cuda", generator=g).bfloat16()
    k_idx = torch.randint(-3, 4, (B, L_max, H, d_idx), device="cuda", generator=g).bfloat16()
    kv = torch.randn((2, B, H, d), device="cuda", generator=g).bfloat16()
    w = torch.rand((B, H, L_max), device="cuda", generator=g)
    w_out = torch.zeros_like(w)  # stays 0 behind the lengths
    outs = {}

    def all_calls():
        msa.msa_kv4_append(c, kv[0], kv[1], lens - 1)
        outs["dense"] = msa.msa_kv4_decode(q, c, lens, weights=w, weights_out=w_out, decay=0.5)
        outs["sparse"] = msa.msa_sparse_decode_kv4(q, q_idx, c, k_idx, lens, 128, k)
        outs["evict"] = msa.msa_kv4_evict(c, to, w, lens, 500, 10, 1)
        outs["read"] = msa.msa_kv4_read(to, i32_zero)

    i32_zero = i32([0] * B)
    all_calls()
    torch.cuda.synchronize()
    eager = {n: [t.clone() for t in v] for n, v in outs.items()}
    eager_w = w_out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        all_calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_calls()
    captured = dict(outs)
    w_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n, v in captured.items():
        for x, y in zip(v, eager[n]):
            assert torch.equal(x, y), n
    assert torch.equal(w_out, eager_w)
    lens.copy_(i32([300, 1200, 2, 1536]))
    q.copy_(torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    replayed = {n: [t.clone() for t in v] for n, v in captured.items()}
    check_decode(c, q, [300, 1200, 2, 1536], *replayed["dense"])
    all_calls()
    for n, v in outs.items():
        for x, y in zip(v, replayed[n]):
            assert torch.equal(x, y), n
    # two streams at once
    want = msa.msa_kv4_decode(q, c, lens)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[msa.msa_kv4_decode(q, c, lens, stream=st) for st in streams] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for o, ls in pair:
            assert torch.equal(o, want[0]) and torch.equal(ls, want[1])
