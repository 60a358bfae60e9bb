"""The 4-bit cache where its inputs are hard: NaN, scales at the ends of fp32, lists of blocks out of order, memory of
calls on a stream of their own, and the kernels' rarer instances. Tolerances are those of test_gpu_kv4.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import block_sparse_long_idx_b200 as msa  # noqa: E402
from tests import ref_kv4 as ref  # noqa: E402
from tests.test_gpu_kv4 import DEVICE_CHECK, check_decode, fill_cache, host_values, i32, make_cache  # noqa: E402


# ------------------------------------------------------------------------------------------ NaN
def check_nan(c, q, lens, out, lse, w_out, w_before, block_idx=None):
    """out, lse and w_out (of no earlier weights) are NaN where the definition's are, and right elsewhere."""
    H, d = c.H_kv, c.d_h
    G = q.shape[1] // H
    for b, n in enumerate(lens):
        for r in range(H):
            pos = np.arange(n)
            if block_idx is not None:
                pos = np.concatenate([np.arange(x * 128, min(n, x * 128 + 128)) for x in block_idx[b][r] if x >= 0]).astype(int)
            K, V = host_values(c, b, r, n)
            K, V = K[pos], V[pos]
            hs = slice(r * G, (r + 1) * G)
            qh = q[b, hs].double().cpu().numpy()
            want, wl, p, pv, _ = ref.attend(qh, K, V)
            qa, ka = np.nan_to_num(np.abs(qh)), np.nan_to_num(np.abs(K))
            e = 2.0 ** -16 * (qa @ ka.T).max() / np.sqrt(d) + 2.0 ** -25 * qa.max() * ka.sum(-1).max() / np.sqrt(d)
            got = out[b, hs].double().cpu().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(want)), (b, r)
            tol = (2.0 ** -11 + 2 * e + 2.0 ** -19) * pv + 2.0 ** -8 * np.abs(want) + 2.0 ** -32 * np.nansum(np.abs(V), 0)
            ok = ~np.isnan(want)
            assert (np.abs(got - want)[ok] <= tol[ok]).all(), (b, r)
            got = lse[b, hs].double().cpu().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(wl)), (b, r, got)
            ok = ~np.isnan(wl)
            assert (np.abs(got - wl)[ok] <= (e + 2.0 ** -22 * np.abs(wl) + 2.0 ** -20)[ok]).all(), (b, r)
            got = w_out[b, r].double().cpu().numpy()
            add = np.zeros(n)
            add[pos] = p.sum(0)
            assert np.array_equal(np.isnan(got[:n]), np.isnan(add)), (b, r)
            ok = ~np.isnan(add)
            assert (np.abs(got[:n] - add)[ok] <= ((2.0 ** -22 + 2 * e + 2.0 ** -19) * add)[ok]).all(), (b, r)
            assert np.array_equal(got[n:], w_before[b, r, n:].double().cpu().numpy()), "behind the length"


@pytest.mark.parametrize("n", [200, 20001], ids=["one_cta", "split"])
@pytest.mark.parametrize("d, G", [(128, 16), (64, 3)])
def test_nan(d, G, n):
    """A NaN in one head's q gives that head NaN, and its KV head's weights; a NaN key gives its KV head NaN; a NaN in V
    gives NaN in its 16 elements alone. Nothing of it reaches the other heads and sequences, and no row that sees
    keys says that it sees none (lse = -inf)."""
    B, H = 2, 4
    lens = [n, 77]
    L_max = (n + 127) // 128 * 128
    g = torch.Generator("cuda").manual_seed(n)
    c = make_cache(B, L_max, H, d)
    k = torch.randn((n + 77, H, d), device="cuda", generator=g)
    v = torch.randn((n + 77, H, d), device="cuda", generator=g)
    k[n - 3, 1, 5] = float("nan")
    v[70, 2, d - 1] = float("nan")
    msa.msa_kv4_append(c, k.bfloat16(), v.bfloat16(), i32([0, 0]), i32([0, n, n + 77]))
    q = torch.randn((B, H * G, d), device="cuda", generator=g)
    q[0, 1, 3] = q[1, 3 * G + 2, 0] = float("nan")    # KV heads 0 and 3
    q = q.bfloat16()
    before = torch.full((B, H, L_max), 3.0, device="cuda")
    w_out = before.clone()
    out, lse = msa.msa_kv4_decode(q, c, i32(lens), weights_out=w_out)
    check_nan(c, q, lens, out, lse, w_out, before)
    # given blocks: the NaN key's block is given to KV head 1 of one list and not of the other
    last = (n - 1) // 128
    for mine in ([last - 1, last], [last - 1, -1]):
        sel = np.tile(np.array([0, -1], np.int32), (B, H, 1))
        sel[0, 1] = mine
        w_out = before.clone()
        out, lse = msa.msa_kv4_decode(q, c, i32(lens), torch.from_numpy(sel).cuda(), weights_out=w_out)
        check_nan(c, q, lens, out, lse, w_out, before, sel)


# ------------------------------------------------------------------------------------------ eviction of NaN weights
def test_evict_nan_weights():
    """A NaN weight counts as the largest whatever its sign, equal to other NaNs: the lower position stays first."""
    B, H, d, L_max, n, keep = 1, 2, 64, 512, 500, 40
    c = fill_cache(B, L_max, H, d, [n], seed=3)
    to = make_cache(B, 128, H, d, (c.k_scale, c.v_scale), fill=0)
    w = torch.rand((B, H, L_max), device="cuda")
    w[0, :, 17] = float("inf")
    bits = w.view(torch.int32)
    bits[0, 0, 100::7], bits[0, 0, 103::7] = 0x7FC00000, -0x400000        # + and - NaN
    bits[0, 1, 50:90] = -1                                                # 40 NaNs, all that stay
    _, kept = msa.msa_kv4_evict(c, to, w, i32([n]), keep)
    w64 = torch.where(w.isnan(), float("inf"), w.clamp(max=3.0)).double().cpu().numpy()
    for r in range(H):
        assert kept[0, r].tolist() == ref.keep_positions(w64[0, r], n, keep, 0, 0).tolist()


# ------------------------------------------------------------------------------------------ scales at the ends of fp32
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("v_scale", [2.0 ** -124, 2.0 ** -110, 2.0 ** 110])
def test_v_scale_range(v_scale, G):
    """A long flat row, whose sum of P passes 2^22, on a V scale near fp32's ends: outputs are normal numbers there."""
    B, H, d, n = 1, 1, 64, 40001
    g = torch.Generator("cuda").manual_seed(G)
    c = make_cache(B, 40064, H, d, (1.0, v_scale))
    k = torch.randn((n, H, d), device="cuda", generator=g) * 0.01
    v = (torch.randn((n, H, d), device="cuda", generator=g) + 4) * v_scale
    msa.msa_kv4_append(c, k.bfloat16(), v.bfloat16(), i32([0]), i32([0, n]))
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    out, _ = msa.msa_kv4_decode(q, c, i32([n]))
    K, V = host_values(c, 0, 0, n)
    qh = q[0].double().cpu().numpy()
    want, _, _, pv, S = ref.attend(qh, K, V)
    e = 2.0 ** -16 * S + 2.0 ** -25 * np.abs(qh).max() * np.abs(K).sum(-1).max() / np.sqrt(d)
    tol = (2.0 ** -11 + 2 * e + 2.0 ** -19) * pv + 2.0 ** -8 * np.abs(want) + 2.0 ** -32 * np.abs(V).sum(0)
    assert (np.abs(out[0].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_k_scale_subnormal(d, G):
    """A subnormal K scale under enormous q: logits of a few units, whose factor keeps all of its bits."""
    B, H, n = 1, 1, 300
    g = torch.Generator("cuda").manual_seed(d)
    c1 = make_cache(B, 384, H, d)
    k = torch.randint(0, 2049, (n, H, 1), device="cuda", generator=g).float().expand(n, H, d)
    v = torch.randn((n, H, d), device="cuda", generator=g)
    msa.msa_kv4_append(c1, k.bfloat16(), v.bfloat16(), i32([0]), i32([0, n]))
    c = msa.KV4Cache(c1.k_codes, c1.k_scales, c1.v_codes, c1.v_scales, 2.0 ** -140, 1.0)
    q = torch.linspace(0.5, 1.0, H * G, device="cuda").view(1, -1, 1).expand(B, H * G, d).mul(2.0 ** 127).bfloat16()
    w_out = torch.zeros((B, H, 384), device="cuda")
    out, lse = msa.msa_kv4_decode(q, c, i32([n]), weights_out=w_out)
    assert lse.max() > 6.2  # log(300) is 5.7: the logits count
    check_decode(c, q, [n], out, lse, w_out=w_out, w_before=torch.zeros_like(w_out))


# ------------------------------------------------------------------------------------------ lists of blocks out of order
@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("G", [4, 16])
def test_blocks_given_twice(G, H):
    """An entry that does not exceed every block before it in its list is left out, from the weights too, and reported;
    entries outside the sequence do not count for those behind them, nor does padding."""
    B, d, L_max, n = 2, 128, 1024, 1000
    lists = [([3, -1, 3, -1], [3]), ([4, 2, 3, 4], [4]), ([2, 0, 2, 7], [2, 7]), ([9, 1, 8, 5], [1, 5]), ([-5, 6, 2 ** 31 - 1, 6], [6]),
             ([1, 1, 1, 1], [1])]
    c = fill_cache(B, L_max, H, d, [n, n], seed=8)
    g = torch.Generator("cuda").manual_seed(9)
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    w = torch.rand((B, H, L_max), device="cuda", generator=g)
    ws = torch.empty(msa.lib.msa_kv4_decode_workspace_size(B, H * G), dtype=torch.uint8, device="cuda")
    for given, kept in lists:
        sel = np.tile(np.array([0, 3, 5, -1], np.int32), (B, H, 1))
        want = sel.copy()
        sel[1, H - 1] = given
        want[1, H - 1] = kept + [-1] * (4 - len(kept))
        w_out = torch.full_like(w, 7.0)
        out, lse = msa.msa_kv4_decode(q, c, i32([n, n]), torch.from_numpy(sel).cuda(), w, w_out, 0.5, workspace=ws)
        assert msa.msa_get_device_error(ws) == DEVICE_CHECK, given
        check_decode(c, q, [n, n], out, lse, want, w, w_out, torch.full_like(w, 7.0), 0.5)
    sel = np.tile(np.array([0, -1, 1, -1], np.int32), (B, H, 1))     # padding in between
    out, lse = msa.msa_kv4_decode(q, c, i32([n, n]), torch.from_numpy(sel).cuda(), workspace=ws)
    assert msa.msa_get_device_error(ws) == 0
    check_decode(c, q, [n, n], out, lse, sel)


# ------------------------------------------------------------------------------------------ out in the place of q
@pytest.mark.parametrize("G", [4, 16])
def test_out_in_place_of_q(G):
    """Without weights the outputs may replace q (segments of one CTA, of several)."""
    B, H, d, L_max = 5, 2, 64, 8064
    lens = [8000, 1, 700, 0, 4095]
    c = fill_cache(B, L_max, H, d, lens, seed=14)
    q = torch.randn((B, H * G, d), device="cuda").bfloat16()
    x = q.clone()
    out, lse = msa.msa_kv4_decode(x, c, i32(lens), out=x)
    assert out is x
    check_decode(c, q, lens, out, lse)
    with pytest.raises(msa.MsaError):
        msa.msa_kv4_decode(x, c, i32(lens), weights_out=torch.zeros((B, H, L_max), device="cuda"), out=x)


# ------------------------------------------------------------------------------------------ rarer instances
@pytest.mark.parametrize("G", [9, 16])
def test_wide_groups_of_64(G):
    """d_h 64 with more than 8 heads a KV head: given blocks, and weights with and without them."""
    B, H, d, k, L_max = 4, 2, 64, 5, 2176
    lens = [2100, 129, 640, 0]
    sel = np.full((B, H, k), -1, np.int32)
    sel[0, 0], sel[0, 1] = [0, 2, 3, 9, 16], [1, 7, -1, -1, -1]
    sel[1, 0, :2], sel[1, 1, :1] = [0, 1], [1]
    sel[2, 0, :1] = [4]                                  # sel[2, 1]: nothing
    c = fill_cache(B, L_max, H, d, lens, seed=G)
    g = torch.Generator("cuda").manual_seed(G)
    q = torch.randn((B, H * G, d), device="cuda", generator=g).bfloat16()
    w = torch.rand((B, H, L_max), device="cuda", generator=g)
    before = torch.full_like(w, 7.0)
    for blocks in (None, sel):
        w_out = before.clone()
        out, lse = msa.msa_kv4_decode(q, c, i32(lens), None if blocks is None else torch.from_numpy(blocks).cuda(), w, w_out, 0.25)
        check_decode(c, q, lens, out, lse, blocks, w, w_out, before, 0.25)


@pytest.mark.parametrize("d", [64, 128])
def test_read_many_rows(d):
    """Rows enough for several row steps to a reading CTA, the last one ragged."""
    B, H, L_max = 3, 4, 9088
    lens, starts = [9001, 4, 8700], [87, 9084, 1]
    T = sum(lens)
    g = torch.Generator("cuda").manual_seed(d)
    x = torch.randn((2, T, H, d), device="cuda", generator=g).bfloat16()
    c = make_cache(B, L_max, H, d, (0.5, 2.0))
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    msa.msa_kv4_append(c, x[0], x[1], i32(starts), cu)
    kr, vr = msa.msa_kv4_read(c, i32(starts), cu, T)
    for got, src, t in ((kr, x[0], 0.5), (vr, x[1], 2.0)):
        want = ref.values(*ref.quantise(src.float().cpu().numpy(), t), t)
        assert torch.equal(got.cpu(), torch.from_numpy(want).float().bfloat16())


def test_prefix_of_a_packed_prefill():
    """Rows read back are the cached prefix of msa_sparse_prefill_varlen: the last row of every chunk selects the blocks
    of, and attends like, the block-sparse decode of the same position on the cache itself."""
    B, H, G, d, d_idx, kk, L_max = 3, 2, 4, 128, 32, 4, 1280
    prefix, chunk = [1024, 0, 384], [200, 77, 640]
    lens = [p + m for p, m in zip(prefix, chunk)]
    c = fill_cache(B, L_max, H, d, lens, seed=33)
    Tk = sum(lens)
    cu_k = np.concatenate([[0], np.cumsum(lens)])
    k, v = msa.msa_kv4_read(c, i32([0] * B), i32(cu_k), Tk)
    g = torch.Generator("cuda").manual_seed(34)
    T = sum(chunk)
    cu = np.concatenate([[0], np.cumsum(chunk)])
    q = torch.randn((T, H * G, d), device="cuda", generator=g).bfloat16()
    q_idx = torch.randint(-3, 4, (T, H, d_idx), device="cuda", generator=g).bfloat16()
    k_idx = torch.randint(-3, 4, (Tk, H, d_idx), device="cuda", generator=g).bfloat16()
    out, lse, sel = msa.msa_sparse_prefill_varlen(q, k, v, q_idx, k_idx, cu, 128, kk, cu_seqlens_k=cu_k)
    k_idx_cache = torch.zeros((B, L_max, H, d_idx), device="cuda", dtype=torch.bfloat16)
    for b in range(B):
        k_idx_cache[b, :lens[b]] = k_idx[cu_k[b]:cu_k[b + 1]]
    last = torch.from_numpy(cu[1:] - 1).cuda()
    o, ls, s = msa.msa_sparse_decode_kv4(q[last].contiguous(), q_idx[last].contiguous(), c, k_idx_cache, i32(lens), 128, kk)
    check_decode(c, q[last], lens, o, ls, s.cpu().numpy())
    assert torch.equal(sel[:, last].transpose(0, 1), s)
    # rows are exact in bf16 (6 bits times 1 or 0.75); half steps of 2^-8 of the largest |V|: of the packed form's P twice (itself
    # and its sum), its partials and both outputs, and one to spare for the rest
    assert (out[last].float() - o.float()).abs().max() <= 6 * 2.0 ** -8 * v.float().abs().max()
    # products of at most S = |q| |K| / sqrt(d) in fp32 on both sides
    S = (q[last].float().norm(dim=-1).max() * k.float().norm(dim=-1).max() / d ** 0.5).item()
    assert (lse[last] - ls).abs().max() <= 2.0 ** -14 * S + 2.0 ** -18
