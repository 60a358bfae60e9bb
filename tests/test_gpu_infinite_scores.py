"""Index scores that leave fp32's range: blocks of nothing but -inf come last, the lower first, in prefill as in
decode, and still fill a selection that has room, so that the combine reads no slot that nothing wrote."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import numpy as np  # noqa: E402

import block_sparse_long_idx_b200 as msa  # noqa: E402


def inputs(N, H_kv, H_q, d_h, d_idx):
    """Blocks 0, 3 (and 6 of the last group) score -inf, block 2 is the best, the others score below 0."""
    g = torch.Generator("cuda").manual_seed(N)
    q = torch.randn((N, H_q, d_h), device="cuda", generator=g).bfloat16()
    k = torch.randn((N, H_kv, d_h), device="cuda", generator=g).bfloat16()
    v = torch.randn((N, H_kv, d_h), device="cuda", generator=g).bfloat16()
    q_idx = torch.full((N, H_kv, d_idx), 2.0 ** 100, device="cuda").bfloat16()
    k_idx = torch.full((N, H_kv, d_idx), -1.0, device="cuda").bfloat16()
    k_idx[:128] = k_idx[384:512] = -2.0 ** 100
    k_idx[768:896, -1] = -2.0 ** 100
    k_idx[256:384] = 1.0
    return q, k, v, q_idx, k_idx


def order(r, H_kv):
    """Blocks, the best first (of nine)."""
    low = [0, 3, 6] if r == H_kv - 1 else [0, 3]
    return [2] + [b for b in range(9) if b != 2 and b not in low] + low


def expected(i, r, H_kv, kk):
    local = i // 128
    best = [b for b in order(r, H_kv) if b < local][: kk - 1]
    sel = sorted(best + [local])
    return sel + [-1] * (kk - len(sel))


def attend(q, k, v, i, sel):
    """fp64 outputs and lse [H_q] of row i over the blocks sel[r] of its sequence."""
    H_q, H_kv = q.shape[1], k.shape[1]
    G = H_q // H_kv
    outs, lses = [], []
    for r in range(H_kv):
        j = torch.cat([torch.arange(b * 128, min(i + 1, b * 128 + 128)) for b in sel[r] if b >= 0]).cuda()
        x = q[i, r * G:(r + 1) * G].double() @ k[j, r].double().T / q.shape[2] ** 0.5
        outs.append(torch.softmax(x, -1) @ v[j, r].double())
        lses.append(torch.logsumexp(x, -1))
    return torch.cat(outs), torch.cat(lses)


@pytest.mark.parametrize("kk", [1, 3, 4, 16])
@pytest.mark.parametrize("packed", [False, True], ids=["one", "packed"])
def test_prefill_selection_infinite_scores(kk, packed):
    N, H_kv, H_q, d_h, d_idx = 1100, 2, 8, 64, 32
    q, k, v, q_idx, k_idx = inputs(N, H_kv, H_q, d_h, d_idx)
    if packed:
        cu = np.array([0, N, 2 * N], np.int32)
        need = msa.lib.msa_sparse_prefill_varlen_workspace_size(cu.ctypes.data, None, 2, H_q, H_kv, d_h, 128, kk, 0)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN where nothing is written
        two = [torch.cat([t, t]) for t in (q, k, v, q_idx, k_idx)]
        out, lse, sel = msa.msa_sparse_prefill_varlen(*two, cu, 128, kk, workspace=ws)
        assert torch.equal(out[:N], out[N:]) and torch.equal(lse[:N], lse[N:]) and torch.equal(sel[:, :N], sel[:, N:])
        out, lse, sel = out[:N], lse[:N], sel[:, :N]
    else:
        sel = msa.msa_index_topk(q_idx, k_idx, 128, kk)
        ws = torch.full((msa.msa_sparse_prefill_workspace_size(N, H_q, H_kv, d_h, 128, kk, 0, True),), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse = msa.msa_sparse_prefill(q, k, v, sel, workspace=ws)
    rows = [0, 127, 128, 400, 511, 640, 1023, 1099]
    for i in rows:
        want = [expected(i, r, H_kv, kk) for r in range(H_kv)]
        assert sel[:, i].tolist() == want, i
        o, ls = attend(q, k, v, i, want)
        # half steps of 2^-8 of the largest |V|: of P twice (itself and its sum), of partials and of outputs, and two to spare
        assert (out[i].double() - o).abs().max() <= 6 * 2.0 ** -8 * v.float().abs().max()
        assert (lse[i].double() - ls).abs().max() <= 1e-3
    # decode selects the same for the same rows
    L_max = 1152
    pad = torch.zeros((L_max - N,) + k.shape[1:], device="cuda", dtype=torch.bfloat16)
    pad_idx = torch.zeros((L_max - N,) + k_idx.shape[1:], device="cuda", dtype=torch.bfloat16)
    kc, vc, ic = torch.cat([k, pad]), torch.cat([v, pad]), torch.cat([k_idx, pad_idx])
    B = len(rows)
    at = torch.tensor(rows, device="cuda")
    _, _, dsel = msa.msa_sparse_decode(q[at].contiguous(), q_idx[at].contiguous(), kc.expand(B, -1, -1, -1).contiguous(),
                                       vc.expand(B, -1, -1, -1).contiguous(), ic.expand(B, -1, -1, -1).contiguous(),
                                       (at + 1).int(), 128, kk)
    assert torch.equal(dsel.transpose(0, 1), sel[:, at])
