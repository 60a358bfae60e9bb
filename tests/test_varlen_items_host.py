"""The packed prefill's workspace holds a work item for every block that the rows of a window can select: more blocks than
the rows' own where sequences are short or continue cached prefixes. No GPU needed (sizes only)."""
import os

import numpy as np
import pytest


@pytest.fixture(scope="module")
def msa():
    from block_sparse_long_idx_b200 import build

    if not os.path.exists(build.LIB):
        build.build()
    import block_sparse_long_idx_b200 as m

    return m


def items_needed(cu, cu_k, H_kv, k, window=2048, chunk=512):
    """The most items that selections of the batch can give: in every window and group k blocks a row, each block as few
    times above whole chunks as hurts most (once)."""
    total = 0
    T = int(cu[-1])
    for lo in range(0, T, window):
        hi = min(T, lo + window)
        visible, entries = 0, 0
        for s in range(len(cu) - 1):
            a, b = max(lo, int(cu[s])), min(hi, int(cu[s + 1]))
            if a < b:
                prefix = int(cu_k[s + 1] - cu_k[s]) - int(cu[s + 1] - cu[s])
                rows = np.arange(a, b) - int(cu[s]) + prefix
                seen = rows // 128 + 1
                visible += min(int(seen[-1]), int(np.minimum(seen, k).sum()))
                entries += int(np.minimum(seen, k).sum())
        # every visible block once, and the other entries in whole chunks on top of it
        total += H_kv * (min(visible, entries) + max(0, entries - visible) // chunk)
    return total


BATCHES = [([1] * 2048, [0] * 2048, 1, 1), ([200, 77, 640], [1024, 0, 384], 2, 4), ([1] * 64, [16384] * 64, 4, 16),
           ([100, 4096], [0, 0], 1, 16), ([700, 1, 0, 3000, 5], [128 * 500, 0, 256, 128 * 300, 128], 2, 16), ([5000], [0], 2, 8)]


@pytest.mark.parametrize("batch", BATCHES, ids=[str(i) for i in range(len(BATCHES))])
def test_workspace_holds_every_item(msa, batch):
    lens, prefix, H_kv, k = batch
    H_q, d_h, B = H_kv, 64, len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(np.array(lens) + np.array(prefix))]).astype(np.int32)
    T, NB = int(cu[-1]), int(((np.diff(cu_k) + 127) // 128).sum())
    windows = -(-T // 2048)
    got = msa.lib.msa_sparse_prefill_varlen_workspace_size(cu.ctypes.data, cu_k.ctypes.data, B, H_q, H_kv, d_h, 128, k, 0)
    pairs = sum((n + 255) // 256 for n in lens)                       # query tiles, two at a time
    others = 3 * 4 * (B + 1) + 8 * pairs + 8 * T + 8 * NB             # offsets, tile pairs, per row and per block tables
    others += 4 * H_kv * (NB + 1) + 4 * H_kv * T * k + 4 * (windows + 1) + 12 * H_kv * NB * windows  # the inversion but its items
    others += windows * 2048 * k * H_q * (2 * d_h + 4)                # partials
    room = got - others
    need = 16 * items_needed(cu, cu_k, H_kv, k)
    assert room >= need, (room, need)
