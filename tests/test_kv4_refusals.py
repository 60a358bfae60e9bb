"""What the 4-bit cache's entry points refuse on the host, and what its handle does not let a program change. No GPU needed."""
import pytest

from tests.test_kv4_host import INVALID, P2, WORKSPACE, WS, cache, caller, msa  # noqa: F401


def test_out_over_q(msa):  # noqa: F811
    """Outputs may replace q, but not shifted, and not where the weights read q again."""
    row = 8 * 128 * 2
    far = P2 + (1 << 30)
    need = msa.lib.msa_kv4_decode_workspace_size(4, 8)
    f = caller(msa.lib.msa_kv4_decode, ["cache", "q", "lens", "H_q", "blocks", "k", "w_in", "w_out", "decay", "out", "lse", "ws", "n",
                                        "stream"],
               [cache(msa), P2, far, 8, None, 0, None, None, 1.0, P2, far, WS, need - 1, None])
    assert f() == WORKSPACE and f(out=P2 + 4 * row) == WORKSPACE                       # accepted but for the size
    assert f(out=P2 + row) == INVALID and f(out=P2 - row) == INVALID and f(out=P2 + 4 * row - 16) == INVALID
    assert f(w_out=far + (1 << 30)) == INVALID
    assert f(w_out=far + (1 << 30), out=P2 + 4 * row) == WORKSPACE
    need = msa.lib.msa_sparse_decode_kv4_workspace_size(4, 1024, 8, 2, 128, 4)
    g = caller(msa.lib.msa_sparse_decode_kv4, ["cache", "q", "q_idx", "k_idx", "lens", "H_q", "d_idx", "B_k", "k", "w_in", "w_out",
                                               "decay", "out", "lse", "sel", "ws", "n", "stream"],
               [cache(msa), P2, far, far, far, 8, 64, 128, 4, None, None, 1.0, P2, None, None, WS, need - 1, None])
    assert g() == WORKSPACE and g(out=P2 + row) == INVALID and g(w_out=far + (1 << 30)) == INVALID
