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


def test_handle_is_fixed(msa, monkeypatch):  # noqa: F811
    """The kernels read the pointers and scales of construction: a field that was set anew would say something else, and a
    tensor that was replaced would leave a stale pointer behind."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(msa.api, "_is", lambda t, *a: t)               # tensors of the CPU, never read
    codes = [torch.zeros((1, 2, 128, 64), dtype=torch.uint8) for _ in range(2)]
    scales = [torch.zeros((1, 2, 128, 8), dtype=torch.uint8) for _ in range(2)]
    c = msa.KV4Cache(codes[0], scales[0], codes[1], scales[1], 0.5, 2.0)
    assert (c.B, c.H_kv, c.L_max, c.d_h, c.k_scale, c.v_scale) == (1, 2, 128, 128, 0.5, 2.0)
    assert c._c.k_codes == codes[0].data_ptr() and c._c.v_scales == scales[1].data_ptr() and c._c.v_scale == 2.0
    for name, value in (("k_scale", 1.0), ("v_scale", 1.0), ("k_codes", codes[1]), ("v_scales", scales[0]), ("L_max", 256)):
        before = getattr(c, name)
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, value)
        with pytest.raises(AttributeError, match=name):
            delattr(c, name)
        assert getattr(c, name) is before
    c.k_scales[:, :, 100:] = 7                                         # contents are the program's
    c.note = "a program's own"
    del c.note
