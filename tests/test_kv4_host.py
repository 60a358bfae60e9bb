"""The 4-bit cache's entry points on the host, no GPU needed: every refusal of the C ABI before the device is
touched, workspace sizes, the binding's checks of tensors, and the float64 reference against its own format."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from tests import ref_kv4 as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
P, P2, WS = 0x10_0000_0000, 0x20_0000_0000, 0x30_0000_0000  # fake, aligned, far apart (never dereferenced)
BIG = 1 << 40


@pytest.fixture(scope="module")
def msa():
    from block_sparse_long_idx_b200 import build

    if not os.path.exists(build.LIB):
        build.build()
    import block_sparse_long_idx_b200 as m

    assert m.lib is not None  # loads the binding
    return m


def cache(msa, base=P, **kw):
    f = dict(k_codes=base, k_scales=base + 0x4000_0000, v_codes=base + 0x8000_0000, v_scales=base + 0xC000_0000, B=4, H_kv=2, d_h=128,
             L_max=1024, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return msa.api.msa_kv4_cache(*f.values())


BAD_CACHES = [(dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID), (dict(k_scales=P + 8), INVALID),
              (dict(B=0), INVALID), (dict(H_kv=0), INVALID), (dict(L_max=0), INVALID), (dict(k_scale=0.0), INVALID),
              (dict(v_scale=-1.0), INVALID), (dict(k_scale=float("nan")), INVALID), (dict(v_scale=float("inf")), INVALID),
              (dict(d_h=96), UNSUPPORTED), (dict(L_max=1000), UNSUPPORTED), (dict(L_max=(1 << 21) + 128), UNSUPPORTED),
              (dict(B=40000), UNSUPPORTED), (dict(B=32768, H_kv=1, L_max=1 << 21), UNSUPPORTED)]


def caller(f, names, values):
    def call(**kw):
        a = dict(zip(names, values))
        for n in kw:
            assert n in a, n
        a.update(kw)
        return f(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a.values()])

    return call


@pytest.mark.parametrize("bad", BAD_CACHES, ids=[str(i) for i in range(len(BAD_CACHES))])
def test_bad_caches(msa, bad):
    fields, status = bad
    c = cache(msa, **fields)
    good = cache(msa, base=0x50_0000_0000)
    B, lib = c.B, msa.lib
    r = ctypes.byref(c)
    assert lib.msa_kv4_append(r, P2, P2, 4096, 4096, B, P2, None, WS, BIG, None) == status
    assert lib.msa_kv4_read(r, P2, P2, B, P2, None, WS, BIG, None) == status
    assert lib.msa_kv4_decode(r, P2, P2, 8, None, 0, None, None, 1.0, P2, None, WS, BIG, None) == status
    assert lib.msa_sparse_decode_kv4(r, P2, P2, P2, P2, 8, 64, 128, 4, None, None, 1.0, P2, None, None, WS, BIG, None) == status
    assert lib.msa_kv4_evict(r, ctypes.byref(good), P2, P2, 8, 0, 0, None, None, 0, None, WS + 512, WS + 1024, WS, BIG, None) == status
    assert lib.msa_kv4_evict(ctypes.byref(good), r, P2, P2, 8, 0, 0, None, None, 0, None, WS + 512, WS + 1024, WS, BIG, None) == status
    assert lib.msa_kv4_decode(None, P2, P2, 8, None, 0, None, None, 1.0, P2, None, WS, BIG, None) == INVALID


def test_rows_validation(msa):
    need = msa.lib.msa_kv4_rows_workspace_size()
    app = caller(msa.lib.msa_kv4_append, ["cache", "k", "v", "ks", "vs", "T", "starts", "cu", "ws", "n", "stream"],
                 [cache(msa), P2, P2, 256, 256, 9, P2, P2, WS, need, None])
    assert app(k=None) == INVALID and app(v=P2 + 2) == INVALID and app(starts=None) == INVALID
    assert app(ks=255) == INVALID and app(ks=248) == INVALID and app(vs=260) == INVALID   # below a row; not a multiple of 8
    assert app(T=-1) == INVALID and app(cu=None) == INVALID                                # T rows need T = B without tables
    assert app(T=4 * 1024 + 1) == INVALID                                                  # more rows than the cache has
    assert app(cu=P2 + 2) == INVALID and app(ws=WS + 16) == INVALID
    assert app(n=need - 1) == WORKSPACE
    rd = caller(msa.lib.msa_kv4_read, ["cache", "k", "v", "T", "starts", "cu", "ws", "n", "stream"],
                [cache(msa), P2, P2, 9, P2, P2, WS, need, None])
    assert rd(k=None) == INVALID and rd(v=P2 + 8) == INVALID and rd(cu=None) == INVALID and rd(n=0) == WORKSPACE
    assert rd(starts=None) == INVALID and rd(T=-3) == INVALID


def test_decode_validation(msa):
    need = msa.lib.msa_kv4_decode_workspace_size(4, 8)
    assert need > 0 and msa.lib.msa_kv4_decode_workspace_size(0, 8) == 0
    assert msa.lib.msa_kv4_decode_workspace_size(4096, 64) >= need + 4 * 4092 * 56
    f = caller(msa.lib.msa_kv4_decode, ["cache", "q", "lens", "H_q", "blocks", "k", "w_in", "w_out", "decay", "out", "lse", "ws", "n",
                                        "stream"],
               [cache(msa), P2, P2, 8, None, 0, None, None, 1.0, P2, P2, WS, need, None])
    assert f(q=None) == INVALID and f(lens=None) == INVALID and f(out=None) == INVALID and f(ws=None) == INVALID
    assert f(q=P2 + 8) == INVALID and f(out=P2 + 8) == INVALID and f(lse=P2 + 2) == INVALID and f(ws=WS + 128) == INVALID
    assert f(H_q=0) == INVALID and f(H_q=7) == INVALID and f(H_q=34) == UNSUPPORTED          # G = 17
    assert f(blocks=P2, k=0) == INVALID and f(blocks=P2 + 2, k=4) == INVALID and f(blocks=P2, k=17) == UNSUPPORTED
    assert f(w_in=P2) == INVALID                                                             # nowhere to write
    assert f(w_in=P2, w_out=P2 + 4) == INVALID                                               # shifted onto itself
    assert f(w_out=P2, decay=float("nan")) == INVALID
    assert f(n=need - 1) == WORKSPACE


def test_sparse_decode_validation(msa):
    need = msa.lib.msa_sparse_decode_kv4_workspace_size(4, 1024, 8, 2, 128, 4)
    assert need > msa.lib.msa_kv4_decode_workspace_size(4, 8)
    assert msa.lib.msa_sparse_decode_kv4_workspace_size(4, 1024, 8, 2, 128, 0) == 0
    f = caller(msa.lib.msa_sparse_decode_kv4, ["cache", "q", "q_idx", "k_idx", "lens", "H_q", "d_idx", "B_k", "k", "w_in", "w_out",
                                               "decay", "out", "lse", "sel", "ws", "n", "stream"],
               [cache(msa), P2, P2, P2, P2, 8, 64, 128, 4, None, None, 1.0, P2, None, None, WS, need, None])
    assert f(q_idx=None) == INVALID and f(k_idx=None) == INVALID and f(q_idx=P2 + 8) == INVALID and f(sel=P2 + 1) == INVALID
    assert f(k=0) == INVALID and f(d_idx=0) == INVALID
    assert f(k=17) == UNSUPPORTED and f(B_k=64) == UNSUPPORTED and f(d_idx=48) == UNSUPPORTED
    wide = cache(msa, H_kv=4)
    assert f(cache=wide, d_idx=128) == UNSUPPORTED                                            # a row of index keys over 512 bytes
    assert f(cache=cache(msa, H_kv=3), H_q=6) == UNSUPPORTED
    assert f(n=need - 1) == WORKSPACE


def test_evict_validation(msa):
    other = cache(msa, base=0x50_0000_0000, L_max=256)
    need = msa.lib.msa_kv4_evict_workspace_size(4, 2, 100)
    f = caller(msa.lib.msa_kv4_evict, ["cache", "to", "w", "lens", "keep", "recent", "first", "k_idx", "k_idx_to", "d_idx", "w_to",
                                       "lens_to", "kept", "ws", "n", "stream"],
               [cache(msa), other, P2, P2 + BIG, 100, 10, 4, None, None, 0, None, WS + 4096, WS + 8192, WS, need, None])
    assert f(w=None) == INVALID and f(lens=None) == INVALID and f(lens_to=None) == INVALID and f(kept=None) == INVALID
    assert f(keep=0) == INVALID and f(recent=-1) == INVALID and f(first=-1) == INVALID
    assert f(recent=97) == INVALID and f(recent=2 ** 31 - 1, first=2 ** 31 - 1) == INVALID    # recent + first > keep
    assert f(keep=257) == INVALID                                                             # more than `to` holds
    for kw in (dict(B=3), dict(H_kv=1), dict(d_h=64), dict(k_scale=2.0), dict(v_scale=2.0)):
        assert f(to=cache(msa, base=0x50_0000_0000, **kw)) == INVALID, kw
    assert f(to=cache(msa)) == INVALID and f(to=cache(msa, base=P + 16)) == INVALID           # the same rows
    assert f(k_idx=P2) == INVALID and f(k_idx_to=P2) == INVALID and f(k_idx=P2, k_idx_to=P2 + BIG, d_idx=0) == INVALID
    assert f(k_idx=P2, k_idx_to=P2 + 2 * BIG, d_idx=48) == UNSUPPORTED
    assert f(w_to=P2) == INVALID and f(lens_to=P2 + BIG) == INVALID and f(k_idx=P2, k_idx_to=P2, d_idx=64) == INVALID
    assert f(n=need - 1) == WORKSPACE


@pytest.mark.parametrize("name", ["msa_kv4_append", "msa_kv4_read", "msa_kv4_decode", "msa_sparse_decode_kv4", "msa_kv4_evict"])
def test_fault_injection(msa, name):
    """MSA_FAULT_INJECT=<entry point> makes that call fail as a launch failure would, before enqueueing."""
    calls = {"msa_kv4_append": "(c, P2, P2, 256, 256, 4, P2, None, WS, BIG, None)",
             "msa_kv4_read": "(c, P2, P2, 4, P2, None, WS, BIG, None)",
             "msa_kv4_decode": "(c, P2, P2, 8, None, 0, None, None, 1.0, P2, None, WS, BIG, None)",
             "msa_sparse_decode_kv4": "(c, P2, P2, P2, P2, 8, 64, 128, 4, None, None, 1.0, P2, None, None, WS, BIG, None)",
             "msa_kv4_evict": "(c, o, P2, P2 + BIG, 8, 0, 0, None, None, 0, None, WS + 512, WS + 1024, WS, BIG, None)"}
    code = ("import sys, ctypes; sys.path.insert(0, %r)\n"
            "import block_sparse_long_idx_b200 as m\n"
            "m.lib\n"
            "P, P2, WS, BIG = %d, %d, %d, %d\n"
            "def mk(x): return ctypes.byref(m.api.msa_kv4_cache(x, x + (1 << 30), x + (2 << 30), x + (3 << 30), 4, 2, 128, 1024, 1.0, 1.0))\n"
            "c, o = mk(P), mk(5 << 36)\n"
            "print('STATUS', m.lib.%s%s)\n" % (ROOT, P, P2, WS, BIG, name, calls[name]))
    out = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, MSA_FAULT_INJECT=name), capture_output=True, text=True,
                         timeout=300)
    assert "STATUS 4" in out.stdout, out.stdout + out.stderr


def test_binding_checks_tensors(msa):
    """Tensors of the wrong kind are refused by name before anything is called (CPU tensors here)."""
    torch = pytest.importorskip("torch")
    u8 = torch.zeros((1, 2, 128, 64), dtype=torch.uint8)
    s = torch.zeros((1, 2, 128, 8), dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_codes"):
        msa.KV4Cache(u8, s, u8, s)                       # not on a GPU
    with pytest.raises(ValueError, match="B, H_kv, L_max"):
        msa.KV4Cache(u8[0], s, u8, s)


def test_reference_format():
    """The reference's own format: the E4M3 table, every code a fixed point, ties and saturation by hand."""
    assert np.nanmax(ref.E4M3) == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[0x38] == 1.0 and np.isnan(ref.E4M3[127])
    x = np.zeros((1, 16), np.float32)
    x[0, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]
    x[0, 8:] = -x[0, :8]
    c, s = ref.quantise(x, 1.0)
    assert s[0, 0] == 0x38                                # scale 1: ties go to the even codes
    assert ref.values(c, s, 1.0)[0, :8].tolist() == [6, 4, 4, 2, 2, 1, 1, 0]
    c2, s2 = ref.quantise(ref.values(c, s, 1.0), 1.0)
    assert np.array_equal(ref.values(c2, s2, 1.0), ref.values(c, s, 1.0))
    c, s = ref.quantise(np.full((1, 16), 1e6, np.float32), 1.0)
    assert s[0, 0] == 0x7E and (ref.values(c, s, 1.0) == 2688).all()
    assert (ref.quantise(np.full((1, 16), 0.005, np.float32), 1.0)[1] == 0).all()
    w = np.array([1, 3, 3, 2, 3, 0, 9, 1], np.float32)
    assert ref.keep_positions(w, 8, 4, 1, 1).tolist() == [0, 1, 6, 7] and ref.keep_positions(w, 3, 4, 1, 1).tolist() == [0, 1, 2]
