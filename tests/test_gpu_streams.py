"""Calls on a stream of their own: what they allocate comes from that stream's memory, not from blocks that work still queued
on the current stream uses."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import block_sparse_long_idx_b200 as msa  # noqa: E402

N, B, H, G, D, DI, K, L = 512, 3, 2, 4, 128, 32, 3, 512


def make_calls():
    g = torch.Generator("cuda").manual_seed(1)

    def bf(*shape):
        return torch.randn(shape, device="cuda", generator=g).bfloat16()

    def small(*shape):
        return torch.randint(-3, 4, shape, device="cuda", generator=g).bfloat16()

    q, k, v, dout = bf(N, H * G, D), bf(N, H, D), bf(N, H, D), bf(N, H * G, D)
    q_idx, k_idx = small(N, H, DI), small(N, H, DI)
    sel = msa.msa_index_topk(q_idx, k_idx, 128, K)
    out, lse = msa.msa_sparse_prefill(q, k, v, sel)
    kv = msa.msa_build_kv2q(sel)
    q8, k8, v8 = (msa.msa_quantize_e4m3(t) for t in (q, k, v))
    lens = torch.tensor([500, 1, 300], dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(lens)
    kc, vc, ic = bf(B, L, H, D), bf(B, L, H, D), small(B, L, H, DI)
    c, to = msa.KV4Cache.empty(B, L, H, D), msa.KV4Cache.empty(B, L, H, D)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * L
    msa.msa_kv4_append(c, kc.view(B * L, H, D), vc.view(B * L, H, D), zero, cu)
    qd, qi = bf(B, H * G, D), small(B, H, DI)
    w = torch.rand((B, H, L), device="cuda", generator=g)

    def rows(x):
        return [x.codes, x.scales, x.rscales, x.blkmax]

    return {
        "index_topk": lambda s: [msa.msa_index_topk(q_idx, k_idx, 128, K, stream=s)],
        "build_kv2q": lambda s: [msa.msa_build_kv2q(sel, stream=s).offsets()],
        "prefill": lambda s: msa.msa_sparse_prefill(q, k, v, sel, stream=s),
        "varlen": lambda s: msa.msa_sparse_prefill_varlen(q, k, v, q_idx, k_idx, [0, 200, N], 128, K, stream=s),
        "backward": lambda s: msa.msa_sparse_backward(q, k, v, out, lse, dout, sel, kv, q_idx=q_idx, k_idx=k_idx, stream=s),
        "quantize": lambda s: rows(msa.msa_quantize_e4m3(q, stream=s)),
        "prefill_fp8": lambda s: msa.msa_sparse_prefill_fp8(q8, k8, v8, sel, stream=s),
        "decode": lambda s: msa.msa_sparse_decode(qd, qi, kc, vc, ic, lens, 128, K, stream=s),
        "kv4_read": lambda s: msa.msa_kv4_read(c, zero, cu, B * L, stream=s),
        "kv4_decode": lambda s: msa.msa_kv4_decode(qd, c, lens, stream=s),
        "decode_kv4": lambda s: msa.msa_sparse_decode_kv4(qd, qi, c, ic, lens, 128, K, stream=s),
        "kv4_evict": lambda s: msa.msa_kv4_evict(c, to, w, lens, 200, stream=s),
    }


def stream_of(t):
    """The stream whose pool holds the tensor's memory."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_allocations_belong_to_the_given_stream(raw, monkeypatch):
    calls = make_calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    taken = []
    real = msa.api._workspace
    monkeypatch.setattr(msa.api, "_workspace", lambda *a: taken.append(real(*a)) or taken[-1])
    for name, call in calls.items():
        taken.clear()
        got = list(call(side.cuda_stream if raw else side)) + taken
        for t in got:
            assert stream_of(t) == side.cuda_stream, name
        here = list(call(torch.cuda.current_stream()))
        for t in here:
            assert stream_of(t) == torch.cuda.current_stream().cuda_stream, name
    torch.cuda.synchronize()


def test_freed_memory_of_the_current_stream_is_not_taken():
    """Work that waits on the current stream and writes to tensors that the program has let go of, then calls elsewhere."""
    calls = make_calls()
    want = {n: [t.clone() for t in f(None)] for n, f in calls.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = {}
    for name, call in calls.items():
        like = [torch.empty_like(t) for t in want[name]]
        torch.cuda._sleep(20_000_000)              # about 10 ms
        for t in like:
            t.view(torch.uint8).fill_(0x55)
        del like, t
        got[name] = list(call(side))
        side.synchronize()
    torch.cuda.synchronize()                       # the fills are done too
    for name in calls:
        for x, y in zip(got[name], want[name]):
            if name == "backward":                 # its fp32 additions have no fixed order: not the fill, all the same
                assert (x.contiguous().view(torch.uint8) != 0x55).any(), name
            else:
                assert torch.equal(x, y), name


def test_given_stream_in_a_capture():
    """Calls on a stream that a capture has forked to are captured with it; the graph holds their memory over replays."""
    calls = {n: f for n, f in make_calls().items() if n not in ("varlen", "backward")}  # (host copies; unordered additions)
    want = {n: [t.clone() for t in f(None)] for n, f in calls.items()}
    side = torch.cuda.Stream()
    for f in calls.values():
        f(side)
    torch.cuda.synchronize()
    graph, got = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        for n, f in calls.items():
            got[n] = list(f(side))
        here.wait_stream(side)
    for _ in range(2):
        for v in got.values():
            for t in v:
                t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in calls:
            for x, y in zip(got[n], want[n]):
                assert torch.equal(x, y), n
