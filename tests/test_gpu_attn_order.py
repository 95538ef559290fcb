"""The attention half's calls in stream order: arrays that the kernel directly before a call writes
(weights, scales and rotation tables as much as activations) are read as it leaves them, however long
it runs and however early it lets the call's kernel start."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import top_routing_grouped_router_gb300 as moe  # noqa: E402
from attn_ref import make_batch  # noqa: E402
from test_gpu_attn import NORMAL, UNIFORM, Dev  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_routing_grouped_router_gb300 import build
    build.build()


class Writer:
    """A kernel of milliseconds on two blocks that lets its successor start at once and writes `target`
    (8 bf16 or fp32 values, 16-byte aligned) at its end: a 4-bit linear of one row and very many inputs."""
    K = 1 << 21

    def __init__(self, target, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        codes = torch.randint(0, 256, (8, self.K // 2), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.rand(8, self.K // 16, generator=g, device="cuda").add_(0.5).bfloat16()
        self.x = torch.zeros(1, self.K, dtype=torch.bfloat16, device="cuda")
        self.x[0, :8] = 1.0
        self.shape = moe.make_q4_linear_shape(1, self.K, 8, "bf16" if target.dtype == torch.bfloat16 else "f32", 16)
        self.weight, self.out = moe.make_q4_weight(codes, scales, NORMAL), target.view(1, 8)

    def __call__(self):
        moe.moe_q4_linear(self.shape, self.x, self.weight, self.out)


def _reads_what_was_written(target, call, result, graph):
    """`call` right after a Writer of `target` gives what it gives once the writer has ended."""
    old, write = target.clone(), Writer(target)
    call()  # every first launch behind us
    stale = result().clone()
    write()
    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    want = result().clone()
    assert not torch.equal(want, stale)  # what is written shows in the result
    run = lambda: (write(), call())  # noqa: E731
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(3):
        target.copy_(old)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert torch.equal(result(), want)


# one and two strips a warp, inputs split over a cluster, a general codebook, blocks of 32, the
# tensor-core kernel alone and over a cluster, other block sizes
Q4 = [(1, 2048, 640, 64, UNIFORM), (8, 512, 20001, 64, UNIFORM), (1, 8192, 64, 64, UNIFORM), (3, 512, 300, 64, NORMAL),
      (16, 256, 20000, 32, NORMAL), (33, 2048, 20000, 64, UNIFORM), (20, 4096, 2112, 128, UNIFORM), (2, 96, 50, 16, UNIFORM)]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("what", ["scales", "codes", "x", "residual"])
@pytest.mark.parametrize("T,K,N,q_block,book", Q4)
def test_q4_linear_reads_what_the_kernel_before_wrote(T, K, N, q_block, book, what, graph):
    g = torch.Generator(device="cuda")
    g.manual_seed(K + N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(N, K // q_block, generator=g, device="cuda").add_(8.0).bfloat16()
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    res = torch.randn(T, N, generator=g, device="cuda").bfloat16()
    out = torch.empty(T, N, device="cuda")
    shape, weight = moe.make_q4_linear_shape(T, K, N, "f32", q_block), moe.make_q4_weight(codes, scales, book)
    target = {"scales": scales.view(-1), "codes": codes.view(torch.bfloat16).view(-1), "x": x.view(-1),
              "residual": res.view(-1)}[what][:8]
    _reads_what_was_written(target, lambda: moe.moe_q4_linear(shape, x, weight, out, residual=res), lambda: out, graph)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("tokens", [3, 700])
@pytest.mark.parametrize("what", ["turns", "gamma", "q"])
def test_rope_append_reads_what_the_kernel_before_wrote(what, tokens, graph):
    d = Dev(make_batch("bf16", 4, 2, 64, 16, [tokens], [tokens], seed=1, fill=5.0))
    gamma = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    rope = moe.make_rope(64, q_gamma=gamma)
    x = torch.randn(tokens, 4, 64, device="cuda").bfloat16()
    k, v = x[:, :2].contiguous(), x[:, 2:].contiguous()
    target = {"turns": rope.tensors[0].view(torch.float32)[:8], "gamma": gamma[:8], "q": x.view(-1)[:8]}[what]
    _reads_what_was_written(target, lambda: moe.moe_rope_append(d.shape, rope, x, k, v, d.cache, d.batch, d.out,
                                                                workspace=d.ws), lambda: d.out, graph)


@pytest.mark.parametrize("T,K,N", [(33, 2048, 20000), (20, 4096, 2112)])
def test_q4_linear_wait_limit_starts_after_the_kernel_before(T, K, N):
    # the waits of the tensor-core kernel are limited in time; the time that the kernel before it still
    # runs does not count
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(N, K // 64, generator=g, device="cuda").add_(0.5).bfloat16()
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    out, want = (torch.empty(T, N, device="cuda") for _ in range(2))
    shape, weight = moe.make_q4_linear_shape(T, K, N, "f32"), moe.make_q4_weight(codes, scales, UNIFORM)
    write = Writer(x.view(-1)[:8])
    for _ in range(2):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        write()
        end.record()
    moe.moe_q4_linear(shape, x, weight, want)
    torch.cuda.synchronize()
    limit = int(start.elapsed_time(end) * 1e6) // 4
    assert limit > 300_000  # ns: far above any wait of the call itself
    moe.moe_debug_set_waits(limit)
    try:
        for _ in range(3):
            write()
            moe.moe_q4_linear(shape, x, weight, out)
            assert moe.moe_q4_linear_read_error() == 0
            assert torch.equal(out, want)
            out.zero_()
    finally:
        moe.moe_debug_set_waits()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("dtype,dim,tokens", [("bf16", 64, 1), ("bf16", 128, 40), ("bf16", 96, 40), ("f32", 64, 2)])
def test_attention_reads_what_the_kernel_before_wrote(dtype, dim, tokens, what, graph):
    d = Dev(make_batch(dtype, 4, 1, dim, 16, [tokens], [tokens + 8], seed=1, fill=0.5))
    target = {"q": d.q.view(-1), "k": d.k[d.table[0, 0]].view(-1), "v": d.v[d.table[0, 0]].view(-1)}[what][:8]
    call = lambda: moe.moe_paged_attention(d.shape, d.q, d.cache, d.batch, d.out, scale=0.1, workspace=d.ws)  # noqa: E731
    _reads_what_was_written(target, call, lambda: d.out, graph)
