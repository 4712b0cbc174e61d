"""The operators around the layer called by several host threads at a time, each on
its own stream with its own sizes: no call is refused, and the results are those of
the same calls alone.  The C entries are called directly, so that the threads are in
the library at the same time (Python's lock is held for a few hundred nanoseconds
between calls)."""
import ctypes
import threading
import time

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_ffn_forward_b200 import block, moe  # noqa: E402

CALLS = 5000


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_ffn_forward_b200 import build
    build.build()
    yield
    block.check()


def together(calls):
    """calls: (function of a stream that returns a status, output, the same of the call alone)."""
    start = threading.Barrier(len(calls))
    streams = [torch.cuda.Stream() for _ in calls]
    statuses = [set() for _ in calls]
    torch.cuda.synchronize()

    def loop(i):
        call, stream, seen = calls[i][0], streams[i].cuda_stream, statuses[i]
        start.wait()
        for _ in range(CALLS):
            seen.add(call(stream))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(s == {moe.MOE_OK} for s in statuses), statuses
    assert all(torch.equal(out, want) for _, out, want in calls)


def norm_call(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    h, y, post, pre = r(rows, cols), r(rows, cols), r(cols), r(cols)
    want = block.block_norm_forward(h, y, post, None, 0.7, pre)[1]
    a = block._norm_args(h, y, post, None, 0.7, pre, 1e-6)[0]
    out, nxt = torch.empty_like(h), torch.empty_like(h)
    a.out, a.next = out.data_ptr(), nxt.data_ptr()
    keep, fn = (h, y, post, pre, out), moe.lib().moe_block_norm
    return (lambda stream, ref=ctypes.byref(a), keep=keep: fn(ref, stream)), nxt, want


def test_norms_of_several_widths():
    """One kernel for all widths, with up to eight times the shared memory for the widest."""
    together([norm_call(300, cols, cols) for cols in (4096, 1024, 2048, 520, 4096, 1024)])


def balance_call(tokens, experts, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((tokens, experts), generator=g, device="cuda")
    ids = torch.topk(logits, 4, 1).indices.int()
    want, counts, slope = block.balance_loss_forward(logits, ids, 0.01, 0)
    loss = torch.empty_like(want)
    size = moe.moe_balance_workspace(tokens, experts, 1)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    keep, fn = (logits, ids, counts, slope, work), moe.lib().moe_balance_loss
    args = (logits.data_ptr(), experts, ids.data_ptr(), tokens, experts, 4, 0, None, 1, None, 0.01, loss.data_ptr(),
            counts.data_ptr(), slope.data_ptr(), work.data_ptr(), size)
    return (lambda stream, keep=keep: fn(*args, stream)), loss, want


def test_balance_losses_of_several_widths():
    """One kernel from 513 experts on, which above 722 needs more shared memory than a kernel has unasked."""
    together([balance_call(64, experts, experts) for experts in (1024, 640, 700, 1024, 640, 900)])


def test_calls_do_not_wait_for_the_expert_cache():
    """While another thread holds the cache (here: for as long as a GPU of 1.5 s of work takes, which a new cache size
    waits for), the operators are launched and counted all the same."""
    import dataclasses
    from routed_expert_ffn_forward_b200 import synth
    from routed_expert_ffn_forward_b200.layer import layer_from_config
    moe.moe_set_cache_bytes(1 << 20)
    L = layer_from_config(dataclasses.replace(synth.TINY, seed=3))   # streamed: the cache is there
    try:
        x = torch.randn((4, 256), device="cuda")
        block.mx_quantize(x)
        torch.cuda.synchronize()
        before = moe.moe_get_stats()["launches"]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            torch.cuda._sleep(int(1.5e9 * 1.9))
        holder = threading.Thread(target=moe.moe_set_cache_bytes, args=(1 << 20,))
        holder.start()
        time.sleep(0.2)
        t = time.perf_counter()
        for _ in range(10):
            block.mx_quantize(x)
        took = time.perf_counter() - t
        waiting = holder.is_alive()
        holder.join()
        assert waiting and took < 0.5, (waiting, took)
        assert moe.moe_get_stats()["launches"] == before + 10
    finally:
        L.destroy()
        moe.moe_set_cache_bytes(moe.SIZE_MAX)
