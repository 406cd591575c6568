"""GPU tests of what follows a wait that ran out (the testing hook: a wait on a barrier that nothing signals, 200 us)."""
import pytest
import torch

from tests.test_gpu_paged_runs import BF16, big, ints

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import paged


@pytest.mark.parametrize("what", ["decode", "chunk", "chunk in waves", "shared", "sparse"])
def test_calls_between_a_wait_that_ran_out_and_the_report(what):
    """They return; the bit stays until it is asked for; and what follows the report is right, calls and replays alike."""
    lens = [5000, 3000]
    heads, kv_heads = (24, 24) if "waves" in what else (8, 2)
    new = 300 if "chunk" in what else 1
    c, g = big(lens, heads, kv_heads, 128, BF16, 16, seed=41, bounds=True, max_tokens=2)
    q = torch.randn(2, new, heads, 128, device="cuda", generator=g).to(BF16)
    pages, plen = c.block_table[0, :300].clone(), ints([4800])
    if what == "shared":
        c.kv_len.fill_(4900)
        c.block_table[1, :300] = pages
        c.block_table[1, 300:307] = c.block_table[1, :7]
    run = {"shared": lambda: c.attend_shared(q, pages, plen, lse=True), "sparse": lambda: c.attend_sparse(q[:, 0], 60, lse=True)}.get(
        what, lambda: c.attend(q, lse=True, flags=paged.CAUSAL))
    want = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = run()
    assert c.get_error() == 0
    for _ in range(2):
        paged.kvc_paged_debug_stall_waits(c.handle, 200_000)
        run()
        paged.kvc_paged_debug_stall_waits(c.handle, 0)
        run()
        graph.replay()
        run()
        assert c.get_error() & paged.DEV_TIMEOUT
        assert c.get_error() == 0
        for x in replayed:
            x.fill_(7)
        graph.replay()
        got = run()
        assert c.get_error() == 0
        for x, y, z in zip(want, got, replayed):
            assert torch.equal(x, y) and torch.equal(x, z)
