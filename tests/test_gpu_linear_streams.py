"""A plan's workspace whose memory work on another stream is still writing: a run waits for it.
The outputs are compared bit for bit with those of an undisturbed run."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

df11 = pytest.importorskip("huffman_decode_df11_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def _weight_and_input(tokens):
    w = workloads.gaussian_bf16(512 * 768, 0.05, 1).view(torch.bfloat16).view(512, 768)
    x = workloads.gaussian_bf16(tokens * 768, 1.0, 2).view(torch.bfloat16).view(tokens, 768)
    return df11.compress_linear(w.cuda()), x.cuda()


def _busy(nbytes):
    """A block of the allocator's that this stream has still to write, and has given back."""
    torch.cuda._sleep(100_000_000)  # some 50 ms
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    block.fill_(255)
    return block.data_ptr()


@pytest.mark.parametrize("tokens", [5, 50])
@pytest.mark.parametrize("captured", [False, True])
def test_a_run_on_another_stream_waits_for_the_workspaces_memory(tokens, captured):
    d, x = _weight_and_input(tokens)
    want, = df11.decode_linear([d], [x], out_dtype=torch.float32)
    y = torch.zeros(tokens, 512, device="cuda")
    nbytes = df11.LinearPlan([d], [x], [y]).workspace_bytes + 256
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    at = _busy(nbytes)
    plan = df11.LinearPlan([d], [x], [y])
    shared = plan._work.data_ptr() - at
    with torch.cuda.stream(side):
        if captured:
            graph.capture_begin(capture_error_mode="thread_local")
            plan.run()
            graph.capture_end()
            graph.replay()
        else:
            plan.run()
    torch.cuda.synchronize()
    assert 0 <= shared < 256  # the block is the workspace, or this shows nothing
    assert torch.equal(y, want)
    graph.reset()


def test_plans_made_in_a_capture_run_there_and_after_it():
    d, x = _weight_and_input(40)
    want, = df11.decode_linear([d], [x], out_dtype=torch.float32)
    ys = [torch.zeros(40, 512, device="cuda") for _ in range(2)]
    side, fork, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        plans = [df11.LinearPlan([d], [x], [y]) for y in ys]
        plans[0].run()
        fork.wait_stream(side)
        plans[1].run(stream=fork)
        side.wait_stream(fork)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want) and torch.equal(ys[1], want)
    ys[0].zero_()
    plans[0].run()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want)
    graph.reset()
