"""The calls of the sparse path from two host threads at once (the binding releases the interpreter lock inside a
call): each thread on a stream and with memory of its own gets the bits of its call alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def draw(shape, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)


def at_once(*jobs):
    """Runs the jobs in threads of their own, started together; raises the first error."""
    errors, gate = [], threading.Barrier(len(jobs))

    def run(job):
        try:
            gate.wait(timeout=60)
            job()
        except BaseException as e:                # noqa: BLE001 (handed to the test's thread)
            errors.append(e)
    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("d", [64, 128])
def test_block_selection_at_two_lengths(d, cuda_dev):
    """Rows of 2 and of 640 blocks use one kernel with different amounts of shared memory."""
    from video_dit_quantized_b200 import sage, sparse

    def job(nT, seed):
        q, k = (draw((1, 1, nT * 128, d), s, cuda_dev) for s in (seed, seed + 1))
        keep = max(1, nT // 9)
        ref = [t.clone() for t in sparse.select_blocks(q, k, keep)]
        scratch = sparse.alloc_select_scratch(1, 1, nT * 128, d, cuda_dev)
        lists, counts = (torch.zeros_like(t) for t in ref)
        stream = torch.cuda.Stream()
        held = (q, k, scratch, lists, counts)

        def call():
            return sage.LIB.sage_select_blocks(held[0].data_ptr(), held[1].data_ptr(), 1, 1, nT * 128, d, keep, 0, 0,
                                               lists.data_ptr(), counts.data_ptr(), held[2].data_ptr(), held[2].numel(),
                                               stream.cuda_stream)

        def run():
            torch.cuda.set_device(cuda_dev)
            for _ in range(20):
                rcs = {call() for _ in range(250)}
                assert rcs == {sage.OK}, rcs
                stream.synchronize()
                assert torch.equal(lists, ref[0]) and torch.equal(counts, ref[1])
        return run
    jobs = [job(2, 1), job(640, 3)]
    torch.cuda.synchronize()
    at_once(*jobs)


def test_the_whole_path(cuda_dev):
    from video_dit_quantized_b200 import sparse

    def job(N, H, d, mode, seed):
        x = draw((1, N, 3, H, d), seed, cuda_dev)
        stream = torch.cuda.Stream()

        def layer():
            q, k = sparse.qk_norm_rope(x[:, :, 0], x[:, :, 1], norm=sparse.NORM_LAYER, scope=sparse.NORM_SCOPE_ALL, stream=stream)
            with torch.cuda.stream(stream):
                v = x[:, :, 2].permute(0, 2, 1, 3).contiguous()
            lists, counts = sparse.select_blocks(q, k, 4, stream=stream)
            return sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, stream=stream)
        torch.cuda.synchronize()
        ref = layer().clone()
        torch.cuda.synchronize()

        def run():
            torch.cuda.set_device(cuda_dev)
            for _ in range(40):
                got = layer()
                stream.synchronize()
                assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
        return run
    at_once(*[job(*a) for a in ((3000, 8, 128, 0, 5), (700, 20, 128, 1, 6), (5000, 6, 64, 2, 7), (129, 3, 64, 0, 8))])
