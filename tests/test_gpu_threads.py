"""Calls from other host threads than the one that has used the GPU: a thread's first
call, and two threads' calls at once."""
import threading

import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from test_gpu_latent import Case
from test_gpu_steps import Step

pytestmark = pytest.mark.gpu


def at_once(*loops):
    """Runs the loops in threads that begin together; what they raised."""
    begin, raised = threading.Barrier(len(loops)), []

    def work(loop):
        begin.wait()
        try:
            loop()
        except Exception as e:  # (of a thread: shown by the caller)
            raised.append(e)

    threads = [threading.Thread(target=work, args=(loop,)) for loop in loops]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return raised


def test_the_first_call_of_a_thread(cuda_lib):
    """A new thread has no context of its own until a call binds one."""
    maps, attn = Step([5, 64], [1, 3], 64, 4, range(9)), Case([2, 1], [300, 64], 16, 64)
    maps_args, ws, stream = maps.d, attn.run(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    attn.fresh()
    args = attn.args()
    assert not at_once(lambda: B.dsa_step_maps(stream=stream, **maps_args))
    assert not at_once(lambda: B.dsa_latent_attn(args, ws, stream))
    errors = []
    assert not at_once(lambda: errors.append(B.device_error()))
    assert errors == [0]
    maps.check()
    attn.check()


@pytest.mark.parametrize("sizes", [(4096, 2600), (8192, 4200), (1100, 4096, 2600, 8192)])
def test_step_maps_of_different_sizes(sizes, cuda_lib):
    """Requests whose running sums take different amounts of shared memory of the same
    kernel (64 KB and 41, 128 and 66).  The packed blocks keep the threads inside the
    library for most of the time."""
    steps = []
    for n in sizes:
        rng = np.random.default_rng(n)
        steps.append(Step(rng.integers(0, 64, n), np.arange(n) < 20, 64, 2, rng.permutation(2 * n), seed=n))
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    refused = [0] * len(sizes)

    def loop(i):
        s, d, stream = steps[i], steps[i].d, streams[i].cuda_stream
        args = B._STEP_MAPS.pack(sizes[i], s.T, s.bs, 2, 2 * sizes[i], *[0 if d[k] is None else d[k].data_ptr() for k in (
            "cached", "fresh", "free_pages", "free_head", "block_table", "cu_tokens", "kv_len", "counts", "seq_of_token",
            "pos", "slot")])

        def calls():
            for _ in range(5000):
                refused[i] += cuda_lib.step_maps_packed(args, stream) != 0
        return calls

    assert not at_once(*[loop(i) for i in range(len(sizes))])
    torch.cuda.synchronize()
    assert refused == [0] * len(sizes)
    for s in steps:
        s.check()
