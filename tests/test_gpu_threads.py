"""Calls from other host threads than the one that has used the GPU: a thread's first
call, and two threads' calls at once."""
import threading

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
