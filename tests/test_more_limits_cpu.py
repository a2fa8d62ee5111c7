"""The ends of the ranges of the step maps and the latent attention, without a GPU:
sizes whose index arithmetic would leave 32 bits, and arrays over one another, are
refused before anything is launched."""
import pytest

from sparse_attention_prolog_gb300 import binding as B
from test_abi_cpu import lib  # noqa: F401
from test_more_operators_cpu import BASE, INVALID, UNSUPPORTED, _with

FAR = 1 << 40  # apart from all else by more than the largest array here


@pytest.mark.parametrize("name", ["T", "n_free"])
def test_step_maps_leave_room_for_a_stride(lib, name):  # noqa: F811
    a = B.StepMapsArgs(4, 16, 64, 32, 100, *[BASE + i * FAR for i in range(11)])
    for n in (2 ** 31 - 2 ** 20 + 1, 2 ** 31 - 1):
        assert lib.dsa_step_maps(_with(a, **{name: n}), None) == UNSUPPORTED, n
    # (the largest is only looked at: something else is wrong with the call)
    assert lib.dsa_step_maps(_with(a, slot=a.slot + 4, **{name: 2 ** 31 - 2 ** 20}), None) == INVALID
