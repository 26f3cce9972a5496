"""What a user's program does around the serving calls: tables that are copied and pickled, empty steps,
batches without own keys or prefixes, workspaces that are views, and native bindings that a change of
torch has made stale."""
import copy
import ctypes
import gc
import pickle

import pytest
import torch

import exact_attention_25_gb300 as fa

gpu = pytest.mark.gpu


# ------------------------------------------------------------------------------ copies of a rope table

def behind(table):
    """What lies at the addresses that every call of rope passes."""
    freq, axis = table._args[:2]
    n = table.pairs
    return (tuple((ctypes.c_double * n).from_address(freq)), tuple((ctypes.c_int * n).from_address(axis)))


def _layer():
    m = torch.nn.Module()
    m.table = fa.RopeTable(64, [0.5 ** i for i in range(16)], [0] * 8 + [1] * 8, True)
    return m


@pytest.mark.parametrize("again", [lambda t: copy.deepcopy(t), lambda t: copy.copy(t),
                                   lambda t: pickle.loads(pickle.dumps(t)),
                                   lambda t: copy.deepcopy({"layers": [t, t]})["layers"][1]],
                         ids=["deepcopy", "copy", "pickle", "nested"])
def test_copies_of_a_table_own_what_they_pass(again):
    t = fa.RopeTable(64, [0.5 ** i for i in range(16)], [0] * 8 + [1] * 8, True)
    want, first = (t.inv_freq, t.axis), t._args[:2]
    u = again(t)
    # not the first table's arrays, unless it holds them itself
    assert not set(u._args[:2]) & set(first) or u._freq is t._freq
    del t
    gc.collect()
    # what the allocator would give the arrays' memory to next
    other = [(ctypes.c_double * 16)(*[7.0] * 16) for _ in range(64)]
    assert behind(u) == want == (u.inv_freq, u.axis)
    assert (u.d, u.pairs, u.axes, u.interleaved) == (64, 16, 2, True) and u._args[2:] == (2, 64, 16, True)
    del other


def test_a_copied_module_keeps_its_table():
    m = _layer()
    n = copy.deepcopy(m)
    assert n.table._args[0] != m.table._args[0]
    del m
    gc.collect()
    assert behind(n.table) == (n.table.inv_freq, n.table.axis)


# ------------------------------------------------------------------------------ workspaces that are views

i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731


@pytest.mark.parametrize("call", ["cache", "shared"])
def test_a_workspace_with_gaps_is_refused(call):
    """The kernels write the workspace as one run of bytes: a view with gaps would have what lies in them
    overwritten."""
    ws = torch.zeros(64, 2, 1024, dtype=torch.uint8)[:, 0]
    assert not ws.is_contiguous()
    q, kv = torch.zeros(2, 4, 64).bfloat16(), torch.zeros(9, 2, 64).bfloat16()
    with pytest.raises(ValueError, match="workspace"):
        if call == "cache":
            fa.fa_fwd_decode_cache(q, fa.new_cache(2, 16, 2, 64, device="cpu"), q.clone(), None, i32(0, 1, 2),
                                   i32(3, 4), torch.zeros(2, 1, dtype=torch.int32), 1, 9, 0.1, False, 2, ws)
        else:
            fa.fa_fwd_decode_shared(q, kv, kv, kv, kv, q.clone(), None, i32(0, 1, 2), i32(0, 4, 9), i32(0, 2),
                                    i32(0, 9), 1, 5, 2, 9, 0.1, False, 2, ws)
