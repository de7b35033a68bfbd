"""The binding of the serving calls where something outside them goes wrong."""
import pytest
import torch

from block_sparse_compressed_gb300 import hca

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def test_a_call_without_memory_is_made_or_not_made():
    # Python's allocations fail one after the other: a plan that takes its blocks in
    # place was made once if it is answered, and not at all if it is declined or raises
    fail = pytest.importorskip("_testcapi")
    hca.load()
    if hca._py is None:
        pytest.skip("built without the headers of Python or torch")
    held, added, free = i32([0]), i32([40]), i32(list(range(8)))
    made = declined = 0
    for n in range(40):
        table, count = torch.full((1, 8), -1, dtype=torch.int32, device=DEV), i32([8])
        args = (held, added, table, free, count, 8, 16, 40, 1, None, None, count, None, True)
        r = None
        fail.set_nomemory(n, n + 1)
        try:
            r = hca._py.cache_plan(*args)
        except MemoryError:
            pass
        finally:
            fail.remove_mem_hooks()
        if r is None:
            declined += 1
            assert int(count) == 8 and bool((table == -1).all())
        else:
            made += 1
            assert int(count) == 5 and table[0].tolist() == [7, 6, 5, -1, -1, -1, -1, -1]
    assert made and declined
