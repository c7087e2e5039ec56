"""Which row keeps a partial page in a fork."""
import numpy as np
import pytest
import torch

from sparse_entmax_kv_b200 import native as nv, pages


@pytest.mark.gpu
@pytest.mark.parametrize("parent,keeper", [([1, 1, -1], 1), ([2, 2, 2], 2), ([2, 2, -1], 0), ([-1, 0, 0], 1)])
def test_the_row_that_keeps_a_partial_page(parent, keeper):
    """The parent's own row where it continues, however many rows before it do; else the first that does."""
    shape = nv.Shape(3, 1, 1, 64, 16, 2, 9)
    table = torch.tensor([[8, 3], [2, 7], [5, 0]], dtype=torch.int32, device="cuda")
    lens = torch.full((3,), 20, dtype=torch.int32, device="cuda")
    pool = torch.arange(9, device="cuda", dtype=torch.int16)[:, None].repeat(1, 16 * 64)
    t_out, l_out = torch.empty_like(table), torch.empty_like(lens)
    pages.entmaxkv_pages_fork(shape, torch.tensor(parent, dtype=torch.int32, device="cuda"), table, lens, t_out, l_out,
                              pages.Buffers([pool]), workspace=pages.alloc_workspace(shape, "cuda"))
    new = [1, 4, 6]  # the free blocks, handed out in the order of the rows
    want = np.full((3, 2), -1, np.int32)
    for b, p in enumerate(parent):
        if p >= 0:
            want[b] = table[p].cpu().numpy()
            if b != keeper:
                want[b, 1] = new.pop(0)
                assert (pool[want[b, 1]] == table[p, 1]).all()
    np.testing.assert_array_equal(t_out.cpu().numpy(), want)
    assert l_out.tolist() == [20 if p >= 0 else 0 for p in parent] and nv.get_status() == 0
