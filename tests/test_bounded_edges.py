"""Edges of the window and paged-cache calls: tensors that are not on a GPU, calls that are
refused half way, caches without a free page, rows whose softmax has no finite logit, and what
the attention weights may be off by."""
import pytest
import torch

from query_oriented_sparse_b200 import binding as Bd

BF, F32 = torch.bfloat16, torch.float32


# ---- tensors on the host ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_host_tensors_are_refused(dtype):
    """Every argument is right but for the device: refused before a kernel is given the pointers."""
    q, k, v = torch.zeros(1, 4, 8, 64, dtype=dtype), torch.zeros(1, 100, 64, dtype=dtype), torch.zeros(1, 100, 64, dtype=dtype)
    kp, vp, w = torch.zeros(6, 2, 16, 64, dtype=dtype), torch.zeros(6, 2, 16, 64, dtype=dtype), torch.zeros(6, 2, 16)
    table, lens = torch.arange(4, dtype=torch.int32)[None], torch.ones(1, dtype=torch.int32)
    rows = torch.zeros(1, 2, 3, 64, dtype=dtype)
    cache = Bd.PagedCache(1, 4, 2, 64, dtype, 6, 16, 4, "cpu", record=True)
    for call in (lambda: Bd.window_chunk_attn(q, k, v, (0, 100), (92,), 10),
                 lambda: Bd.window_chunk_attn(q[:, :, :1].contiguous(), k, v, (0, 100), (92,), 10),
                 lambda: Bd.paged_append(rows, rows.clone(), kp, vp, table, lens, weight_pages=w),
                 lambda: Bd.paged_decode_attn(q[:, :, :1].contiguous(), kp, vp, table, lens, 64, weight_pages=w),
                 lambda: Bd.paged_evict(kp, vp, w, table, lens, 64, lens, 8, table.clone()),
                 lambda: cache.append(rows, rows.clone()),
                 lambda: cache.attend(q[:, :, :1].contiguous())):
        with pytest.raises(Bd.QuokaError, match="not on a CUDA device") as e:
            call()
        assert e.value.status == Bd.QUOKA_ERR_INVALID_ARG
