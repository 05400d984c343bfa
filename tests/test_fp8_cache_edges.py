"""The 8-bit paged KV cache on the CPU: refusals at the far ends of the arguments' ranges."""

import pytest
import torch

import attention_forward_09_gb300 as gb
from test_fp8_cache import _args, lib  # noqa: F401


@pytest.mark.parametrize("dtype", [torch.float32, torch.uint8, torch.int64, torch.bfloat16])
def test_status_word_of_another_type_is_refused(lib, dtype):  # noqa: F811
    """Bits set in a float32 word would read as 0."""
    a, status = _args(), torch.zeros(1, dtype=dtype)
    table, cu = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: gb.attn_kv_cache_write_fp8(a["key"], a["value"], a["slots"], a["cache"], a["scales"], dev_status=status),
                 lambda: gb.attn_kv_cache_read_fp8(a["cache"], a["scales"], table, cu, 10, dev_status=status),
                 lambda: gb.attn_fwd_paged_fp8(q, a["cache"], a["scales"], table, cu[:1], 256, dev_status=status)):
        with pytest.raises(ValueError, match="dev_status"):
            call()
