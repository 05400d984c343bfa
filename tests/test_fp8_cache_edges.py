"""The 8-bit paged KV cache on the CPU: refusals at the far ends of the arguments' ranges."""

import pytest
import torch

import attention_forward_09_gb300 as gb
from test_fp8_cache import INVALID, UNSUPPORTED, P, _args, lib, paged  # noqa: F401


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


def test_sizes_at_the_ends_of_their_types(lib):  # noqa: F811
    """Refused before the plan's arithmetic, which counts heads in 32 bits."""
    most = 2 ** 31 - 1
    size = lib.attn_fwd_paged_fp8_workspace_size
    for hq, hkv in ((65536, 1), (65536, 65536), (most, 1), (most, most), (2 ** 30, 2)):
        for s, n in ((1, 100), (most, most)):
            assert size(s, hq, hkv, 64, n) == 0
        assert paged(lib, Hq=hq, Hkv=hkv, S=1, maxlen=100, D=64, ws=None, wsb=0) == UNSUPPORTED
    for hq, hkv in ((65535, 1), (65535, 65535), (8, 1)):
        for s in (1, most):
            size(s, hq, hkv, 64, most)
    assert paged(lib, S=most, maxlen=most, maxb=most, qs=2 ** 40) == UNSUPPORTED  # units of work past 32 bits


def test_null_arrays_are_for_no_sequences_only(lib):  # noqa: F811
    none = dict(q=None, bt=None, sl=None, out=None, ws=None, wsb=0, maxb=0)
    assert paged(lib, S=0, **none) == 0
    for name in ("q", "bt", "sl", "out"):
        assert paged(lib, S=1, **{name: None}) == INVALID
    assert paged(lib, S=0, cache=None) == INVALID and paged(lib, S=0, D=80, **none) == UNSUPPORTED
    bf16 = lambda s, q, bt, sl, out: lib.attn_fwd_paged(q, P, 16, 128, bt, 0 if bt is None else 4, sl, s, 512, 8, 2, 128, 0.1, 1, out, 1,  # noqa: E731
                                                        None, None, 0, None, None)
    assert bf16(0, None, None, None, None) == 0
    for i in range(4):
        arrays = [P] * 4
        arrays[i] = None
        assert bf16(1, *arrays) == INVALID
