"""Which form of its down product the layer for one token takes, told from the
workspace it asks for (no GPU needed): h, and the sums of the form with shared
rows, one set a part."""
import ctypes

import pytest
import torch

from tests import few_cases


@pytest.mark.parametrize("dtype,wdtype", few_cases.TYPES)
def test_one_token(dtype, wdtype):
    from combine_symmetric_memory_amd import _capi
    i8 = wdtype == torch.int8
    code = {few_cases.BF: _capi.CCO_BF16, few_cases.FP: _capi.CCO_F16}[dtype]
    for T, H, I, E, K, parts in few_cases.one_token(wdtype):
        assert T == 1
        d = _capi.cco_few_desc(H, I, E, K, code, _capi.CCO_I8 if i8 else code, 16, 16,
                               16 if i8 else None, 16 if i8 else None)
        h = T * K * 2 * ((I + 255) // 256 * 256) * 2
        # (one part needs no sums, and would not be told from none)
        assert parts != 1
        assert _capi.lib.cco_moe_few_workspace(ctypes.byref(d), T) == h + parts * T * H * 4, \
            (T, H, I, E, K)
