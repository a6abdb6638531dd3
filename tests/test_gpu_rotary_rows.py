"""Rotary positions with the append where a batch row has more than 2^31 rows of heads: the sizes are limited each by
itself, not their product.  Tolerances are those of test_gpu_rotary.py."""
import numpy as np
import pytest

from oracle import context
from test_gpu_paged_kv import host, ints, sv, values  # noqa: F401
from test_gpu_rotary import close, reach

pytestmark = pytest.mark.gpu


def test_rows_of_heads_beyond_31_bits(sv):  # noqa: F811
    import torch
    N, HQ, D, ps = 33000, 65536, 2, 16
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((1, N, HQ, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    key, value = (torch.randn((1, N, 1, D), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    pages = (N + ps - 1) // ps + 1
    k, v = (torch.zeros((pages, 1, ps, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = ints(np.arange(pages)[None, ::-1])
    freq = torch.tensor([0.37], dtype=torch.float64, device="cuda")
    tokens = [0, 1, 16384, 32766, 32767, 32768, N - 1]  # 2^31 rows end with token 32767
    before = host(q[:, tokens])
    out = sv.spec_rotary_append(q, key, value, freq, k, v, table, ints([3]), out=q)
    pos = context.positions([3], N)
    close(host(out[:, tokens]), context.rotary(before, [0.37], pos[:, tokens]), reach(before, 1, False), "bf16")
    place = np.arange(3, 3 + N)
    got_k, got_v = (values(x)[(pages - 1) - place // ps, 0, place % ps] for x in (k, v))
    close(got_k, context.rotary(host(key), [0.37], pos)[0, :, 0], reach(host(key), 1, False)[0, :, 0], "bf16")
    assert np.array_equal(got_v, host(value)[0, :, 0])
