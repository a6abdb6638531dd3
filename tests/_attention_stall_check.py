"""Child process of test_gpu_attention_timeout.py: run with SPEC_VERIFY_TEST_STALL_ATTENTION=<row>
(read once by the library), so that every CTA of that batch row in the tcgen05 kernel waits
in vain for one tile's notes.  Checks that the row's real queries and their lse are NaN, that
what lies behind them is left alone, that every other row matches the plain form, and that
the next call works."""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from test_gpu_attention import case, check, run  # noqa: E402

SHAPES = [  # B, Q, Hq, H, D, page_size, ctx, tree, workspace
    (3, 6, 8, 1, 128, 16, 900, False, "auto"),   # two stretches a CTA, splits joined
    (3, 6, 8, 1, 128, 24, 900, False, "auto"),   # rows copied without the copy engine
    (3, 6, 8, 1, 64, 16, 900, False, None),      # not split
    (3, 20, 4, 1, 128, 16, 300, True, "auto"),   # one stretch of 128 rows
    (3, 61, 4, 1, 128, 64, 2500, True, "auto"),  # two tiles of 128 rows, split
    (3, 61, 4, 1, 128, 16, 40, False, "auto"),
    (3, 40, 4, 1, 256, 16, 1500, True, "auto"),  # wide heads
    (3, 40, 4, 1, 256, 24, 100, False, "auto"),
    (3, 40, 4, 1, 128, 16, 0, False, "auto"),    # every tile holds new tokens
]


def main():
    import torch
    import speculative_decoding_verification_53_gb300 as sv
    stall = int(os.environ["SPEC_VERIFY_TEST_STALL_ATTENTION"])
    for cache in ("bf16", "e4m3"):
        for n, (B, Q, Hq, H, D, ps, ctx, tree, ws) in enumerate(SHAPES):
            c = list(case(np.random.default_rng([n, cache == "e4m3"]), B, Q, Hq, H, D, ps, ctx, cache, tree, False,
                          ragged=False))
            real = Q - 2
            c[7] = np.array(c[7])
            c[7][stall] = real
            q, k, v, ks, vs, table, base, new_len, mask = c
            others = [b for b in range(B) if b != stall]
            for rep in range(2):
                o, l = run(sv, c, workspace=ws)
                assert o[stall, :real].isnan().all() and l[stall, :real].isnan().all(), (cache, n)
                assert (o[stall, real:] == 5).all() and (l[stall, real:] == 6).all(), (cache, n)
                check(o[others], l[others], q[others], k, v, ks, vs, table[others], base[others], new_len[others],
                      None if mask is None else mask[others], D ** -0.5, 5.0, 6.0)
    # few query rows take the kernel without such waits
    c = case(np.random.default_rng(9), 2, 2, 4, 1, 128, 16, 300, "e4m3", False, False, ragged=False)
    o, l = run(sv, c)
    check(o, l, *c[:9], 128 ** -0.5, 5.0, 6.0)
    torch.cuda.synchronize()
    print("ok")


if __name__ == "__main__":
    main()
