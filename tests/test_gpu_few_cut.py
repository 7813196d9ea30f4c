"""The expert layer for a few tokens where an expert has more tokens than the
kernels take at a time: few pairs in all against the experts there are, but of
one or two experts (uneven routing, a shared expert as a further expert)."""

import numpy as np
import pytest
import torch

from test_gpu_few import DEV, MAKE, _bf, _check

pytestmark = pytest.mark.gpu

# T, H, I, E, k, tokens of expert 0, of expert 1, ...; the others choose among the rest
CASES = [("fp8", 5, 64, 32, 8, 1, (5,)), ("fp8", 8, 144, 48, 8, 1, (8,)), ("fp8", 9, 272, 80, 8, 1, (9,)),
         ("fp8", 16, 2064, 32, 8, 1, (16,)), ("fp8", 16, 4112, 48, 8, 1, (9, 7)), ("fp8", 13, 8208, 16, 8, 1, (8, 5)),
         ("fp8", 16, 528, 272, 64, 2, (16, 9)), ("fp8", 16, 256, 528, 128, 8, (16, 13, 9, 8, 5)),
         ("fp8", 16, 96, 64, 300, 9, (16, 4, 12)), ("fp8", 7, 1040, 16, 20, 5, (7, 6, 5)),
         ("nvfp4", 5, 128, 128, 8, 1, (5,)), ("nvfp4", 8, 256, 128, 8, 1, (8,)), ("nvfp4", 9, 384, 256, 8, 1, (9,)),
         ("nvfp4", 16, 2176, 128, 8, 1, (16,)), ("nvfp4", 16, 4224, 128, 8, 1, (9, 7)), ("nvfp4", 13, 8320, 128, 7, 1, (8, 5)),
         ("nvfp4", 16, 512, 640, 32, 2, (16, 9)), ("nvfp4", 16, 256, 384, 65, 8, (16, 13, 9, 8, 5)),
         ("nvfp4", 7, 640, 1152, 20, 5, (7, 6, 5))]


@pytest.mark.parametrize("fmt,T,H,I,E,k,counts", CASES)
def test_few_experts_of_many_tokens(fmt, T, H, I, E, k, counts):
    print(f"[case] {fmt} T={T} H={H} I={I} E={E} k={k} counts={counts}", flush=True)
    rng = np.random.default_rng(T * 31 + H + I + E)
    make, call = MAKE[fmt]
    args, w1, w2 = make(rng, E, H, I)
    x = _bf(rng, T, H)
    rows = [[] for _ in range(T)]
    for e, n in enumerate(counts):                        # to the tokens with most room
        for t in sorted(rng.permutation(T), key=lambda t: len(rows[t]))[:n]:
            rows[t].append(e)
    rest = list(range(len(counts), E))
    ids = np.array([rng.permutation(r + list(rng.choice(rest, k - len(r), replace=False)) if len(r) < k else r) for r in rows],
                   np.int32).reshape(T, k)
    if T * k > sum(counts):                               # pairs without an expert among the rest
        ids[(ids >= len(counts)) & (rng.random((T, k)) < 0.3)] = -1
    assert T > 4 and T * k <= 2 * E and [int((ids == e).any(1).sum()) for e in range(len(counts))] == list(counts)
    w = rng.random((T, k)).astype(np.float32)
    dev = x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
    out = call(*dev, *args)
    _check(out, x, ids, w, w1, w2)
    assert torch.equal(call(*dev, *args).view(torch.int16), out.view(torch.int16))
    # a token's result does not hang on the others'
    for t in (0, T - 1):
        one = call(*(a[t:t + 1] for a in dev), *args)
        _check(one, x[t:t + 1], ids[t:t + 1], w[t:t + 1], w1, w2)
