"""Random paged caches for the tests of attn_sink_cache.h, on the CPU."""
from __future__ import annotations

import torch

BF16 = torch.bfloat16


class Paged:
    """Sequences of these lengths over a cache of random pages, rows without a key holding
    infinities and NaN."""

    def __init__(self, seed, lens, *, hq=8, hkv=2, page=16, spare=3, cols=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.page = list(lens), hq, hkv, page
        count = [-(-n // page) for n in lens]
        self.cols = max(count, default=0) + 1 if cols is None else cols
        self.pages = sum(count) + spare
        perm = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), self.cols), -1, dtype=torch.int32)
        self.free = perm[sum(count):].tolist()
        at = 0
        used = torch.zeros(self.pages, page, dtype=torch.bool)
        for b, (n, c) in enumerate(zip(lens, count)):
            self.table[b, :c] = perm[at:at + c]
            for col in range(c):
                used[int(perm[at + col]), : min(page, n - col * page)] = True
            at += c
        odd = torch.tensor([float("inf"), float("nan"), -float("inf"), 3e38])
        self.k, self.v = (torch.randn(self.pages, page, hkv, 64, generator=g).to(BF16)
                          for _ in range(2))
        for x in (self.k, self.v):
            x[~used] = odd[torch.randint(0, 4, x[~used].shape, generator=g)].to(BF16)
        self.sink = torch.randn(hq, generator=g)

    def q(self, rows=None, scale=1.0):
        rows = len(self.lens) if rows is None else rows
        return (scale * torch.randn(rows, self.hq, 64, generator=self.g)).to(BF16)

    def lens_gpu(self):
        return ints(self.lens)

    def gpu(self):
        return self.k.cuda(), self.v.cuda(), self.table.cuda(), self.lens_gpu()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
