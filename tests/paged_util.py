"""Seeded paged caches for the tests: a pool on the host (numpy), the page
table of a ragged batch with its pages in random order, and the same on the
device as a ``PagedKV``."""
import numpy as np
import torch

from oracle import qg_oracle as O
from tests.gpu_util import bf16_dev, dev

BLOCK = O.KV_BLOCK


def bf16_bits(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).view(
        torch.int16).numpy().view(np.uint16).copy()


class Cache:
    """Host pool of B sequences that can hold ``cap`` tokens each. ``lens``
    of them are filled; all other contents are junk that must not matter:
    codes of any value and NaN scales, or NaN rows in bf16."""

    def __init__(self, kind, B, Hkv, D, page, cap, lens, seed, spare=2):
        rng = np.random.default_rng(seed)
        self.kind, self.B, self.Hkv, self.D, self.page = kind, B, Hkv, D, page
        self.max_pages = (max(cap, 1) + page - 1) // page
        P = B * self.max_pages + spare
        self.table = rng.permutation(P)[:B * self.max_pages].reshape(B, -1).astype(np.int32)
        self.k, self.ks = self._fill(rng, P, lens)
        self.v, self.vs = self._fill(rng, P, lens)

    def _fill(self, rng, P, lens):
        shape = (P, self.Hkv, self.page, self.D)
        if self.kind == "int8":
            codes = rng.integers(-128, 128, shape).astype(np.int8)
            scales = np.full(shape[:2] + (self.page // BLOCK,), np.nan, np.float32)
        else:
            codes, scales = np.full(shape, 0x7FC0, np.uint16), None
        for b in range(self.B):
            for t in range(int(lens[b])):
                p, r = self.table[b, t // self.page], t % self.page
                if self.kind == "int8":
                    codes[p, :, r] = np.clip(np.rint(rng.standard_normal((self.Hkv, self.D)) * 40),
                                             -127, 127)
                    if t % BLOCK == 0:
                        scales[p, :, r // BLOCK] = 0.02 + 0.03 * rng.random(self.Hkv)
                else:
                    codes[p, :, r] = bf16_bits(rng.standard_normal((self.Hkv, self.D)))
        return codes, scales

    def place(self, b, t):
        return self.table[b, t // self.page], t % self.page

    def values(self, b, L):
        """Sequence b's first L tokens in float64: (k, v), each [Hkv, L, D]."""
        out = []
        for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
            x = np.zeros((self.Hkv, L, self.D))
            for t in range(L):
                p, r = self.place(b, t)
                if self.kind == "int8":
                    x[:, t] = codes[p, :, r].astype(np.float64) * \
                        scales[p, :, r // BLOCK].astype(np.float64)[:, None]
                else:
                    x[:, t] = O.bf16_bits_to_f64(codes[p, :, r])
            out.append(x)
        return out

    def upload(self, qg, device="cuda"):
        """(PagedKV, page table) on the device."""
        if self.kind == "int8":
            t = [torch.from_numpy(a.copy()).to(device) for a in (self.k, self.v, self.ks, self.vs)]
        else:
            t = [bf16_dev(self.k, device), bf16_dev(self.v, device)]
        return qg.PagedKV(*t), dev(self.table, device)

    def download(self, kv):
        """The device pool's contents as this class holds them."""
        if self.kind == "int8":
            return [t.cpu().numpy() for t in (kv.k_pages, kv.k_scales, kv.v_pages, kv.v_scales)]
        return [kv.k_pages.view(torch.int16).cpu().numpy().view(np.uint16), None,
                kv.v_pages.view(torch.int16).cpu().numpy().view(np.uint16), None]


def starts(n):
    return np.concatenate(([0], np.cumsum(n))).astype(np.int32)
