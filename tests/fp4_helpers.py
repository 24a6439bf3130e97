"""The latent cache in 4 bits for tests: its rows packed and unpacked by look-up
in 64 bits, and a bf16 cache of the values that a 4-bit one stands for."""
import numpy as np
import torch

import edge_moe_serving_gb300 as moe
from kv_helpers import DEV, Paged

SIZES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([m * 2.0 ** -17 for m in range(8)] +
                  [(8 + m) * 2.0 ** (e - 18) for e in range(1, 31) for m in range(8)])


def nearest(x, values):
    """Index of the nearest of ascending values to each x >= 0, the even one of two equally near, the last beyond it."""
    hi = np.minimum(np.searchsorted(values, x), len(values) - 1)
    lo = np.maximum(hi - 1, 0)
    a, b = x - values[lo], values[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def row_bytes(rank, rope):
    n = rank // 2 + 2 * rope + rank // 16
    return -(-n // 16) * 16


def pack(rows, rank, rope):
    """bf16 rows [n, rank + rope] on the CPU -> bytes [n, row bytes]."""
    x = rows.double().numpy()
    lat = x[:, :rank].reshape(len(x), rank // 16, 16)
    ok = np.isfinite(lat).all(-1)
    lat = np.where(ok[..., None], lat, 0.0)
    scale = nearest(np.abs(lat).max(-1) / 6, SCALES)
    s = SCALES[scale][..., None]
    code = nearest(np.abs(lat) / np.where(s > 0, s, 1.0), SIZES) + 8 * np.signbit(lat)
    code = np.where(s > 0, code, 0).reshape(len(x), rank)
    scale = np.where(ok, scale, 255)
    out = np.zeros((len(x), row_bytes(rank, rope)), np.uint8)
    out[:, :rank // 2] = code[:, 0::2] + 16 * code[:, 1::2]
    at = rank // 2 + 2 * rope
    if rope and len(x):
        out[:, rank // 2:at] = rows[:, rank:].contiguous().view(torch.uint8).numpy()
    out[:, at:at + rank // 16] = scale
    return torch.from_numpy(out)


def unpack(data, rank, rope):
    """Bytes [n, row bytes] on the CPU -> the values in 64 bits [n, rank + rope]."""
    b = data.numpy()
    at = rank // 2 + 2 * rope
    code = np.stack([b[:, :rank // 2] & 15, b[:, :rank // 2] >> 4], -1).reshape(len(b), rank)
    scale = np.concatenate([SCALES, np.full(8, np.nan)])[b[:, at:at + rank // 16]]
    v = SIZES[code & 7] * np.where(code & 8, -1.0, 1.0) * np.repeat(scale, 16, 1)
    r = np.zeros((len(b), rope))
    if r.size:
        r = data[:, rank // 2:at].contiguous().view(torch.bfloat16).double().numpy()
    return torch.from_numpy(np.concatenate([v, r], 1))


class Paged4(Paged):
    """A cache in 4 bits: every byte of its pages starts as 255, NaN wherever it is read as a scale or a rotary key."""

    def __init__(self, n_pages, page, rank, rope, max_seqs, max_blocks, layers=1, device=DEV):
        super().__init__(n_pages, page, rank, rope, max_seqs, max_blocks, layers, device)
        self.bytes = moe.moe_kv_row_bytes(rank, rope, moe.MOE_KV_FP4)
        self.bf16 = self.pages
        self.pages = torch.full((layers, n_pages, page, self.bytes), 255, dtype=torch.uint8, device=device)
        self.handle.pages = self.pages.data_ptr()
        self.handle.format = moe.MOE_KV_FP4

    def fill(self, lens, seed=0, layer=0, shared_blocks=0, spread=1.0):
        """As Paged.fill, the rows packed without the library; the bf16 pages keep what the packed ones stand for.
        Returns those values in 64 bits, per sequence."""
        packed, self.pages = self.pages, self.bf16
        rows = super().fill(lens, seed, layer, shared_blocks, spread)
        self.pages = packed
        out = []
        for i, x in enumerate(rows):
            data = pack(x.to(torch.bfloat16), self.rank, self.rope)
            values = unpack(data, self.rank, self.rope)
            for b in range(-(-len(x) // self.page)):
                p, part = int(self.table[i, b]), slice(b * self.page, (b + 1) * self.page)
                n = len(data[part])
                self.pages[layer, p, :n] = data[part].to(self.pages.device)
                self.bf16[layer, p, :n] = values[part].to(torch.bfloat16).to(self.pages.device)
            out.append(values)
        return out

    def twin(self):
        """The bf16 cache of the same values and the same tables."""
        h = self.handle
        t = Paged.__new__(Paged)
        t.__dict__.update(self.__dict__)
        t.pages = self.bf16
        t.handle = moe.moe_kv_cache(self.bf16.data_ptr(), h.table, h.lens, h.refs, h.n_layers, h.n_pages, h.page_tokens,
                                    h.rank, h.rope, h.max_seqs, h.max_blocks, moe.MOE_KV_BF16)
        return t
