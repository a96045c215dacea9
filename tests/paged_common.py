"""Ragged batches over page pools for the paged operators' tests: seeded pools in shuffled pages, and
each sequence's tokens in order for the oracle.  Slots and pages that hold no token of a sequence
get NaN (dense: every element; q4_0: the scales), which no result may depend on."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

import oracle
from gpu_common import np64

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
NAN_BITS = {torch.float16: 0x7E00, torch.bfloat16: 0x7FC0}


def q4_buffer(x: torch.Tensor) -> torch.Tensor:
    """The q4_0 buffer (uint8, CPU) of a pool [N, H, page, D], by the oracle's quantizer."""
    nib, sc = oracle.quantize_q4_0(x.to(torch.float32).numpy())
    flat = nib.reshape(-1)
    off = (flat.size + 255) // 256 * 256
    buf = np.zeros(off + 2 * sc.size, dtype=np.uint8)
    buf[:flat.size] = flat
    buf[off:] = np.ascontiguousarray(sc).reshape(-1).view(np.uint8)
    return torch.from_numpy(buf)


def q4_planes(buf: torch.Tensor, shape):
    """Views (nibbles [N, H, page, D/2] uint8, scale bits [N, H, page, D/32] int16) of a buffer."""
    n, h, s, d = shape
    nib = n * h * s * d // 2
    off = (nib + 255) // 256 * 256
    return (buf[:nib].view(n, h, s, d // 2),
            buf[off:off + n * h * s * (d // 16)].view(torch.int16).view(n, h, s, d // 32))


@dataclasses.dataclass
class Ragged:
    """A batch: host sizes, and the pools as CPU tensors (dense [N, H, page, D] or q4_0 buffer)."""
    new: list
    lens: list
    shape: tuple
    kf: str
    vf: str
    dtype: str
    table: torch.Tensor
    starts: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor

    def batch(self):
        """(block_table, row_starts, seq_lens) on the device."""
        return (self.table.cuda(), self.starts.cuda(),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))

    def pool(self, fa, side: str):
        t, fmt = (self.k, self.kf) if side == "k" else (self.v, self.vf)
        return t.cuda() if fmt == "dense" else fa.Q4Tensor(t.cuda(), *self.shape)

    def sequence(self, side: str, b: int) -> np.ndarray:
        """[Hkv, len, D] f64: the values of sequence b's tokens in order."""
        t, fmt = (self.k, self.kf) if side == "k" else (self.v, self.vf)
        page, n = self.shape[2], self.lens[b]
        if n == 0:
            return np.zeros((self.shape[1], 0, self.shape[3]))
        ids = [int(self.table[b, p]) for p in range((n + page - 1) // page)]
        if fmt == "dense":
            x = np64(t[ids])
        else:
            nib, sc = q4_planes(t, self.shape)
            x = oracle.dequantize_q4_0(nib[ids].numpy(),
                                       sc[ids].contiguous().numpy().view(np.uint16))
        return np.concatenate(list(x), axis=1)[:, :n]


def make_ragged(new, lens, Hkv, D, page, dtype, kf, vf, seed, *, first_row=0, spare=2,
                poison=True) -> Ragged:
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    pages = [(n + page - 1) // page for n in lens]
    pps = max(1, max(pages))
    N = sum(pages) + spare
    shape = (N, Hkv, page, D)
    perm = torch.randperm(N, generator=g).tolist()
    table = torch.full((B, pps), -7, dtype=torch.int32)  # unused entries are never read
    held = torch.zeros(N, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        for p in range(pages[b]):
            table[b, p] = perm[at]
            held[perm[at], :min(page, n - p * page)] = True
            at += 1
    starts = torch.tensor([first_row + sum(new[:i]) for i in range(B + 1)], dtype=torch.int32)

    def pool(fmt):
        x = torch.randn(shape, generator=g).to(DT[dtype])
        free = (~held)[:, None, :].expand(N, Hkv, page)
        if fmt == "dense":
            if poison:
                x.view(torch.int16)[free] = NAN_BITS[DT[dtype]]
            return x
        buf = q4_buffer(x)
        if poison:
            q4_planes(buf, shape)[1][free] = 0x7E00
        return buf

    k, v = pool(kf), pool(vf)
    return Ragged(list(new), list(lens), shape, kf, vf, dtype, table, starts, k, v)
