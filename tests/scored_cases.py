"""Caches with unwritten positions and random trees for the attn_scored, attn_tree
and tree_accept tests."""
import numpy as np

from compressed_kv_attention_gb300 import inputs
from oracle import ckv_oracle as O
from tests import helpers as H


class Cache:
    """A packed cache on the GPU whose sequence b holds positions [start[b], len[b]); every other byte is 0xFF (NaN
    scales and norms). ``k`` and ``v`` are the dequantised contents in float64, [B][Hkv, len, D]."""

    def __init__(self, D, Hkv, lens, capacity, bits=3, rot=False, start=None, seed=0):
        import torch

        import compressed_kv_attention_gb300 as ckv
        B = len(lens)
        s1, s2 = inputs.tbq_signs(D), inputs.tbq_signs(D, 43) if rot else None
        self.packed = ckv.PackedCache(D, Hkv, B, capacity, s1, v_bits=bits, signs2=s2)
        self.packed.data.fill_(0xFF)
        nbytes, groups = self.packed.data.numel() // B, D // 128 if rot else 1
        self.bits, self.groups, self.D, self.Hkv, self.capacity = bits, groups, D, Hkv, capacity
        outl = inputs.outlier_channels(D, max(1, D // 100), seed)
        for b, T in enumerate(lens):
            first = start[b] if start else 0
            if T > first:
                one = ckv.PackedCache(D, Hkv, 1, capacity, s1, v_bits=bits, signs2=s2,
                                      data=self.packed.data[b * nbytes:(b + 1) * nbytes])
                k = inputs.normal_tensor((1, T - first, Hkv, D), seed + b, "k", outl)
                v = inputs.normal_tensor((1, T - first, Hkv, D), seed + b, "v", outl[:0])
                ckv.kv_pack(one, first, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
        self.s1, self.s2, self.lens, self.start = s1, s2, list(lens), start
        self.read()

    def records(self):
        return self.packed.data.cpu().numpy().reshape(len(self.lens), self.Hkv, self.capacity // 16, -1)

    def fields(self, b, h, T):
        return H.read_fields(self.records()[b, h], self.D, T, self.bits, self.groups)

    def read(self):
        self.k, self.v = [], []
        rec = self.records()
        for b, T in enumerate(self.lens):
            ks, vs = np.zeros((self.Hkv, T, self.D)), np.zeros((self.Hkv, T, self.D))
            first = self.start[b] if self.start else 0
            for h in range(self.Hkv):
                if T > first:
                    qs, d, c, n = (x[first:] for x in H.read_fields(rec[b, h], self.D, T, self.bits, self.groups))
                    ks[h, first:] = O.q8_0_dequantize(qs, d.view(np.float16))
                    n = np.ascontiguousarray(n).view(np.float16)
                    vs[h, first:] = (O.tbq_dequantize(c, n, self.s1, self.bits) if self.s2 is None
                                     else O.tbq_dequantize_blocked(c, n.reshape(len(n), -1), self.s1, self.s2, self.bits))
            self.k.append(ks)
            self.v.append(vs)


def random_tree(n, rng, width=3):
    """Masks (uint64) of a random tree of n nodes, parents before children."""
    m = np.zeros(n, np.uint64)
    for i in range(n):
        parent = int(rng.integers(max(0, i - width), i)) if i else -1
        m[i] = np.uint64(1 << i) | (m[parent] if i else np.uint64(0))
    return m
