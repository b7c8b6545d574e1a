"""Linear layers that answer from quantised weights, for inference.

``CodedLinear`` holds a layer as the packed hard code that training ends in, ``Int4Linear`` as 4-bit
codes with a scale for each group of columns, the round-to-nearest baseline that needs no training.
Both are called on x [..., cols] in fp32, fp16 or bf16 and return [..., rows] of that type; the
weights are decoded inside the product and never written out. They give no gradients.
"""
from __future__ import annotations

import torch

from . import bcjr


def _products(call, x, rows, cols):
    if x.shape[-1] != cols:
        raise ValueError(f"x has {x.shape[-1]} columns, the layer {cols}")
    x2 = x if x.dim() == 2 else x.reshape(-1, cols)
    if x2.dim() == 2 and cols > 1 and (x2.stride(1) != 1 or x2.stride(0) < cols):
        x2 = x2.contiguous()
    y = call(x2)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], rows)


class CodedLinear:
    """A [rows, cols] layer cut row-major into trellis chains of L weights (whole chains in a row).

    code uint32 [rows cols / L, words] as ``bcjr.bcjr_pack_code`` gives it; codebook fp32 [2^n]; scales
    fp32 [rows cols / L], a factor for each chain, or None."""

    def __init__(self, code, codebook, n: int, k: int, L: int, cols: int, scales=None):
        if cols < 1 or L < 1 or cols % L or code.shape[0] % (cols // L):
            raise ValueError(f"{code.shape[0]} chains of {L} weights are no whole rows of {cols} columns")
        self.code, self.codebook, self.scales = code, codebook, scales
        self.n, self.k, self.L, self.cols, self.rows = n, k, L, cols, code.shape[0] // (cols // L)

    @classmethod
    def from_weights(cls, w, codebook, n: int, k: int, L: int, scales=None):
        """The Viterbi code of latent weights w fp32 [rows, cols], which are in the codebook's units: a
        chain's scale is not divided out."""
        rows, cols = w.shape
        if cols % L:
            raise ValueError(f"rows of {cols} weights do not cut into chains of {L}")
        states, _ = bcjr.viterbi_decode(codebook, w.reshape(-1, L).contiguous(), n, k, want_w_hard=False)
        return cls(bcjr.bcjr_pack_code(states, n, k), codebook, n, k, L, cols, scales)

    def __call__(self, x):
        return _products(lambda x2: bcjr.bcjr_code_matvec(x2, self.code, self.codebook, self.n, self.k, self.L, self.scales),
                         x, self.rows, self.cols)

    def weights(self):
        """The weights the code stands for, fp32 [rows, cols]."""
        _, w = bcjr.bcjr_unpack_code(self.code, self.n, self.k, self.L, codebook=self.codebook)
        return (w if self.scales is None else w * self.scales[:, None]).view(self.rows, self.cols)

    def nbytes(self) -> int:
        """Bytes of code and scales (the codebook is shared by a model's layers)."""
        return 4 * self.code.numel() + (0 if self.scales is None else 4 * self.scales.numel())


class Int4Linear:
    """A [rows, cols] layer of 4-bit codes; the parts as ``bcjr.bcjr_int4_quantize`` gives them."""

    def __init__(self, q, scales, zeros, cols: int, group: int):
        bcjr._int4_weights(q, scales, zeros, cols, bcjr._group(group))
        self.q, self.scales, self.zeros = q, scales, zeros
        self.cols, self.group, self.rows = cols, group, q.shape[0]

    @classmethod
    def from_weights(cls, w, group: int = 128, zeros: bool = False):
        """w [rows, cols] rounded to nearest, with zero points or symmetric."""
        q, scales, z = bcjr.bcjr_int4_quantize(w, group, zeros)
        return cls(q, scales, z, w.shape[1], group)

    def __call__(self, x):
        return _products(lambda x2: bcjr.bcjr_int4_matvec(x2, self.q, self.scales, self.zeros, self.group), x, self.rows, self.cols)

    def weights(self):
        """The weights the codes stand for, fp32 [rows, cols]."""
        return bcjr.bcjr_int4_dequantize(self.q, self.scales, self.zeros, self.cols, self.group)

    def nbytes(self) -> int:
        return 4 * self.q.numel() + 4 * self.scales.numel() + (0 if self.zeros is None else self.zeros.numel())
