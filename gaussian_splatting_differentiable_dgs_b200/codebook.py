"""Colours shared through a codebook.

Every Gaussian's spherical-harmonics coefficients are a row of one table,
scaled: sh_i = scale * table[codes[i]].  The table is trained in place of the
coefficients: its gradient sums those of all Gaussians with the same code, and
Adam runs over its rows.  A scene's 3 (D+1)^2 colour parameters per Gaussian
become one int32 code.

The model's SH planes always hold the decoded colours, so projection and
rendering read them as they do without a codebook.  Hand the codebook to the
Stepper:

    codebook = ColorCodebook(table, codes)
    stepper = Stepper(model, codebook=codebook)
"""
from __future__ import annotations

import torch

from . import binding as B

SH_PLANE = 11  # first SH plane of the model

INTEGERS = (torch.int8, torch.int16, torch.int32, torch.int64, torch.uint8, torch.uint16,
            torch.uint32, torch.bool)


class ColorCodebook:
    """table: [K][3 (D+1)^2] fp32 rows (coefficient k, channel c at 3 k + c,
    the order of the model's SH planes), copied to the device; codes: [n]
    integers in [0, K), or negative for a Gaussian without colour
    coefficients (its SH planes are zero).  Holds Adam's moments of the table
    and its gradient.  Calls on different streams are ordered by the caller,
    as for any tensor: they share the table and self.grad."""

    def __init__(self, table, codes, scale: float = 1.0, device="cuda"):
        self.table = torch.as_tensor(table, dtype=torch.float32).to(device).contiguous().clone()
        if self.table.dim() != 2:
            raise ValueError(f"table must be [K][coefficients], not {tuple(self.table.shape)}")
        codes = torch.as_tensor(codes)
        if codes.dim() != 1 or codes.dtype not in INTEGERS:
            raise ValueError("codes must be a 1-D array of integers (of up to 32 bits, or int64)")
        codes = codes.to(torch.int64)
        if codes.numel() and int(codes.max()) >= self.table.shape[0]:
            raise ValueError(f"code {int(codes.max())} of a table of {self.table.shape[0]} rows")
        # every negative code means the same; one below -2^31 would wrap
        self.codes = codes.clamp(min=-1).to(torch.int32).to(device).contiguous()
        self.scale = float(scale)
        self.m = torch.zeros_like(self.table)
        self.v = torch.zeros_like(self.table)
        self.grad = torch.zeros_like(self.table)

    @property
    def rows(self):
        return self.table.shape[0]

    @property
    def cols(self):
        return self.table.shape[1]

    def check(self, model):
        """Raises if the codebook does not fit the model."""
        if self.cols != model.P - SH_PLANE:
            raise ValueError(f"a table of {self.cols} columns for {model.P - SH_PLANE} SH planes")
        if self.codes.numel() != model.n:
            raise ValueError(f"{self.codes.numel()} codes for {model.n} Gaussians")

    def decode(self, model, dev_status=None, stream=None):
        """Writes the colours of all Gaussians into the model's SH planes (after
        the table or the codes were changed by hand; the Stepper does it after
        every update)."""
        B.gs_lookup(self.table, self.codes, model.params[SH_PLANE:, :model.n].t(),
                    scale=self.scale, dev_status=dev_status, stream=stream)

    def gradient(self, g, cand_idx=None, dev_status=None, stream=None):
        """The table's gradient (self.grad) from the gradient of the SH planes,
        g: [planes][C] of the candidates cand_idx (or of all Gaussians).  Its
        workspace (about 4 C (planes + 5) bytes where the table has more than
        1024 rows) is taken from the caching allocator for the call, on the
        call's own stream: nothing outlives the call, a later call on another
        stream cannot be given memory that this one still uses, and the view
        step counts it in its working set."""
        g = g.t()
        need = B.gs_lookup_bwd_workspace_size(g, self.rows)
        # in steps of an eighth, so that views of similar size share a block
        step = 1 << max(need.bit_length() - 4, 8)
        with torch.cuda.stream(self._on(stream)):
            ws = torch.empty(-(-need // step) * step, dtype=torch.uint8, device=self.table.device)
        return B.gs_lookup_bwd(g, self.codes, self.grad, ws, scale=self.scale,
                               index=cand_idx, dev_status=dev_status, stream=stream)

    def _on(self, stream):
        """`stream` as torch knows streams (a raw handle, 0 among them, too)."""
        if stream is None or not isinstance(stream, int):
            return stream
        if stream == 0:
            return torch.cuda.default_stream(self.table.device)
        return torch.cuda.ExternalStream(stream, device=self.table.device)
